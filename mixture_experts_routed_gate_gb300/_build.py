"""Builds ``libmoe_routed_gb300.so`` in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` is compiled in parallel to an object under ``_build/`` and
the objects are linked into one shared library next to this file.  A rebuild
happens only when a source or header is newer than the library.

``csrc/host_calls.cpp``, the binding's shortest calls as a Python extension, is
compiled beside them against PyTorch's headers.  The binding makes the same calls
without it, so where it cannot be built the compiler's words are printed and
the build goes on.
"""
from __future__ import annotations

import concurrent.futures
import contextlib
import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "moe_routed_gb300")
LIB = os.path.join(PKG, "libmoe_routed_gb300.so")
HOST_SRC = os.path.join(CSRC, "host_calls.cpp")
HOST_LIB = os.path.join(PKG, "_host_calls.so")
HOST_DONE = os.path.join(BUILD, "host_calls.done")  # host_key() of the extension there is

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fvisibility=hidden"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None and spec.submodule_search_locations else None


def host_key() -> str:
    """The PyTorch and the Python that the extension is compiled against, whose layouts it holds: it is
    loaded by these alone."""
    parts, where = [sys.version, str(sysconfig.get_config_var("EXT_SUFFIX"))], _torch_dir()
    if where is not None:
        with open(os.path.join(where, "version.py")) as f:
            parts.append(f.read())
    return hashlib.sha256("\0".join(parts).encode()).hexdigest()


def host_is_stale() -> bool:
    if not os.path.exists(HOST_DONE) or not os.path.exists(HOST_LIB):
        return True
    with open(HOST_DONE) as f:
        if f.read() != host_key():
            return True
    t = os.path.getmtime(HOST_DONE)
    return any(os.path.getmtime(p) > t for p in [HOST_SRC, LIB, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h")))


def _run(cmd) -> str | None:
    """What went wrong with a command; None if nothing."""
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:  # there is no such program, say
        return str(e)
    return None if r.returncode == 0 else r.stderr[-2000:] or f"exit code {r.returncode}"


def _host_object() -> str | None:
    """host_calls.cpp compiled; None where PyTorch, a header or a compiler is missing."""
    where = _torch_dir()
    if where is None:
        return None
    torch_inc = os.path.join(where, "include")
    try:
        cuda_inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    except RuntimeError as e:
        print(f"host_calls.cpp not built (the binding goes without it):\n{e}")
        return None
    obj = os.path.join(BUILD, f"host_calls.{os.getpid()}.o")  # several processes may build at once
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f'-DMOE_BUILT_FOR="{host_key()}"',
           "-I", torch_inc, "-I", os.path.join(torch_inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"], "-I", cuda_inc, "-c", HOST_SRC, "-o", obj]
    wrong = _run(cmd)
    if wrong is not None:
        print(f"host_calls.cpp not built (the binding goes without it):\n{wrong}")
        return None
    return obj


def _remove(*paths) -> None:
    for path in paths:
        with contextlib.suppress(FileNotFoundError):  # another process may have been faster
            os.remove(path)


def _link_host(obj: str | None) -> None:
    """The extension from its object; none at all where there is no object or it cannot be linked, so that the
    next build tries again."""
    if obj is None:
        _remove(HOST_DONE, HOST_LIB)
        return
    torch_lib = os.path.join(_torch_dir(), "lib")
    tmp = HOST_LIB + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:" + os.path.basename(LIB), "-L", torch_lib, "-ltorch_python", "-ltorch_cpu",
           "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    wrong = _run(cmd)
    _remove(obj)
    if wrong is not None:
        _remove(HOST_DONE, HOST_LIB, tmp)
        print(f"host_calls not linked (the binding goes without it):\n{wrong}")
        return
    os.replace(tmp, HOST_LIB)
    done = HOST_DONE + f".tmp{os.getpid()}"
    with open(done, "w") as f:
        f.write(host_key())
    os.replace(done, HOST_DONE)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if not force and not is_stale():
        if host_is_stale():
            _link_host(_host_object())
        return LIB
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            print(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        host = ex.submit(_host_object)
        objs = list(ex.map(compile_one, srcs))
        host = host.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fvisibility=hidden"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_host(host)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
