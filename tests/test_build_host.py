"""The build of the short calls' extension: what it is compiled against, and what a build does that cannot
make it.  Compilers are stand-ins."""
import os
import subprocess
import types

import pytest

from mixture_experts_routed_gate_gb300 import _build, binding


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A tree of its own with an up-to-date library, and a compiler that writes what it is told to."""
    build, pkg = tmp_path / "_build", tmp_path / "pkg"
    build.mkdir(), pkg.mkdir()
    monkeypatch.setattr(_build, "BUILD", str(build))
    monkeypatch.setattr(_build, "PKG", str(pkg))
    monkeypatch.setattr(_build, "LIB", str(pkg / "lib.so"))
    monkeypatch.setattr(_build, "HOST_LIB", str(pkg / "_host_calls.so"))
    monkeypatch.setattr(_build, "HOST_DONE", str(build / "host_calls.done"))
    (pkg / "lib.so").write_text("library")
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(_build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return types.SimpleNamespace(run=run, ran=ran, lib=pkg / "_host_calls.so", done=build / "host_calls.done")


def test_built_once(place):
    _build.build()
    assert place.lib.read_text() == "built" and len(place.ran) == 2 and not _build.host_is_stale()
    _build.build()
    assert len(place.ran) == 2


def test_another_pytorch_or_python(place, monkeypatch):
    """An extension of another PyTorch is built anew."""
    _build.build()
    key = _build.host_key()
    monkeypatch.setattr(_build, "host_key", lambda: "another")
    assert key != "another" and _build.host_is_stale()
    _build.build()
    assert len(place.ran) == 4 and not _build.host_is_stale() and '-DMOE_BUILT_FOR="another"' in place.ran[2]


def test_the_key_is_pytorchs_version(tmp_path, monkeypatch):
    keys = []
    for version in ("1", "2", "1"):
        (tmp_path / "version.py").write_text(version)
        monkeypatch.setattr(_build, "_torch_dir", lambda: str(tmp_path))
        keys.append(_build.host_key())
    assert keys[0] == keys[2] != keys[1]
    monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: ".another.so")
    assert _build.host_key() not in keys


def test_an_extension_of_another_pytorch_is_not_used(monkeypatch):
    _build.build()
    lib, host = binding.lib(), binding._host
    assert host is not None and host.built_for == _build.host_key()
    monkeypatch.setattr(_build, "host_key", lambda: "another")
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_host", None)
    with pytest.warns(UserWarning, match="another PyTorch"):
        binding.lib()
    assert binding._host is None and binding._lib._name == lib._name


@pytest.mark.parametrize("fails", ["-c", "-shared"])
def test_a_build_that_failed_is_tried_again(place, monkeypatch, capsys, fails):
    """Neither an extension nor a stamp stays behind a failed compile or link; the next build makes both."""
    _build.build()
    assert place.lib.exists()
    place.lib.with_name("lib.so").write_text("a newer library")
    os.utime(place.lib.with_name("lib.so"), ns=(1 << 62, 1 << 62))
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "no such header")
                        if fails in cmd else place.run(cmd, **kw))
    _build.build()
    assert "no such header" in capsys.readouterr().out and not place.lib.exists() and not place.done.exists()
    os.utime(place.lib.with_name("lib.so"))
    monkeypatch.setattr(subprocess, "run", place.run)
    _build.build()
    assert place.lib.exists() and place.done.exists() and not _build.host_is_stale()


def test_pytorch_that_comes_later(place, monkeypatch):
    """Without PyTorch there is nothing to build, and nothing says that it was built."""
    with monkeypatch.context() as m:
        m.setattr(_build, "_torch_dir", lambda: None)
        _build.build()
    assert not place.ran and not place.lib.exists()
    _build.build()
    assert len(place.ran) == 2 and place.lib.exists()


@pytest.mark.parametrize("missing", ["g++", "nvcc", "the linker"])
def test_without_a_compiler(place, monkeypatch, capsys, missing):
    """An up-to-date library and no g++ or no CUDA toolkit: the build says so and goes on without the extension."""
    def run(cmd, **kw):
        if missing == "g++" or (missing == "the linker" and "-shared" in cmd):
            raise FileNotFoundError(2, "No such file or directory", cmd[0])
        return place.run(cmd, **kw)

    def nvcc():
        if missing == "nvcc":
            raise RuntimeError("nvcc not found")
        return "/usr/local/cuda/bin/nvcc"
    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(_build, "nvcc", nvcc)
    assert _build.build() == _build.LIB
    told = capsys.readouterr().out
    assert "goes without it" in told and ("nvcc not found" if missing == "nvcc" else "No such file") in told
    assert not place.lib.exists() and not place.done.exists()


def test_two_builds_at_once(place, monkeypatch):
    """A build from another process in the middle of this one, at every step of it: both end well, and neither
    takes away what the other made."""
    for step in range(2):
        for old in (place.lib, place.done):
            old.unlink(missing_ok=True)
        others, pid = [], os.getpid()

        def run(cmd, **kw):
            if len(others) == 0 and ("-shared" in cmd) == (step == 1):
                others.append(cmd)
                with monkeypatch.context() as m:  # the other process
                    m.setattr(os, "getpid", lambda: pid + 1)
                    _build.build()
                assert place.lib.exists() and place.done.exists()
            return place.run(cmd, **kw)
        monkeypatch.setattr(subprocess, "run", run)
        _build.build()
        assert others and place.lib.read_text() == "built" and not _build.host_is_stale()
    made = [cmd[cmd.index("-o") + 1] for cmd in place.ran]
    assert len(set(made)) == 4 and not [n for n in os.listdir(place.done.parent) if n.endswith(".o")]


def test_what_another_build_has_removed(place, monkeypatch):
    """Two failed builds remove the same files."""
    _build.build()
    monkeypatch.setattr(_build, "_host_object", lambda: None)
    exists = os.path.exists
    monkeypatch.setattr(os.path, "exists", lambda p: True if str(p).startswith(str(place.lib.parent)) else exists(p))
    _build._link_host(None)
    _build._link_host(None)
    monkeypatch.undo()
    assert not place.lib.exists()
