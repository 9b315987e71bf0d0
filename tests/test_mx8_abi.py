"""Host-side checks of the 8-bit entry points and of the combine's gradient:
every refusal happens before any CUDA call, so none of this needs a GPU."""
import ctypes

import pytest

from mixture_experts_routed_gate_gb300 import _build, binding

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F16, BF16, F32, E4M3 = 0, 1, 2, 3
NONE = ctypes.c_size_t(-1).value
A = 0x1000  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.lib()


def norm(lib, y=A, res=A, w_post=A, gate=None, kind=0, alpha=1.0, w_next=A, eps=1e-6, T=4, H=64, dtype=BF16, out=A, u=A, q=A, sf=A,
         r_post=None, r_next=None):
    return lib.moe_residual_norm_mx8(y, res, w_post, gate, kind, alpha, w_next, eps, T, H, dtype, out, u, q, sf, r_post, r_next, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=E4M3), UNSUPPORTED), (dict(H=48), INVALID), (dict(H=0), INVALID), (dict(H=16416), UNSUPPORTED), (dict(T=-1), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID), (dict(alpha=float("nan")), INVALID),
    (dict(kind=4), INVALID), (dict(kind=1), INVALID), (dict(gate=A), INVALID), (dict(res=None), INVALID), (dict(out=None), INVALID),
    (dict(w_next=None), INVALID), (dict(q=None), INVALID), (dict(sf=None), INVALID), (dict(y=None, out=None), INVALID),
    (dict(w_post=None, r_post=A), INVALID), (dict(y=A + 8), INVALID), (dict(u=A + 2), INVALID), (dict(q=A + 8), INVALID),
    (dict(T=0), OK), (dict(T=0, y=None, res=None, out=None, q=None, sf=None), OK),
])
def test_residual_norm(lib, change, status):
    assert norm(lib, **change) == status


def backward(lib, d_out=A, x=A, n=8, pos=A, w=A, token=A, T=4, K=2, H=256, din=BF16, dout=BF16, d_x=A, d_w=A):
    return lib.moe_reduce_fused_backward(d_out, x, n, pos, w, token, T, K, H, din, dout, d_x, d_w, None, None)


@pytest.mark.parametrize("change,status", [
    (dict(H=255), INVALID), (dict(H=0), INVALID), (dict(H=1 << 21), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=33), INVALID),
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(n=1 << 31), UNSUPPORTED), (dict(din=F16), UNSUPPORTED), (dict(dout=F16), UNSUPPORTED),
    (dict(dout=F32), UNSUPPORTED), (dict(din=E4M3, dout=E4M3), UNSUPPORTED), (dict(din=E4M3), UNSUPPORTED), (dict(d_out=None), INVALID),
    (dict(x=None), INVALID), (dict(pos=None), INVALID), (dict(token=None), INVALID), (dict(d_x=None), INVALID), (dict(x=A + 8), INVALID),
    (dict(d_x=A + 4), INVALID), (dict(d_out=A + 2), INVALID), (dict(n=0, T=0), OK), (dict(n=0, T=0, d_out=None, x=None, d_x=None), OK),
])
def test_reduce_fused_backward(lib, change, status):
    assert backward(lib, **change) == status


def test_quantise_and_sort(lib):
    q = lambda x=A, n=4, K=64, dt=BF16, o=A, s=A: lib.moe_quantize_mx8(x, n, K, dt, o, s, None)  # noqa: E731
    assert q(K=48) == INVALID and q(K=0) == INVALID and q(n=-1) == INVALID and q(dt=E4M3) == UNSUPPORTED and q(K=1 << 21) == UNSUPPORTED
    assert q(x=None) == INVALID and q(o=None) == INVALID and q(s=None) == INVALID and q(x=A + 8) == INVALID and q(o=A + 4) == INVALID
    assert q(n=0) == OK and q(n=1 << 31) == UNSUPPORTED
    d = lambda n=4, K=64, dt=F32, o=A, s=A: lib.moe_dequantize_mx8(A, s, n, K, dt, o, None)  # noqa: E731
    assert d(K=33) == INVALID and d(dt=E4M3) == UNSUPPORTED and d(o=None) == INVALID and d(o=A + 8) == INVALID and d(n=0) == OK
    assert d(s=None) == INVALID
    r = lambda q=A, s=A, p=A, T=4, k=2, n=8, K=64, o=A, so=A: lib.moe_sort_rows_mx8(q, s, p, T, k, n, K, o, so, None)  # noqa: E731
    assert r(K=48) == INVALID and r(k=0) == INVALID and r(k=33) == INVALID and r(T=-1) == INVALID and r(n=-1) == INVALID
    assert r(q=None) == INVALID and r(s=None) == INVALID and r(p=None) == INVALID and r(o=None) == INVALID and r(so=None) == INVALID
    assert r(q=A + 8) == INVALID and r(o=A + 8) == INVALID and r(K=1 << 21) == UNSUPPORTED and r(n=1 << 31) == UNSUPPORTED
    assert r(T=0, q=None) == OK and r(n=0, o=None) == OK


def test_products_and_forward(lib):
    def gemm(a=A, b=A, mb=3, rows=8, N=128, K=64, E=8, dt=BF16, c=A, g=A):
        return lib.moe_grouped_gemm_mx8(a, A, b, A, A, A, A, g, mb, rows, N, K, E, dt, c, None, None)
    assert gemm(K=48) == INVALID and gemm(N=0) == INVALID and gemm(dt=E4M3) == UNSUPPORTED and gemm(mb=99) == INVALID
    assert gemm(a=None) == INVALID and gemm(b=A + 8) == INVALID and gemm(c=None) == INVALID and gemm(rows=0) == OK and gemm(g=None) == INVALID
    assert gemm(N=1 << 21) == UNSUPPORTED and gemm(rows=1 << 31) == UNSUPPORTED and gemm(E=0) == INVALID

    def up(d_h=64, d_e=64, q_h=A, sf_h=A, mb=3):
        return lib.moe_grouped_gate_up_silu_mx8(A, A, A, A, A, A, A, A, A, A, mb, 8, d_h, d_e, 8, q_h, sf_h, None, None)
    assert up(d_e=48) == INVALID and up(d_h=40) == INVALID and up(q_h=None) == INVALID and up(q_h=A + 8) == INVALID
    assert up(sf_h=None) == INVALID and up(mb=0) == INVALID

    def fwd(T=4, q=None, sf=None, d_h=256, d_e=64, E=8, k=2, dt=F16, ws=0x100000, n=1 << 30, out=A):
        return lib.moe_forward_mx8(A, q, sf, A, None, A, A, A, A, A, A, T, d_h, d_e, E, k, dt, ws, n, out, None, None)
    assert fwd(dt=F32) == UNSUPPORTED and fwd(d_h=128) == INVALID and fwd(d_e=32) == INVALID and fwd(k=9) == INVALID
    assert fwd(n=256) == WORKSPACE and fwd(ws=0x100008) == INVALID and fwd(out=None) == INVALID and fwd(T=0) == OK
    assert fwd(q=A) == INVALID and fwd(sf=A) == INVALID and fwd(q=A + 8, sf=A) == INVALID
    assert lib.moe_forward_mx8_workspace_bytes(4096, 7168, 2048, 256, 8, BF16) >= 32768 * (7168 * 3 + 2048) + 4096 * 7168
    assert lib.moe_forward_mx8_workspace_bytes(4, 256, 64, 8, 2, F32) == NONE


def test_binding_refuses_what_is_not_on_the_gpu():
    import torch
    q, sf = torch.zeros((4, 64), dtype=torch.float8_e4m3fn), torch.zeros((4, 2), dtype=torch.uint8)
    pos, token = torch.zeros((4, 2), dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    x = torch.zeros((8, 256))
    for call in (lambda: binding.moe_quantize_mx8(x), lambda: binding.moe_dequantize_mx8(q, sf), lambda: binding.moe_sort_rows_mx8(q, sf, pos),
                 lambda: binding.moe_residual_norm_mx8(None, x, w_next=x[0]), lambda: binding.moe_reduce_fused_backward(x[:4], x, pos, None, token),
                 lambda: binding.moe_grouped_gemm_mx8(q, sf, q[None], sf[None], {}), lambda: binding.Mx8Experts(*(q[None], sf[None]) * 3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_the_short_calls_extension_is_built(lib):
    """Where PyTorch's headers are, the binding has the extension; without a GPU's tensors it makes no call."""
    import torch
    assert binding._host is not None
    x, q = torch.zeros((4, 64)), torch.zeros((4, 64), dtype=torch.float8_e4m3fn)
    assert binding._host.norm_mx8(None, x, None, None, 1.0, x[0], 1e-6, True, None) is None
    assert binding._host.sort_rows_mx8(q, x, x) is None and binding._host.sort_rows_mx8(q) is None
    assert binding._host.reduce_fused_backward(x, x, None, None, None, None) is None
    assert binding._host.grouped_gemm_mx8(*[None] * 10) is None and binding._host.grouped_gate_up_silu_mx8(*[3] * 11) is None
    assert binding._host.experts_mx8(*[q] * 6) is None
