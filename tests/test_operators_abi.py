"""Host-side checks of the norms, the few-token layer and the 4-bit entry
points: every refusal happens before any CUDA call, so none of this needs a
GPU."""
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


def norm(lib, y=A, res=A, w_post=A, gate=None, kind=0, alpha=1.0, w_next=A, eps=1e-6, T=4, H=64, dtype=BF16, out=A, u=A,
         r_post=None, r_next=None):
    return lib.moe_residual_norm(y, res, w_post, gate, kind, alpha, w_next, eps, T, H, dtype, out, u, r_post, r_next, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=E4M3), UNSUPPORTED), (dict(H=0), INVALID), (dict(H=16385), UNSUPPORTED), (dict(T=-1), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID), (dict(alpha=float("nan")), INVALID),
    (dict(kind=4), INVALID), (dict(kind=-1), INVALID), (dict(kind=1), INVALID), (dict(gate=A), INVALID), (dict(res=None), INVALID),
    (dict(out=None), INVALID), (dict(u=None), INVALID), (dict(w_next=None), INVALID), (dict(y=None, out=None), INVALID),
    (dict(y=None, w_post=None), INVALID), (dict(y=None, w_post=None, out=None, w_next=None, u=None), INVALID),
    (dict(w_post=None, r_post=A), INVALID), (dict(y=A + 8), INVALID), (dict(u=A + 2), INVALID), (dict(w_post=A + 4), INVALID),
    (dict(T=0), OK), (dict(T=0, y=None, res=None, out=None, u=None, kind=2), OK),
])
def test_residual_norm(lib, change, status):
    assert norm(lib, **change) == status


def backward(lib, d_out=A, d_u=A, y=A, out=A, w_post=A, gate=None, kind=0, w_next=A, r_post=A, r_next=A, T=4, H=64, dtype=F16,
             d_res=A, d_y=A, d_gate=None, d_wp=A, d_wn=A, ws=A, nws=1 << 20):
    return lib.moe_residual_norm_backward(d_out, d_u, y, out, w_post, gate, kind, 1.0, w_next, r_post, r_next, T, H, dtype, d_res,
                                          d_y, d_gate, d_wp, d_wn, ws, nws, None)


@pytest.mark.parametrize("change,status", [
    (dict(d_out=None, d_u=None, w_next=None, d_wn=None), INVALID), (dict(d_u=None), INVALID), (dict(w_next=None), INVALID),
    (dict(out=None), INVALID), (dict(r_next=None), INVALID), (dict(r_post=None), INVALID), (dict(d_res=None), INVALID),
    (dict(d_y=None), INVALID), (dict(d_gate=A), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 8), INVALID),
    (dict(nws=8), WORKSPACE), (dict(dtype=E4M3), UNSUPPORTED), (dict(w_post=None, r_post=None), INVALID), (dict(d_y=A + 2), INVALID),
])
def test_residual_norm_backward(lib, change, status):
    assert backward(lib, **change) == status


def test_workspace_sizes(lib):
    assert lib.moe_residual_norm_backward_workspace_bytes(0, 64) >= 0
    assert lib.moe_residual_norm_backward_workspace_bytes(2, 64) >= 2 * 3 * 64 * 4
    assert lib.moe_residual_norm_backward_workspace_bytes(-1, 64) == NONE
    assert lib.moe_residual_norm_backward_workspace_bytes(4, 16385) == NONE
    small, large = (lib.moe_forward_few_workspace_bytes(T, 2048, 768, 64, 6, F16) for T in (1, 16))
    assert 2 * 6 * 768 * 2 <= small < large and small % 256 == 0
    for bad in ((17, 2048, 768, 64, 6, F16), (1, 2048, 768, 64, 6, F32), (1, 2048, 768, 1025, 6, F16), (1, 2048, 768, 64, 33, F16)):
        assert lib.moe_forward_few_workspace_bytes(*bad) == NONE
    assert lib.moe_forward_mx4_workspace_bytes(4096, 7168, 2048, 256, 8, BF16) >= 32768 * (7168 * 2 + (7168 + 2048) // 2)
    assert lib.moe_forward_mx4_workspace_bytes(4, 256, 64, 8, 2, F32) == NONE


def few(lib, x=A, w_down=A, T=2, d_h=256, d_e=64, E=4, k=2, dtype=F16, ws=0x100000, nws=1 << 30, out=A):
    return lib.moe_forward_few(x, A, None, A, A, w_down, T, d_h, d_e, E, k, dtype, ws, nws, out, None, None)


@pytest.mark.parametrize("change,status", [
    (dict(T=17), UNSUPPORTED), (dict(dtype=F32), UNSUPPORTED), (dict(d_h=128), INVALID), (dict(d_e=96), INVALID), (dict(k=5), INVALID),
    (dict(k=33, E=64), INVALID), (dict(E=1025), INVALID), (dict(x=None), INVALID), (dict(w_down=None), INVALID), (dict(out=None), INVALID),
    (dict(ws=0x100010), INVALID), (dict(nws=64), WORKSPACE), (dict(x=A + 8), INVALID), (dict(T=0, x=None), OK), (dict(T=-1), INVALID),
])
def test_forward_few(lib, change, status):
    assert few(lib, **change) == status


def test_mx4_entry_points(lib):
    q = lambda x=A, idx=None, n=4, T=4, K=64, dt=BF16, o=A, s=A: lib.moe_quantize_mx4(x, idx, n, T, K, dt, o, s, None, None)  # noqa: E731
    assert q(K=48) == INVALID and q(K=0) == INVALID and q(n=5) == INVALID and q(dt=E4M3) == UNSUPPORTED
    assert q(x=None) == INVALID and q(o=None) == INVALID and q(s=None) == INVALID and q(x=A + 8) == INVALID and q(o=A + 4) == INVALID
    assert q(n=0) == OK and q(K=1 << 21) == UNSUPPORTED
    d = lambda n=4, K=64, dt=F32, o=A: lib.moe_dequantize_mx4(A, A, n, K, dt, o, None)  # noqa: E731
    assert d(K=33) == INVALID and d(dt=E4M3) == UNSUPPORTED and d(o=None) == INVALID and d(o=A + 8) == INVALID and d(n=0) == OK

    def gemm(a=A, b=A, mb=3, rows=8, N=128, K=64, E=8, dt=BF16, c=A):
        return lib.moe_grouped_gemm_mx4(a, A, b, A, A, A, A, A, mb, rows, N, K, E, dt, c, None, None)
    assert gemm(K=48) == INVALID and gemm(N=0) == INVALID and gemm(dt=E4M3) == UNSUPPORTED and gemm(mb=99) == INVALID
    assert gemm(a=None) == INVALID and gemm(b=A + 8) == INVALID and gemm(c=None) == INVALID and gemm(rows=0) == OK
    assert gemm(N=1 << 21) == UNSUPPORTED

    def up(d_h=64, d_e=64, q_h=A):
        return lib.moe_grouped_gate_up_silu_mx4(A, A, A, A, A, A, A, A, A, A, 3, 8, d_h, d_e, 8, q_h, A, None, None)
    assert up(d_e=48) == INVALID and up(d_h=40) == INVALID and up(q_h=None) == INVALID and up(q_h=A + 8) == INVALID

    def fwd(T=4, d_h=256, d_e=64, E=8, k=2, dt=F16, ws=0x100000, n=1 << 30, out=A):
        return lib.moe_forward_mx4(A, A, None, A, A, A, A, A, A, T, d_h, d_e, E, k, dt, ws, n, out, None, None)
    assert fwd(dt=F32) == UNSUPPORTED and fwd(d_h=128) == INVALID and fwd(d_e=32) == INVALID and fwd(k=9) == INVALID
    assert fwd(n=256) == WORKSPACE and fwd(ws=0x100008) == INVALID and fwd(out=None) == INVALID and fwd(T=0) == OK
