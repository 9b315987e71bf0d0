"""Tensors of more than 2^31 elements: the last rows of a long call are, to the
last bit, what a call with those rows alone gives."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding

pytestmark = pytest.mark.gpu

LAST = 100


def rows(T, H, seed, std=1.0):
    """[T, H] bf16: zeros but for the first and the last rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:LAST].normal_(generator=g).mul_(std)
    x[-LAST:].normal_(generator=g).mul_(std)
    return x


@pytest.mark.parametrize("T,H", [(135000, 16000), (1100000, 2001)])
def test_norms(T, H):
    require_cuda()
    assert T * H > 2 ** 31
    y, res = rows(T, H, 1), rows(T, H, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    w_post, w_next = (1 + 0.2 * torch.randn(H, generator=g, device="cuda").bfloat16() for _ in range(2))
    gate = torch.randn((T, 1), generator=g, device="cuda").bfloat16()
    got = binding.moe_residual_norm(y, res, w_post, gate, 0.5, w_next, 1e-6)
    tail = lambda t: t[-LAST:].clone()  # noqa: E731  (a slice need not start on 16 bytes)
    want = binding.moe_residual_norm(tail(y), tail(res), w_post, tail(gate), 0.5, w_next, 1e-6)
    for k in want:
        assert torch.equal(got[k][-LAST:], want[k]), k
    assert bool((got["out"][LAST:-LAST] == 0).all())
    d_u = res  # as good as any
    back = binding.moe_residual_norm_backward(None, d_u, y, got["out"], w_post, gate, 0.5, w_next, got["rstd_post"], got["rstd_next"])
    part = binding.moe_residual_norm_backward(None, tail(d_u), tail(y), want["out"], w_post, tail(gate), 0.5, w_next,
                                              want["rstd_post"], want["rstd_next"])
    for k in ("d_res", "d_y", "d_gate"):
        assert torch.equal(back[k][-LAST:], part[k]), k
    head = binding.moe_residual_norm_backward(None, d_u[:LAST].clone(), y[:LAST].clone(), got["out"][:LAST].clone(), w_post,
                                              gate[:LAST].clone(), 0.5, w_next, got["rstd_post"][:LAST].clone(),
                                              got["rstd_next"][:LAST].clone())
    for k in ("d_w_post", "d_w_next"):  # the rows between are zeros; sums of 200 terms in two orders
        whole, parts = back[k].double(), head[k].double() + part[k].double()
        assert float((whole - parts).abs().max()) <= 2.0 ** -18 * float(parts.abs().max()) + 2.0 ** -18, k


def test_quantised_rows():
    require_cuda()
    R, K = 300000, 7200
    assert R * K > 2 ** 31
    x = rows(R, K, 4)
    q, sf = binding.moe_quantize_mx4(x)
    want = binding.moe_quantize_mx4(x[-LAST:].clone())
    assert torch.equal(q[-LAST:], want[0]) and torch.equal(sf[-LAST:], want[1])
    idx = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda")
    back_q, back_sf = binding.moe_quantize_mx4(x, idx)
    assert torch.equal(back_q[:LAST], want[0].flip(0)) and torch.equal(back_sf[:LAST], want[1].flip(0))
    del back_q, back_sf
    values = binding.moe_dequantize_mx4(q, sf)
    assert torch.equal(values[-LAST:], binding.moe_dequantize_mx4(*want))
    assert bool((values[LAST:-LAST] == 0).all())


@pytest.mark.parametrize("N", [2048, 2000, 1999])  # whole stores, their last columns, transposed ones
def test_product(N):
    require_cuda()
    E, K, n = 3, 32, 1100000
    sizes = [n - 1000, 0, 1000]
    assert n * N > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(5)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)  # noqa: E731
    qa, sa, qb, sb = u8(0, 256, n, K // 2), u8(120, 132, n, K // 32), u8(0, 256, E, N, K // 2), u8(118, 126, E, N, K // 32)

    def tables(sizes):
        e = torch.repeat_interleave(torch.arange(E, dtype=torch.int32), torch.tensor(sizes)).cuda().view(-1, 1)
        return binding.moe_build_dispatch(e, None, E)

    got = binding.moe_grouped_gemm_mx4(qa, sa, qb, sb, tables(sizes), torch.bfloat16)
    want = binding.moe_grouped_gemm_mx4(qa[-1000:].clone(), sa[-1000:].clone(), qb, sb, tables([0, 0, 1000]), torch.bfloat16)
    assert torch.equal(got[-1000:], want)
    at = n - 1000 - 256  # the last rows of the first expert
    want = binding.moe_grouped_gemm_mx4(qa[at:at + 256].clone(), sa[at:at + 256].clone(), qb, sb, tables([256, 0, 0]), torch.bfloat16)
    assert torch.equal(got[at:at + 256], want)
