"""The 8-bit path repeats itself bit for bit, whatever ran before it and whatever lay in its memory; and where
h, rounded to 8 bits between the products, is not its 64-bit value's rounding, that value lies as near to the
middle between two of them as the sums' error."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding
from test_gpu_mx8 import E4M3, grid, norm_inputs, power, routed, silu_products, values64

pytestmark = pytest.mark.gpu


def weights(E, N, K, g):
    parts = []
    for n, m in ((N, K), (N, K), (K, N)):
        q, s = binding.moe_quantize_mx8(torch.randn((E * n, m), generator=g, device="cuda") * m ** -0.5)
        parts += [q.view(E, n, m), s.view(E, n, m // 32)]
    return binding.Mx8Experts(*parts)


def dirty():
    """Freed memory full of NaNs, of every type."""
    for size in (1 << 12, 1 << 16, 1 << 20, 1 << 25):
        [torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(4)]


@pytest.mark.parametrize("T,k,E,K,N", [(1, 8, 16, 512, 256), (64, 6, 64, 2048, 768), (1000, 2, 5, 1056, 352), (900, 4, 8, 7168, 512), (3000, 2, 6, 4096, 544)])
def test_calls_repeat_themselves(T, k, E, K, N):
    require_cuda()
    passes = []
    for seed in (1, 2):
        t, g = routed(T, k, E, seed)
        a, e = norm_inputs(T, K, torch.bfloat16, "channel", True, True, seed), weights(E, N, K, g)
        w, d_out = torch.rand((T, k), generator=g, device="cuda"), torch.randn((T, K), generator=g, device="cuda").bfloat16()

        def run(t=t, a=a, e=e, w=w, d_out=d_out):
            n = binding.moe_residual_norm_mx8(**a)
            q, s = binding.moe_sort_rows_mx8(n["q"], n["sf"], t["token_topk_to_pos"])
            qh, sh = binding.moe_grouped_gate_up_silu_mx8(q, s, e, t)
            y = binding.moe_grouped_gemm_mx8(qh, sh, e.q_down, e.sf_down, t)
            back = () if K % 256 else binding.moe_reduce_fused_backward(d_out, y, t["token_topk_to_pos"], w, t["sorted_token_idx"])
            return [*n.values(), q, s, qh, sh, y, *back]
        passes.append(run)
    want = [[v.clone() for v in run()] for run in passes]
    for i in range(12):
        dirty()
        for run, first in zip(passes, want):
            for v, w in zip(run(), first):
                assert torch.equal(v.view(torch.uint8), w.view(torch.uint8)), i


def rounded(h, unit):
    """h [R, N] to 8 bits at the scales unit [R, N / 32]: to nearest, ties to even, 448 at most."""
    held = grid(h.device)
    a = (h.abs().view(*unit.shape, 32) / unit[..., None]).clamp(max=448.0).contiguous()
    middle = (held[1:] + held[:-1]) / 2
    low, high = torch.searchsorted(middle, a), torch.searchsorted(middle, a, right=True)  # they differ at a tie
    return (torch.sign(h).view(a.shape) * held[torch.where(low % 2 == 0, low, high)] * unit[..., None]).view(h.shape)


@pytest.mark.parametrize("T,k,E,K,N", [(64, 6, 64, 2048, 768), (500, 2, 8, 7168, 512), (2000, 2, 5, 4096, 1056), (301, 3, 5, 1056, 352)])
def test_h_is_rounded_from_within_the_sums_error(T, k, E, K, N):
    require_cuda()
    t, g = routed(T, k, E, T)
    qa, sa = binding.moe_quantize_mx8(torch.randn((T * k, K), generator=g, device="cuda"))
    e = weights(E, N, K, g)
    q, sf = binding.moe_grouped_gate_up_silu_mx8(qa, sa, e, t)
    h, off = silu_products(t, qa, sa, (e.q_gate, e.sf_gate), (e.q_up, e.sf_up))
    got, unit = values64(q, sf), power(sf.long() - 127)
    assert q.dtype == E4M3
    assert (rounded(h - off, unit) <= got).all() and (got <= rounded(h + off, unit)).all()
    # so many elements at most lie that near to a middle: steps are 2^-4 of a value at least, and 2^-9 of the unit
    step = torch.maximum(2.0 ** -4 * h.abs(), 2.0 ** -9 * unit.repeat_interleave(32, 1))
    assert (got != rounded(h, unit)).double().mean() <= (2 * off / step).clamp(max=1.0).mean()
