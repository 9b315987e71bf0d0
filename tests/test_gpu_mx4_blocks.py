"""The 4-bit products over more blocks of rows than a CTA lists in shared
memory (512), where every role looks each tile up in the tables, and at that
number itself."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding
from test_gpu_mx4 import DT, check, operands, product64, quantize64, tables_for, values64

pytestmark = pytest.mark.gpu


def groups(E, full):
    """E groups of 0 to 2 rows, `full` of them with rows."""
    g = torch.Generator().manual_seed(E + full)
    sizes = torch.zeros(E, dtype=torch.int64)
    at = torch.randperm(E, generator=g)[:full]
    sizes[at] = torch.randint(1, 3, (full,), generator=g)
    return sizes.tolist()


# one, two and three slices of 256 columns, partly filled; more tiles than CTAs, in one and two columns of tiles
@pytest.mark.parametrize("K", [32, 288, 512, 544])
@pytest.mark.parametrize("E,full", [(600, 600), (700, 530), (520, 512), (520, 513)])
def test_product_of_many_blocks(E, full, K):
    require_cuda()
    sizes = groups(E, full)
    for N, dtype in ((40, "f32"), (200, "bf16")):
        ops = operands(sum(sizes), E, N, K, seed=E)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = binding.moe_grouped_gemm_mx4(*ops, tables_for(sizes), DT[dtype], err=err)
        want, mag = product64(*ops, sizes)
        assert int(err.item()) == 0
        check(got, want, mag, dtype)


def test_product_of_many_full_blocks():
    """Experts of several blocks among them."""
    require_cuda()
    sizes = groups(520, 500)
    sizes[3], sizes[200], sizes[519] = 1500, 129, 128
    ops = operands(sum(sizes), 520, 64, 256, seed=1)
    got = binding.moe_grouped_gemm_mx4(*ops, tables_for(sizes), torch.float16)
    want, mag = product64(*ops, sizes)
    check(got, want, mag, "f16")


@pytest.mark.parametrize("E,full", [(600, 600), (700, 530), (520, 512), (520, 513)])
def test_gate_up_of_many_blocks(E, full):
    """As the product's own test of it: between the quantised ends."""
    require_cuda()
    d_h, d_e, sizes = 288, 128, groups(E, full)
    rows = sum(sizes)
    qa, sa, qg, sg = operands(rows, E, d_e, d_h, seed=1)
    _, _, qu, su = operands(rows, E, d_e, d_h, seed=2)
    e = binding.Mx4Experts(qg, sg, qu, su, torch.zeros((E, d_h, d_e // 2), dtype=torch.uint8, device="cuda"),
                           torch.zeros((E, d_h, d_e // 32), dtype=torch.uint8, device="cuda"))
    qh, sh = binding.moe_grouped_gate_up_silu_mx4(qa, sa, e, tables_for(sizes))
    g, mg = product64(qa, sa, qg, sg, sizes)
    u, mu = product64(qa, sa, qu, su, sizes)
    silu = g * torch.sigmoid(g)
    h = silu * u
    off = 2.0 ** -20 * (1.1 * mg * u.abs() + silu.abs() * mu + h.abs()) + 1e-30
    (lo, el), (hi, eh) = quantize64(h - off), quantize64(h + off)
    got = values64(qh, sh)
    steady = ((el == eh) & (sh.long() - 127 == el)).repeat_interleave(32, 1)
    assert float(steady.double().mean()) > 0.9
    assert bool(((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi)))[steady].all())


@pytest.mark.parametrize("T,E,k", [(3000, 600, 8), (2500, 513, 2)])
def test_forward_of_many_blocks(T, E, k):
    """The 4-bit forward is its parts there too."""
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda std, *s: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    x, w_g = n(1.0, T, 256), n(1 / 16, E, 256)
    ex = binding.Mx4Experts.from_weights(n(1 / 16, E, 64, 256), n(1 / 16, E, 64, 256), n(1 / 8, E, 256, 64))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.moe_forward_mx4(x, w_g, None, ex, k, err=err)
    idx, w = binding.moe_gate_topk(x, w_g, None, k)
    tab = binding.moe_build_dispatch(idx, w, E)
    qa, sa = binding.moe_quantize_mx4(x, tab["sorted_token_idx"])
    qh, sh = binding.moe_grouped_gate_up_silu_mx4(qa, sa, ex, tab)
    y = binding.moe_grouped_gemm_mx4(qh, sh, ex.q_down, ex.sf_down, tab, x.dtype)
    assert int(err.item()) == 0
    assert torch.equal(out, binding.moe_reduce_fused(y, tab["token_topk_to_pos"], w))
    sizes = tab["group_sizes"].tolist()
    assert sum(-(-n // 128) for n in sizes) > 512
    want, mag = product64(qh, sh, ex.q_down, ex.sf_down, sizes)
    check(y, want, mag, "bf16")
