"""The 4-bit forward against its definition in 64 bits, and the block that runs it
against its parts.

The definition quantises h; where h lies, within the error of fp32 sums, at the
boundary of two 4-bit values, either may come out, and with it either scale of
the block.  Bound of an output: the weighted sum over the experts of |W_down|
times half of what h's two ends are apart (plus a step of the larger scale where
the ends' scales differ), the sums' 2^-20 of their magnitudes, half a unit in
the last place for each expert's rounded output and for the result."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding
from mixture_experts_routed_gate_gb300.block import MoEBlock, run_blocks
from test_gpu_mx4 import DT, product64, quantize64, values64

pytestmark = pytest.mark.gpu

UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def make(T, d_h, d_e, E, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda std, *s: (torch.randn(s, generator=g, device="cuda") * std).to(DT[dtype])  # noqa: E731
    w = n(d_h ** -0.5, E, d_e, d_h), n(d_h ** -0.5, E, d_e, d_h), n(d_e ** -0.5, E, d_h, d_e)
    return n(1.0, T, d_h), n(d_h ** -0.5, E, d_h), binding.Mx4Experts.from_weights(*w), n


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,d_h,d_e,E,k", [(1, 256, 64, 4, 2), (37, 512, 192, 16, 3), (300, 768, 320, 6, 2), (1100, 256, 128, 80, 4)])
def test_forward_against_its_definition(T, d_h, d_e, E, k, dtype):
    require_cuda()
    x, w_g, ex, _ = make(T, d_h, d_e, E, dtype, T + E)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.moe_forward_mx4(x, w_g, None, ex, k, err=err).double()
    assert int(err.item()) == 0
    idx, p = binding.moe_gate_topk(x, w_g, None, k)  # its own tests hold it to the oracle
    a = quantize64(x)[0]
    want, off = torch.zeros_like(got), torch.zeros_like(got)
    gate, up, down = values64(ex.q_gate, ex.sf_gate), values64(ex.q_up, ex.sf_up), values64(ex.q_down, ex.sf_down)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        g, u = a[t] @ gate[e].t(), a[t] @ up[e].t()
        mg, mu = a[t].abs() @ gate[e].abs().t(), a[t].abs() @ up[e].abs().t()
        silu = g * torch.sigmoid(g)
        h = silu * u
        eh = 2.0 ** -20 * (1.1 * mg * u.abs() + silu.abs() * mu + h.abs()) + 1e-30
        (lo, el), (hi, e2) = quantize64(h - eh), quantize64(h + eh)
        apart = (lo - hi).abs() / 2 + torch.where(el != e2, torch.exp2(torch.maximum(el, e2) + 1.0), 0.0).repeat_interleave(32, 1)
        mid = (lo + hi) / 2
        y = mid @ down[e].t()
        ey = apart @ down[e].abs().t() + 2.0 ** -20 * (mid.abs() @ down[e].abs().t())
        w = p[t, j].double()[:, None]
        want.index_add_(0, t, w * y)
        off.index_add_(0, t, w * (ey + UNIT[dtype] * (y.abs() + ey) + 2.0 ** -24))
    bound = off + UNIT[dtype] * (want.abs() + off) + 2.0 ** -24 + 2.0 ** -20 * want.abs()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / bound).max()))
    assert float((got - want).norm() / want.norm()) < 8 * UNIT[dtype]  # few elements are at a boundary


@pytest.mark.parametrize("T", [1, 8, 9, 130])
def test_blocks_are_their_parts(T):
    require_cuda()
    blocks, parts = [], []
    for i in range(3):
        x, w_g, ex, n = make(T, 512, 128, 16, "bf16", 50 + i)
        w_post, w_next = 1 + n(0.2, 512), 1 + n(0.2, 512) if i < 2 else None
        gate = 1 + n(0.2, 512) if i == 1 else None
        blocks.append(MoEBlock(w_g=w_g, bias=None, experts=ex, k=4, w_post=w_post, gate=gate, alpha=0.5, w_next=w_next))
        parts.append((w_g, ex, w_post, gate, w_next))
    w_first = 1 + n(0.2, 512)
    u, res = run_blocks(blocks, x, w_first)
    assert u is None
    v, s = binding.moe_residual_norm(None, x, w_next=w_first)["u"], x
    for w_g, ex, w_post, gate, w_next in parts:
        y = binding.moe_forward_mx4(v, w_g, None, ex, 4)
        r = binding.moe_residual_norm(y, s, w_post, gate, 0.5, w_next)
        v, s = r.get("u"), r["out"]
    assert torch.equal(res, s)
