"""The pre-norm block: norms, the routed layer's three paths and the residual
stream together, against the same steps in 64 bits.

The layer's own errors are tested elsewhere; here its output is compared with
the relative error of the whole stream: each 16-bit tensor on the way rounds
by 2^-11 (fp16) or 2^-8 (bf16), a block adds a handful of such roundings, and
the routing is taken from the library so that a near tie does not decide."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding
from mixture_experts_routed_gate_gb300.block import FEW_TOKENS, MoEBlock, run_blocks

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def make_blocks(n, d_h, d_e, E, k, dtype, mx4=False):
    g = torch.Generator(device="cuda").manual_seed(n * 31 + d_h)
    r = lambda std, *s: (torch.randn(s, generator=g, device="cuda") * std).to(DT[dtype])  # noqa: E731
    one = lambda: (1 + 0.2 * torch.randn(d_h, generator=g, device="cuda")).to(DT[dtype])  # noqa: E731
    blocks = []
    for i in range(n):
        w = (r(d_h ** -0.5, E, d_e, d_h), r(d_h ** -0.5, E, d_e, d_h), r(d_e ** -0.5, E, d_h, d_e))
        blocks.append(MoEBlock(w_g=r(d_h ** -0.5, E, d_h), bias=None, experts=binding.Mx4Experts.from_weights(*w) if mx4 else w, k=k,
                               w_post=one(), gate=one() if i % 2 else None, alpha=0.5, w_next=one() if i + 1 < n else None))
    return blocks, one(), r


def norm64(v, w, eps=1e-6):
    return v / (v.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, FEW_TOKENS, FEW_TOKENS + 1, 70])
def test_blocks_against_64_bits(T, dtype):
    require_cuda()
    blocks, w_first, r = make_blocks(3, 512, 128, 16, 4, dtype)
    x = r(1.0, T, 512)
    keep = x.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    u, res = run_blocks(blocks, x, w_first, err=err)
    assert u is None and torch.equal(x, keep) and int(err.item()) == 0
    # the same stream in 64 bits; the routing of each block from the library's own input to it
    s = x.double()
    v16 = binding.moe_residual_norm(None, x, w_next=w_first)["u"]
    stream = x.clone()
    v = norm64(s, w_first)
    for b in blocks:
        idx, p = binding.moe_gate_topk(v16, b.w_g, None, b.k)
        y = torch.zeros_like(s)
        for t in range(T):
            for e, weight in zip(idx[t].tolist(), p[t].double().tolist()):
                g, up = b.experts[0][e].double() @ v[t], b.experts[1][e].double() @ v[t]
                y[t] += weight * (b.experts[2][e].double() @ (g * torch.sigmoid(g) * up))
        z = norm64(y, b.w_post) * (1.0 if b.gate is None else b.gate.double())
        s = s + b.alpha * z
        v16, stream = b(v16, stream)
        if b.w_next is not None:
            v = norm64(s, b.w_next)
    assert torch.equal(stream, res)
    off = float((res.double() - s).norm() / s.norm())
    assert off <= 12 * UNIT[dtype], off


def test_blocks_with_4_bit_experts():
    """Near the 16-bit blocks' stream: 4-bit rows and weights each round by about
    a tenth, halved by alpha and under the residual."""
    require_cuda()
    four, w_first, r = make_blocks(2, 512, 128, 16, 4, "bf16", mx4=True)
    full, _, _ = make_blocks(2, 512, 128, 16, 4, "bf16")
    for T in (1, 200):
        x = r(1.0, T, 512)
        a, b = run_blocks(four, x, w_first)[1].float(), run_blocks(full, x, w_first)[1].float()
        assert 1e-4 < float((a - b).norm() / b.norm()) < 0.3


def test_a_decode_step_in_a_graph():
    require_cuda()
    blocks, w_first, r = make_blocks(2, 1024, 256, 32, 4, "f16")
    x = r(1.0, 4, 1024)
    want = run_blocks(blocks, x, w_first)[1]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = run_blocks(blocks, x, w_first)[1]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_only_the_last_block_ends_the_stream():
    require_cuda()
    blocks, w_first, r = make_blocks(1, 512, 128, 16, 4, "f16")
    with pytest.raises(ValueError):
        run_blocks(blocks * 2, r(1.0, 2, 512), w_first)
