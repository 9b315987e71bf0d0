"""moe_forward_few against the layer's definition in 64 bits.

Tolerance, per output element, from the roundings the kernel makes: one unit in
the last place of the output's type, and, times the magnitudes they act on:
  e_dot = 2^-18 of a dot product's sum of magnitudes (fp32 chains and trees),
  2^-15 of each |p * W_down| * |h| (h as a 16-bit value and its 16-bit rest,
  __expf, the fp32 sums over the experts)."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
ULP = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}


def make(T, d_h, d_e, E, k, dtype, seed=0, bias=False):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + T * 31 + E)
    n = lambda std, *s: (torch.randn(s, generator=g, device="cuda") * std).to(DT[dtype])  # noqa: E731
    return dict(x=n(1.0, T, d_h), w_g=n(d_h ** -0.5, E, d_h), bias=torch.randn(E, generator=g, device="cuda") if bias else None,
                w_gate=n(d_h ** -0.5, E, d_e, d_h), w_up=n(d_h ** -0.5, E, d_e, d_h), w_down=n(d_e ** -0.5, E, d_h, d_e))


def definition(s, idx, w):
    """Outputs and error bounds (without the output's own rounding) for a given
    routing and its weights, one routed pair at a time."""
    x = s["x"].double()
    out, off = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        for e, p in zip(idx[t].tolist(), w[t].double().tolist()):
            wg, wu, wd = (s[n][e].double() for n in ("w_gate", "w_up", "w_down"))
            g, u = wg @ x[t], wu @ x[t]
            eg, eu = (2.0 ** -18 * (m.abs() @ x[t].abs()) for m in (wg, wu))
            silu = g * torch.sigmoid(g)
            h = silu * u
            eh = 1.1 * eg * u.abs() + silu.abs() * eu + eg * eu + 2.0 ** -15 * h.abs()
            out[t] += p * (wd @ h)
            off[t] += abs(p) * (wd.abs() @ eh) + 2.0 ** -15 * abs(p) * (wd.abs() @ h.abs())
    return out, off


def check(s, k, dtype, got, err):
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    idx, w = binding.moe_gate_topk(s["x"], s["w_g"], s["bias"], k)  # its own tests hold it to the oracle
    want, off = definition(s, idx, w)
    bound = ULP[dtype] * want.abs() + off + 1e-7
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / bound).max()))


def call(s, k, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    return binding.moe_forward_few(s["x"], s["w_g"], s["bias"], s["w_gate"], s["w_up"], s["w_down"], k, err=err, **kw), err


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,d_h,d_e,E,k", [
    (1, 256, 64, 1, 1),          # the smallest
    (1, 2048, 768, 64, 6),       # the decode layer
    (8, 2048, 768, 64, 6),
    (16, 2048, 768, 64, 6),
    (16, 256, 64, 1, 1),         # every token to one expert
    (16, 512, 192, 8, 8),        # every token to every expert
    (9, 768, 320, 40, 32),       # the largest k
    (3, 256, 64, 1000, 5),       # many experts, one warp's share over 31
    (5, 512, 576, 33, 3),        # a last chunk of 64 columns
    (7, 1280, 1024, 3, 2),
    (13, 256, 2048, 17, 4),
    (2, 7168, 2048, 24, 8),
])
def test_against_the_definition(T, d_h, d_e, E, k, dtype):
    require_cuda()
    s = make(T, d_h, d_e, E, k, dtype, bias=T % 2 == 1)
    got, err = call(s, k)
    check(s, k, dtype, got, err)


def test_every_token_count():
    require_cuda()
    for T in range(1, 17):
        s = make(T, 512, 128, 12, 3, "bf16", seed=2)
        got, err = call(s, 3)
        check(s, 3, "bf16", got, err)


def test_ties_equal_tokens_and_masked_experts():
    require_cuda()
    s = make(6, 512, 128, 32, 4, "f16", seed=4)
    s["w_g"][1::2] = s["w_g"][0::2]        # pairs of equal logits: the lower id first
    s["x"][3] = s["x"][2]
    s["x"][4] = 0                          # all logits equal: experts 0 to 3
    got, err = call(s, 4)
    check(s, 4, "f16", got, err)
    assert torch.equal(got[2], got[3])
    assert bool((got[4] == 0).all())
    s["bias"] = torch.zeros(32, device="cuda")
    s["bias"][5:] = float("-inf")          # five experts left of 32
    got, err = call(s, 4)
    check(s, 4, "f16", got, err)
    s["bias"][2:] = float("-inf")          # fewer than k left: the rest have weight 0
    got, err = call(s, 4)
    check(s, 4, "f16", got, err)
    s["bias"][2:] = torch.finfo(torch.float32).min
    got, err = call(s, 4)
    check(s, 4, "f16", got, err)


def test_a_bad_token_stays_alone():
    require_cuda()
    s = make(8, 512, 128, 16, 2, "bf16", seed=6)
    ref, _ = call(s, 2)
    s["x"][5, 17] = float("nan")
    s["x"][2, 3] = float("inf")
    got, err = call(s, 2)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for t in (0, 1, 3, 4, 6, 7):
        assert torch.equal(got[t], ref[t]), t
    assert not bool(got[5].isfinite().any()) and not bool(got[2].isfinite().all())


def test_repeat_stream_graph_and_dirty_workspace():
    require_cuda()
    s = make(4, 1024, 256, 48, 5, "bf16", seed=8)
    ref, err = call(s, 5)
    check(s, 5, "bf16", ref, err)
    n = binding.forward_few_workspace_bytes(4, 1024, 256, 48, 5, torch.bfloat16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        for _ in range(20):
            got, err = call(s, 5, ws=ws)
            assert torch.equal(got, ref)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured, _ = call(s, 5, ws=ws)
    for _ in range(5):
        captured.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, ref)


@pytest.mark.parametrize("T,d_h,d_e,E,k", [(1, 256, 64, 5, 2), (11, 512, 192, 9, 3), (16, 1280, 320, 70, 7)])
def test_writes_stay_inside(T, d_h, d_e, E, k):
    require_cuda()
    s = make(T, d_h, d_e, E, k, "f16", seed=10)
    n = binding.forward_few_workspace_bytes(T, d_h, d_e, E, k, torch.float16)
    raw = torch.full((4096 + n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    raw_out = torch.full((4096 + T * d_h * 2 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = raw_out[4096:-4096].view(torch.float16).view(T, d_h)
    got, err = call(s, k, ws=raw[4096:4096 + n], out=out)
    check(s, k, "f16", got, err)
    for r, m in ((raw, n), (raw_out, T * d_h * 2)):
        assert bool((r[:4096] == 0xA5).all()) and bool((r[4096 + m:] == 0xA5).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,d_h,d_e,E,k", [(8, 512, 128, 16, 4), (16, 512, 128, 16, 4), (3, 768, 576, 9, 3), (11, 1280, 64, 7, 1)])
def test_the_bits_do_not_depend_on_the_order_of_work(T, d_h, d_e, E, k, dtype, monkeypatch):
    """Tiles are taken from a shared counter: one CTA, a few, or more than fit at
    once, on workspaces that hold other bytes every time, give the same bits."""
    require_cuda()
    s = make(T, d_h, d_e, E, k, dtype, seed=14)
    n = binding.forward_few_workspace_bytes(T, d_h, d_e, E, k, DT[dtype])
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ref, err = call(s, k, ws=ws)
    check(s, k, dtype, ref, err)
    outs = []
    for grid in (None, "1", "7", "304"):
        if grid is not None:
            monkeypatch.setenv("MOE_MLP_GRID", grid)
        for i in range(50 if grid is None else 5):
            ws.fill_(0x7F if i % 2 else 0xFF)
            outs.append(call(s, k, ws=ws)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_near_the_forward():
    """moe_forward on the same tokens, within its own tolerance."""
    require_cuda()
    s = make(16, 2048, 768, 64, 6, "f16", seed=12)
    got, _ = call(s, 6)
    ref = binding.moe_forward(s["x"], s["w_g"], None, s["w_gate"], s["w_up"], s["w_down"], 6)
    assert bool(((got.float() - ref.float()).abs() <= 2e-3 + 2e-2 * ref.float().abs()).all())


def test_refusals():
    require_cuda()
    s = make(2, 256, 64, 4, 2, "f16")
    more = {**s, "x": torch.zeros((17, 256), dtype=torch.float16, device="cuda")}
    with pytest.raises(ValueError):
        call(more, 2)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(binding.MoEError, match="UNSUPPORTED"):
        call(more, 2, ws=ws)
    with pytest.raises(binding.MoEError, match="INVALID_ARG"):
        call(s, 5, ws=ws)
    with pytest.raises(binding.MoEError, match="WORKSPACE"):
        call(s, 2, ws=ws[:256])
    with pytest.raises(binding.MoEError, match="INVALID_ARG"):
        call(s, 2, ws=ws[16:])
    with pytest.raises(ValueError):
        call({**s, "bias": torch.zeros(3, device="cuda")}, 2)
    with pytest.raises(TypeError):
        call({**s, "w_up": s["w_up"].bfloat16()}, 2)
    with pytest.raises(ValueError):
        call({**s, "w_down": s["w_down"].transpose(1, 2).contiguous()}, 2)
    none = {**s, "x": s["x"][:0]}
    assert call(none, 2, ws=ws)[0].shape == (0, 256)
