"""moe_forward_few on weights with infinities and NaN, on activations that the
16-bit types barely hold, and past their range."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding
from test_gpu_few import DT, ULP, call, definition, make

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
HALF_STEP = {"f16": 2.0 ** -25, "bf16": 0.0}  # half the distance of the smallest outputs


def check(s, k, dtype, got, err, pick=None):
    """As the layer's own tests, without their flat 1e-7."""
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    idx, w = binding.moe_gate_topk(s["x"], s["w_g"], s["bias"], k)
    want, off = definition(s, idx, w)
    bound = ULP[dtype] * want.abs() + off + HALF_STEP[dtype]
    bad = ~((got.double() - want).abs() <= bound)
    if pick is not None:
        bad &= pick
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / bound)[bad].max()))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,d_h,d_e,E,k", [(3, 512, 192, 8, 2), (8, 768, 576, 12, 3), (16, 512, 128, 20, 4), (5, 1024, 2048, 6, 1)])
def test_bad_weights_reach_the_tokens_routed_to_them(T, d_h, d_e, E, k, dtype):
    require_cuda()
    s = make(T, d_h, d_e, E, k, dtype, seed=21)
    idx, _ = binding.moe_gate_topk(s["x"], s["w_g"], None, k)
    ref, err = call(s, k)
    check(s, k, dtype, ref, err)
    counts = torch.bincount(idx.flatten().long(), minlength=E).tolist()
    e = next(i for i, n in enumerate(counts) if 0 < n < T)
    routed = (idx == e).any(1)
    rows = (0, 17, d_h - 1)
    for value in (INF, -INF, NAN):
        t = {**s, "w_down": s["w_down"].clone()}
        for row, col in zip(rows, (0, 65, d_e - 1)):
            t["w_down"][e, row, col] = value
        got, err = call(t, k)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        hit = torch.zeros_like(ref, dtype=torch.bool)
        hit[:, list(rows)] = True
        assert torch.equal(got[~hit], ref[~hit])
        assert not bool(got[hit & routed[:, None]].isfinite().any())
        # the others' sums over their own experts, the definition's
        check(s, k, dtype, got, err, pick=hit & ~routed[:, None])
        for name in ("w_gate", "w_up"):
            t = {**s, name: s[name].clone()}
            t[name][e, 3, 9] = value
            got, err = call(t, k)
            torch.cuda.synchronize()
            assert int(err.item()) == 0
            assert torch.equal(got[~routed], ref[~routed])
            assert not bool(got[routed].isfinite().all(1).any())
        again, _ = call(t, k)
        assert torch.equal(again.nan_to_num(7.0), got.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -5, 2.0 ** -7, 2.0 ** -9])
@pytest.mark.parametrize("T,E,k", [(1, 256, 6), (16, 64, 8), (8, 1024, 4)])
def test_small_activations_and_many_experts(T, E, k, size, dtype):
    """A flat routing, weights near 1 / E, times h of about size^2 / 2: the
    products reach far into fp16's subnormals (2^-29), h itself to 2^-19, and the
    results keep the tolerance of the layer's own tests.  W_down is large, so
    that the outputs are no subnormals themselves."""
    require_cuda()
    s = make(T, 512, 128, E, k, dtype, seed=31)
    s["x"] = (s["x"].float() * size).to(DT[dtype])
    s["w_down"] = (s["w_down"].float() * 512).to(DT[dtype])
    got, err = call(s, k)
    check(s, k, dtype, got, err)


def test_past_the_largest_fp16():
    """h of 90,000 times a weight of 1 is held (the weight counts as 0.5); h of
    360,000 is an infinity of its sign as moe_forward's, not a NaN."""
    require_cuda()
    s = make(5, 512, 64, 1, 1, "f16", seed=41)
    s["w_gate"].zero_()
    s["w_up"].zero_()
    s["w_gate"][0, 7, 0] = 1
    s["w_up"][0, 7, 0] = 1
    s["x"][:, 0] = 300
    got, err = call(s, 1)
    check(s, 1, "f16", got, err)
    s["x"][:, 0] = 600
    got, err = call(s, 1)
    ref = binding.moe_forward(s["x"], s["w_g"], None, s["w_gate"], s["w_up"], s["w_down"], 1)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    some = s["w_down"][0, :, 7] != 0
    assert bool(got[:, some].isinf().all()) and torch.equal(got[:, some], ref[:, some])
