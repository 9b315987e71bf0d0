"""The norm that writes 8-bit rows, at factors whose products with one another leave fp32's range while the
result does not: each product is taken in the order of moe_residual_norm."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(T, H, dt, seed, y=1.0, w_post=None, gate=None, kind="none", alpha=1.0, res=1.0, eps=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    shape = dict(none=None, channel=(H,), token=(T, 1), full=(T, H))[kind]
    return dict(y=(n(T, H) * y).to(dt), res=(n(T, H) * res).to(dt), w_post=None if w_post is None else ((1 + 0.2 * n(H)) * w_post).to(dt),
                gate=None if shape is None else ((1 + 0.2 * n(*shape)) * gate).to(dt), alpha=alpha, w_next=(1 + 0.2 * n(H)).to(dt), eps=eps)


CASES = {
    # rstd is 2^60 and alpha times the gate 2^80
    "small rows, large factors": dict(y=2.0 ** -60, w_post=1.0, gate=2.0 ** 40, kind="token", alpha=2.0 ** 40, res=2.0 ** 70),
    "small rows, a large alpha": dict(y=2.0 ** -60, w_post=1.0, alpha=2.0 ** 80, res=2.0 ** 70),
    # rstd is 2^-50 and alpha times the gate 2^-110
    "large rows, small factors": dict(y=2.0 ** 50, w_post=1.0, gate=2.0 ** -55, kind="token", alpha=2.0 ** -55, res=2.0 ** -110, eps=1e-6),
    # the weight times the gate is 2^140, alpha brings the result back
    "large weights and gates": dict(w_post=2.0 ** 70, gate=2.0 ** 70, kind="channel", alpha=2.0 ** -90, res=2.0 ** 50, column=2.0 ** -30),
    "large weights and gates of elements": dict(w_post=2.0 ** 70, gate=2.0 ** 70, kind="full", alpha=2.0 ** -90, res=2.0 ** 50, column=2.0 ** -30),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(3, 64), (130, 2080), (650, 2048), (40, 10240)])
@pytest.mark.parametrize("name", CASES)
def test_products_in_turn(name, T, H, dtype):
    """Off by the roundings of fp32 alone: 2^-18 of the terms' magnitudes, and half a step of the type.  `column`:
    weights and gates of all columns but one are 1, and that one's y is so many times the others', so that no
    partial product (y rstd, times the weight, times the gate) leaves fp32."""
    require_cuda()
    c, dt = dict(CASES[name]), DT[dtype]
    column = c.pop("column", None)
    a = make(T, H, dt, T + H, **c)
    if column is not None:
        at = H // 3
        big, large = a["w_post"][at].clone(), a["gate"][..., at].clone()
        a["w_post"].fill_(1.0), a["gate"].fill_(1.0)
        a["w_post"][at], a["gate"][..., at] = big, large
        a["y"][:, at] *= column
    got = binding.moe_residual_norm_mx8(**a)
    d = {n: v.double() if isinstance(v, torch.Tensor) else v for n, v in a.items()}
    z = d["y"] * torch.rsqrt(d["y"].square().mean(1, keepdim=True) + a["eps"]) * d["w_post"]
    z = a["alpha"] * z * (1.0 if a["gate"] is None else d["gate"])
    want, m = d["res"] + z, d["res"].abs() + z.abs()
    assert float(want.abs().max()) < torch.finfo(dt).max and (z != 0).any()
    half = torch.finfo(dt).eps / 2
    off = 2.0 ** -18 * m + half * want.abs() + torch.finfo(dt).smallest_normal * half
    assert ((got["out"].double() - want).abs() <= off).all()
    assert not (got["sf"] == 255).any() and got["u"].isfinite().all()
    other = binding.moe_residual_norm(**a)
    assert ((other["out"].double() - want).abs() <= off).all()
