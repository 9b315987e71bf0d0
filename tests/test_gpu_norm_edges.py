"""The norms at their edges: rows of less than 16 bytes, no rows at all, rows
whose size lies far from one.  The references and their tolerances are those of
the norms' own tests."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding
from test_gpu_norm import ALPHA, DT, EPS, backward64, check, forward64, make

pytestmark = pytest.mark.gpu


def check_forward(got, want, w_next, eps):
    """A row of one or two elements may be all cancellation (out far below what
    was added), and its rstd then carries out's own error, off * mag: by first
    order a share of mean(|out| mag) / (mean(out^2) + eps) of it."""
    assert set(got) == {k for k in want if k != "mag"}
    if "rstd_post" in want:
        check(got["rstd_post"], want["rstd_post"], want["rstd_post"], "rstd_post")
    check(got["out"], want["out"], want["mag"], "out")
    if w_next is not None:
        o, r, u = want["out"], want["rstd_next"][:, None], want["u"]
        share = (o.abs() * want["mag"]).mean(1, keepdim=True) / (o.square().mean(1, keepdim=True) + eps)
        check(got["rstd_next"][:, None], r, r * (1 + share), "rstd_next")
        check(got["u"], u, w_next.double().abs() * r * want["mag"] + u.abs() * (1 + share), "u")


NARROW = [(T, H) for H in (1, 2, 3, 4, 5, 6, 7, 8, 9, 13) for T in list(range(1, 18)) + [700, 5003]]


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_rows_of_a_few_bytes(dtype, gate):
    """Several rows lie in the tensor's last, incomplete 16 bytes."""
    require_cuda()
    for T, H in NARROW:
        if H == 1 and gate == "full":
            continue  # [T, 1] is one factor per token
        s = make(T, H, dtype, True, True, gate)
        got = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
        check_forward(got, forward64(s), s["w_next"], EPS)
        g = torch.Generator(device="cuda").manual_seed(T + H)
        d_out, d_u = (torch.randn((T, H), generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
        back = binding.moe_residual_norm_backward(d_out, d_u, s["y"], got["out"], s["w_post"], s["gate"], ALPHA, s["w_next"],
                                                  got["rstd_post"], got["rstd_next"])
        want, mag = backward64(s, d_out, d_u, got["out"], got["rstd_post"], got["rstd_next"])
        assert set(back) == set(want)
        for k in want:
            check(back[k], want[k], mag[k], f"{k} {T} {H}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e15, 1e-15])
@pytest.mark.parametrize("post,nxt", [(True, False), (False, True), (True, True)])
def test_gradients_of_very_large_and_very_small_rows(post, nxt, scale, dtype):
    """eps = 0; no step on the way may hold rstd^3, 1e45 or 1e-45 here."""
    require_cuda()
    for T, H in ((9, 200), (5, 2047), (3, 7168)):
        for gate in ("channel", "token", "full", "none"):
            s = make(T, H, dtype, post, nxt, gate, seed=1)
            s["y"], s["res"] = s["y"] * scale, s["res"] * scale
            got = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], 0.0)
            check_forward(got, forward64(s, eps=0.0), s["w_next"], 0.0)
            g = torch.Generator(device="cuda").manual_seed(T)
            d_out = (torch.randn((T, H), generator=g, device="cuda") / scale).to(DT[dtype])
            d_u = torch.randn((T, H), generator=g, device="cuda").to(DT[dtype]) if nxt else None
            back = binding.moe_residual_norm_backward(d_out, d_u, s["y"], got["out"], s["w_post"], s["gate"], ALPHA, s["w_next"],
                                                      got.get("rstd_post"), got.get("rstd_next"))
            want, mag = backward64(s, d_out, d_u, got["out"], got.get("rstd_post"), got.get("rstd_next"))
            for k in want:
                check(back[k], want[k], mag[k], f"{k} {T} {H} {gate}")


def test_gradient_of_a_gate_per_token_at_width_one():
    """[T, 1] is a gate per token at any width: its gradient is fp32."""
    require_cuda()
    s = make(7, 1, "bf16", True, False, "token")
    got = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, None, EPS)
    d_out = torch.randn((7, 1), device="cuda").bfloat16()
    back = binding.moe_residual_norm_backward(d_out, None, s["y"], got["out"], s["w_post"], s["gate"], ALPHA, None, got["rstd_post"])
    want, mag = backward64(s, d_out, None, got["out"], got["rstd_post"], None)
    assert back["d_gate"].dtype is torch.float32
    check(back["d_gate"], want["d_gate"], mag["d_gate"], "d_gate")


@pytest.mark.parametrize("post,nxt,gate", [(True, False, "none"), (True, False, "channel"), (False, False, "token"), (False, True, "full")])
def test_no_rows(post, nxt, gate):
    require_cuda()
    H = 48
    s = make(0, H, "bf16", post, nxt, gate)
    none, stat = s["res"], torch.empty(0, device="cuda")
    got = binding.moe_residual_norm(s["y"], none, s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
    assert got["out"].shape == (0, H)
    back = binding.moe_residual_norm_backward(none, none if nxt else None, s["y"], none, s["w_post"], s["gate"], ALPHA, s["w_next"],
                                              stat if post else None, stat if nxt else None)
    for k in ("d_w_post", "d_w_next"):
        if k in back:
            assert torch.equal(back[k], torch.zeros(H, device="cuda")), k
    if gate == "channel":
        assert torch.equal(back["d_gate"], torch.zeros(H, device="cuda"))
