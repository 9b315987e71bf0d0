"""moe_residual_norm and its gradients against the formulas in 64 bits.

Tolerance, per element: one unit in the last place of the output's type, plus
2^-19 of the sum of the magnitudes that were added (fp32 sums of up to 16384
terms in a fixed tree of at most 32-term chains: 32 * 2^-24 of that sum)."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ULP = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7, torch.float32: 2.0 ** -22}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 1e-38, torch.float32: 1e-38}
SUM = 2.0 ** -19
ALPHA, EPS = 0.375, 1e-5


def check(got, want, mag, what):
    dt = got.dtype
    g = got.double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    bound = ULP[dt] * want.abs() + SUM * mag + TINY[dt]
    bad = ~((g - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(((g - want).abs() / bound).max()))


def make(T, H, dtype, post, nxt, gate, seed=0, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed + 1000 * T + H)
    n = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    dt = DT[dtype]
    shape = dict(none=None, channel=(H,), token=(T, 1), full=(T, H))[gate]
    return dict(y=(2 * n(T, H)).to(dt), res=n(T, H).to(dt), w_post=(1 + 0.3 * n(H)).to(dt) if post else None,
                gate=None if shape is None else (0.5 + n(*shape)).to(dt), w_next=(1 + 0.3 * n(H)).to(dt) if nxt else None)


def forward64(s, alpha=ALPHA, eps=EPS):
    d = {k: None if v is None else v.double() for k, v in s.items()}
    got = {}
    if d["y"] is None:
        o = d["res"]
    else:
        z = d["y"]
        if d["w_post"] is not None:
            got["rstd_post"] = 1 / (z.square().mean(1) + eps).sqrt()
            z = z * got["rstd_post"][:, None] * d["w_post"]
        if d["gate"] is not None:
            z = z * d["gate"]
        o = d["res"] + alpha * z
        got["out"] = o
        got["mag"] = d["res"].abs() + abs(alpha) * z.abs()
    if d["w_next"] is not None:
        got["rstd_next"] = 1 / (o.square().mean(1) + eps).sqrt()
        got["u"] = o * got["rstd_next"][:, None] * d["w_next"]
    return got


def backward64(s, d_out, d_u, out, rp, rn, alpha=ALPHA):
    """Gradients and, for each, the sum of magnitudes behind it."""
    y = None if s["y"] is None else s["y"].double()
    H = out.shape[1]
    d = torch.zeros_like(out, dtype=torch.float64) if d_out is None else d_out.double()
    g, m = {}, {}
    md = d.abs()
    if s["w_next"] is not None:
        o, r = out.double(), rn.double()[:, None]
        v = d_u.double() * s["w_next"].double()
        d = d + r * v - o * r ** 3 / H * (v * o).sum(1, keepdim=True)
        md = md + r * v.abs() + o.abs() * r ** 3 / H * (v * o).abs().sum(1, keepdim=True)
        g["d_w_next"] = (d_u.double() * o * r).sum(0)
        m["d_w_next"] = (d_u.double() * o * r).abs().sum(0)
    g["d_res"], m["d_res"] = d, md
    if y is None:
        return g, m
    gate = torch.ones_like(y) if s["gate"] is None else s["gate"].double().expand_as(y)
    r = torch.ones_like(y[:, :1]) if s["w_post"] is None else rp.double()[:, None]
    w = torch.ones_like(y[0]) if s["w_post"] is None else s["w_post"].double()
    if s["gate"] is not None:
        dg, mg = alpha * d * y * r * w, abs(alpha) * md * (y * r * w).abs()
        axis = {1: 0, 2: None}[s["gate"].dim()]
        if axis == 0:
            g["d_gate"], m["d_gate"] = dg.sum(0), mg.sum(0)
        elif s["gate"].shape[1] == 1 and H != 1:
            g["d_gate"], m["d_gate"] = dg.sum(1, keepdim=True), mg.sum(1, keepdim=True)
        else:
            g["d_gate"], m["d_gate"] = dg, mg
    dz, mz = alpha * gate * d, abs(alpha) * gate.abs() * md
    if s["w_post"] is None:
        g["d_y"], m["d_y"] = dz, mz
        return g, m
    v, mv = dz * w, mz * w.abs()
    g["d_y"] = r * v - y * r ** 3 / H * (v * y).sum(1, keepdim=True)
    m["d_y"] = r * mv + y.abs() * r ** 3 / H * (mv * y.abs()).sum(1, keepdim=True)
    g["d_w_post"], m["d_w_post"] = (dz * y * r).sum(0), (mz * (y * r).abs()).sum(0)
    return g, m


def check_forward(got, want):
    assert set(got) == {k for k in want if k != "mag"}
    for k in ("rstd_post", "rstd_next"):
        if k in want:
            check(got[k], want[k], want[k], k)
    if "out" in want:
        check(got["out"], want["out"], want["mag"], "out")
    if "u" in want:
        # u follows out, whose fp32 error is SUM * mag
        o = want["out"] if "out" in want else None
        scale = want["u"].abs()
        if o is not None:
            scale = scale + want["u"].abs() * (want["mag"] / o.abs().clamp_min(1e-300))
        check(got["u"], want["u"], scale, "u")


SHAPES = [(1, 1), (3, 33), (5, 2047), (2, 256), (7, 1000), (4, 7168), (2, 16384), (300, 64), (61, 513), (40, 8192), (3, 9001)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_and_backward(T, H, dtype):
    require_cuda()
    for i, (post, nxt, gate) in enumerate([(True, True, "channel"), (True, False, "full"), (False, True, "token"),
                                           (True, True, "none"), (False, False, "token"), (False, True, "full")]):
        if H == 1 and gate == "full":
            continue  # [T, 1] is one factor per token
        s = make(T, H, dtype, post, nxt, gate, seed=i)
        got = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
        check_forward(got, forward64(s))
        g = torch.Generator(device="cuda").manual_seed(i)
        d_out = torch.randn((T, H), generator=g, device="cuda").to(DT[dtype])
        d_u = torch.randn((T, H), generator=g, device="cuda").to(DT[dtype]) if nxt else None
        if nxt and i % 2:
            d_out = None
        back = binding.moe_residual_norm_backward(d_out, d_u, s["y"], got["out"], s["w_post"], s["gate"], ALPHA, s["w_next"],
                                                  got.get("rstd_post"), got.get("rstd_next"))
        want, mag = backward64(s, d_out, d_u, got["out"], got.get("rstd_post"), got.get("rstd_next"))
        assert set(back) == set(want)
        for k in want:
            check(back[k], want[k], mag[k], f"{k} {post} {nxt} {gate}")


# several rows a CTA, tensors that end inside 16 bytes, rows of less than 16
# bytes, rows that fit the staging buffers in part and not at all
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,H", [(5001, 3), (4999, 7), (2501, 249), (4403, 510), (4403, 511), (1001, 2047), (457, 7167), (307, 9001), (305, 13001),
                                 (306, 16382), (307, 7168), (304, 14336)])
def test_many_rows_of_any_width(T, H, dtype):
    require_cuda()
    for i, (post, nxt, gate) in enumerate([(True, True, "channel"), (True, True, "full"), (False, False, "token")]):
        s = make(T, H, dtype, post, nxt, gate, seed=i)
        got = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
        check_forward(got, forward64(s))
        g = torch.Generator(device="cuda").manual_seed(i)
        d_out = torch.randn((T, H), generator=g, device="cuda").to(DT[dtype])
        d_u = torch.randn((T, H), generator=g, device="cuda").to(DT[dtype]) if nxt else None
        back = binding.moe_residual_norm_backward(d_out, d_u, s["y"], got["out"], s["w_post"], s["gate"], ALPHA, s["w_next"],
                                                  got.get("rstd_post"), got.get("rstd_next"))
        want, mag = backward64(s, d_out, d_u, got["out"], got.get("rstd_post"), got.get("rstd_next"))
        assert set(back) == set(want)
        for k in want:
            check(back[k], want[k], mag[k], f"{k} {post} {nxt} {gate}")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_norm_alone(dtype):
    """y None: the norm before the first block, and its gradients."""
    require_cuda()
    for T, H in [(1, 2048), (9, 77), (130, 4096)]:
        s = make(T, H, dtype, False, True, "none")
        s["y"] = None
        got = binding.moe_residual_norm(None, s["res"], w_next=s["w_next"], eps=EPS)
        check_forward(got, forward64(s))
        d_u = torch.randn((T, H), device="cuda").to(DT[dtype])
        back = binding.moe_residual_norm_backward(None, d_u, None, s["res"], w_next=s["w_next"], rstd_next=got["rstd_next"])
        want, mag = backward64(s, None, d_u, s["res"], None, got["rstd_next"])
        assert set(back) == set(want)
        for k in want:
            check(back[k], want[k], mag[k], k)


def test_gradients_against_differences():
    """The change of <d_out, out> + <d_u, u> along random directions, from the
    64-bit formula at +-1e-4: central differences are off by about 1e-8 of the
    third derivative, the gradients (f32) by 1e-6."""
    require_cuda()
    T, H = 13, 90
    for gate in ("channel", "token", "full"):
        s = make(T, H, "f32", True, True, gate, seed=5)
        f = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
        d_out, d_u = torch.randn((T, H), device="cuda"), torch.randn((T, H), device="cuda")
        g = binding.moe_residual_norm_backward(d_out, d_u, s["y"], f["out"], s["w_post"], s["gate"], ALPHA, s["w_next"],
                                               f["rstd_post"], f["rstd_next"])

        def loss(v):
            w = forward64(v)
            return float((w["out"] * d_out.double()).sum() + (w["u"] * d_u.double()).sum())

        for name, grad in (("y", "d_y"), ("res", "d_res"), ("w_post", "d_w_post"), ("w_next", "d_w_next"), ("gate", "d_gate")):
            way = torch.randn(s[name].shape, device="cuda", dtype=torch.float64)
            step = 1e-4
            up = loss({**s, name: s[name].double() + step * way})
            down = loss({**s, name: s[name].double() - step * way})
            want = (up - down) / (2 * step)
            have = float((g[grad].double() * way).sum())
            size = float((g[grad].double() * way).abs().sum())
            assert abs(have - want) <= 1e-5 * size, (gate, name, have, want)


def test_special_rows():
    """Zero rows, large rows, and rows with a NaN or an infinity: each stays in
    its row."""
    require_cuda()
    T, H = 8, 2048
    s = make(T, H, "f32", True, True, "channel", seed=3)
    s["y"][1] = 0
    s["res"][1] = 0
    s["y"][2] *= 1e16
    s["y"][3, 5] = float("nan")
    s["y"][4, 9] = float("inf")
    s["res"][5, 7] = float("-inf")
    got = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
    want = forward64(s)
    fine = [0, 1, 2, 6, 7]
    pick = lambda d: {k: v[fine] for k, v in d.items()}  # noqa: E731
    check_forward(pick(got), pick(want))
    assert torch.equal(got["out"][1], torch.zeros(H, device="cuda"))
    assert bool(got["u"][3].isnan().all()) and bool(got["out"][4, 9].isnan()) and bool((got["u"][5, 7]).isnan())
    assert bool((got["u"][5, :7] == 0).all())
    # eps = 0 is allowed where no row is zero
    live = {**s, "y": s["y"][6:].contiguous(), "res": s["res"][6:].contiguous()}
    check_forward(binding.moe_residual_norm(live["y"], live["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], 0.0),
                  forward64(live, eps=0.0))


def test_in_place_stream_graph_and_repeat():
    require_cuda()
    T, H = 257, 1536
    s = make(T, H, "bf16", True, True, "token", seed=9)
    ref = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
    d_out, d_u = torch.randn((T, H), device="cuda").bfloat16(), torch.randn((T, H), device="cuda").bfloat16()
    back = lambda: binding.moe_residual_norm_backward(d_out, d_u, s["y"], ref["out"], s["w_post"], s["gate"], ALPHA,  # noqa: E731
                                                      s["w_next"], ref["rstd_post"], ref["rstd_next"])
    first = back()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        res = s["res"].clone()
        got = binding.moe_residual_norm(s["y"], res, s["w_post"], s["gate"], ALPHA, s["w_next"], EPS, out=res)
        again = back()
    stream.synchronize()
    assert got["out"].data_ptr() == res.data_ptr()
    for k in ref:
        assert torch.equal(ref[k], got[k]), k
    for k in first:
        assert torch.equal(first[k], again[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = binding.moe_residual_norm(s["y"], s["res"], s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
        captured_back = back()
    graph.replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], captured[k]), k
    for k in first:
        assert torch.equal(first[k], captured_back[k]), k


def test_no_rows():
    require_cuda()
    H = 96
    s = make(1, H, "bf16", True, True, "channel")
    none = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    stat = torch.empty(0, device="cuda")
    got = binding.moe_residual_norm(none, none, s["w_post"], s["gate"], ALPHA, s["w_next"], EPS)
    assert got["out"].shape == (0, H) and got["u"].shape == (0, H)
    back = binding.moe_residual_norm_backward(none, none, none, none, s["w_post"], s["gate"], ALPHA, s["w_next"], stat, stat)
    for k in ("d_w_post", "d_w_next", "d_gate"):
        assert torch.equal(back[k], torch.zeros(H, device="cuda")), k


def test_refusals():
    require_cuda()
    s = make(4, 64, "bf16", True, True, "channel")
    y, res = s["y"], s["res"]
    with pytest.raises(ValueError):
        binding.moe_residual_norm(None, res)
    with pytest.raises(ValueError):
        binding.moe_residual_norm(None, res, w_post=s["w_post"], w_next=s["w_next"])
    with pytest.raises(ValueError):
        binding.moe_residual_norm(y, res, gate=torch.ones((3, 1), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        binding.moe_residual_norm(y.t(), res.t())
    with pytest.raises(TypeError):
        binding.moe_residual_norm(y, res, w_post=s["w_post"].float())
    with pytest.raises(ValueError):
        binding.moe_residual_norm(y[:2], res)
    with pytest.raises(binding.MoEError, match="INVALID_ARG"):
        binding.moe_residual_norm(y, res, w_next=s["w_next"], eps=-1.0)
    wide = torch.zeros((1, 16385), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.MoEError, match="UNSUPPORTED"):
        binding.moe_residual_norm(wide, wide)
    with pytest.raises(ValueError):
        binding.moe_residual_norm_backward(None, None, y, y)
    with pytest.raises(ValueError):
        binding.moe_residual_norm_backward(y, y, y, y)
    with pytest.raises(ValueError):
        binding.moe_residual_norm_backward(y, None, y, y, w_post=s["w_post"])
    with pytest.raises(binding.MoEError, match="WORKSPACE"):
        binding.moe_residual_norm_backward(y, None, y, y, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 64)
    with pytest.raises(binding.MoEError, match="INVALID_ARG"):
        binding.moe_residual_norm(flat, res)
