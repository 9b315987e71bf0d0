"""Microscaled 8-bit rows: the quantiser, the norm that writes them, the sort, the
grouped products, the layer of them and the block.

Quantisation, dequantisation and the sort are held bit for bit to a list of what 8
bits can hold.  The products' terms are exact, so their error is that of the tensor
cores' sums.  Those add 32 products and the sum so far at a time: each is cut at 2^-25
of the largest one's power of two (2^16 + 16 2^-9 is exact, 2^16 + 16 2^-10 gives
2^16) and the result at 24 bits (1 + 2^-23 is exact, 1 + 2^-24 gives 1).  No partial
sum and no product exceeds m, the sum of the terms' magnitudes, so one step is off by
at most (32 2^-25 + 2^-23) m = 1.125 2^-20 m, and K / 32 of them by that many times
as much; to that comes half a step of the output's type.  Sums that need no more than
24 bits are exact, which a test of whole numbers holds them to."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding
from mixture_experts_routed_gate_gb300.block import MoEBlock, Rows8, run_blocks

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


def sum_off(K):
    """How far a sum of K terms may be, relative to the sum of their magnitudes."""
    return -(-K // 32) * 1.125 * 2.0 ** -20


def grid(device):
    """The magnitudes of codes 0 to 126: 4 bits of exponent, 3 of mantissa."""
    return torch.tensor([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device=device)


def power(e):
    return ((e + 1023) << 52).view(torch.float64)


def quantize64(x):
    """Values and scale bytes of x [R, K] in 64 bits; NaN and 255 where the block has a NaN or an infinity."""
    held = grid(x.device)
    b = x.double().view(x.shape[0], -1, 32)
    a = b.abs()
    bad = ~a.isfinite().all(2, keepdim=True)
    a = torch.where(bad, torch.zeros_like(a), a)
    top = a.amax(2, keepdim=True)
    e = torch.full_like(top, -127, dtype=torch.int64)
    for n in range(-126, 121):  # the least power of two that brings the block to 448 or less
        e += (top > 448 * 2.0 ** (n - 1)).long()
    a = a / power(e)
    low = torch.searchsorted(held, a.contiguous(), right=True) - 1  # held[low] <= a
    high = (low + 1).clamp(max=126)
    up = held[high] - a < a - held[low]
    tie = held[high] - a == a - held[low]
    code = torch.where(up | (tie & (low % 2 == 1)), high, low)
    v = torch.sign(b) * held[code] * power(e)
    return torch.where(bad, torch.full_like(v, float("nan")), v).view(x.shape), torch.where(bad, torch.full_like(e, 128), e)[:, :, 0] + 127


def values64(q, sf):
    """What elements and scale bytes stand for, from the format."""
    bits = q.view(torch.uint8).long()
    held = torch.cat((grid(q.device), torch.full((1,), float("nan"), dtype=torch.float64, device=q.device)))
    v = torch.where(bits > 127, -1.0, 1.0).double() * held[bits % 128]
    unit = torch.where(sf == 255, torch.full_like(sf, float("nan"), dtype=torch.float64), power(sf.long() - 127))
    return (v.view(*q.shape[:-1], -1, 32) * unit[..., None]).view(q.shape)


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def rows8(R, K, g):
    x = torch.randn((R, K), generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-6, 6, (R, K // 32), generator=g, device="cuda").float()).repeat_interleave(32, 1)
    return binding.moe_quantize_mx8(x)


# ----------------------------------------------------------------------------- to 8 bits and back

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (64, 2048), (5, 1056), (130, 288), (2, 7168), (33, 64)])
def test_quantize(R, K, dtype):
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(R * 17 + K)
    x = torch.randn((R, K), generator=g, device="cuda")
    x = (x * torch.exp2(torch.randint(-6, 6, (R, K // 32), generator=g, device="cuda").float()).repeat_interleave(32, 1)).to(DT[dtype])
    q, sf = binding.moe_quantize_mx8(x)
    want, byte = quantize64(x)
    assert q.dtype == E4M3 and torch.equal(sf.long(), byte)
    assert same(values64(q, sf), want)
    for out in ("bf16", "f32"):  # both hold every value
        assert torch.equal(binding.moe_dequantize_mx8(q, sf, DT[out]).double(), want), out


def test_quantize_ties_and_edges():
    require_cuda()
    ties = torch.tensor([448.0, 447.9, 432.0, 432.1, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -6, 15 * 2.0 ** -10, 1.0625, 1.1875, 0.5, 256.0, 8.5, 0.0],
                        device="cuda")
    rows = [torch.cat((ties, -ties)) * s for s in (1.0, 2.0 ** -20, 2.0 ** 100, 2.0 ** -126, 2.0 ** -135)]
    over = torch.cat((ties, -ties))
    over[5] = 448.00003  # one step over: the scale is 2
    rows += [over, torch.zeros(32, device="cuda"), -torch.zeros(32, device="cuda"), torch.full((32,), 2.0 ** -149, device="cuda"),
             torch.full((32,), 1.75 * 2.0 ** 127, device="cuda")]
    for bad in (float("nan"), float("inf"), float("-inf"), -float("nan")):
        r = torch.randn(32, device="cuda")
        r[31] = bad
        rows.append(r)
    x = torch.stack(rows)
    q, sf = binding.moe_quantize_mx8(x)
    want, byte = quantize64(x)
    assert torch.equal(sf.long(), byte)
    assert same(values64(q, sf), want)
    assert same(binding.moe_dequantize_mx8(q, sf, torch.float32).double(), want)
    # every code with every scale byte, through the values' own types
    q = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(1, 256).expand(256, 256).contiguous().view(E4M3)
    sf = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(256, 1).expand(256, 8).contiguous()
    for dtype in ("f32", "bf16", "f16"):
        assert same(binding.moe_dequantize_mx8(q, sf, DT[dtype]), values64(q, sf).to(DT[dtype])), dtype


# ----------------------------------------------------------------------------- the norm

def norm_inputs(T, H, dt, gate, post, y, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    shape = dict(none=None, channel=(H,), token=(T, 1), full=(T, H))[gate]
    return dict(y=(2 * n(T, H)).to(dt) if y else None, res=n(T, H).to(dt), w_post=(1 + 0.2 * n(H)).to(dt) if post else None,
                gate=None if shape is None else (0.5 + 0.5 * n(*shape)).to(dt), alpha=0.7, w_next=(1 + 0.2 * n(H)).to(dt), eps=1e-5)


def norm64(a):
    """out, u and the statistics in 64 bits, and how far the kernel's fp32 values may be from them.

    A row's sum of squares takes an element through at most 27 additions, its rstd has half of their relative
    error, three roundings of the mean and two units of the root: 2^-19.  z = y * (alpha * gate * rstd) * (w * gate)
    has four roundings more and out one: 2^-18 of the terms' magnitudes m = |res| + |z|.  rstd_next has out's error,
    ||2^-18 m|| / ||out||, and its own; u that of out, of rstd_next and two roundings."""
    d = {n: v.double() if isinstance(v, torch.Tensor) else v for n, v in a.items()}
    got, z = {}, torch.zeros_like(d["res"])
    if a["y"] is not None:
        z = d["y"]
        if a["w_post"] is not None:
            r = torch.rsqrt(z.square().mean(1, keepdim=True) + a["eps"])
            got["rstd_post"] = r[:, 0], 2.0 ** -19 * r[:, 0]
            z = z * r * d["w_post"]
        z = a["alpha"] * z * (1.0 if a["gate"] is None else d["gate"])
    o, m = d["res"] + z, d["res"].abs() + z.abs()
    if a["y"] is not None:
        got["out"] = o, 2.0 ** -18 * m
    r = torch.rsqrt(o.square().mean(1, keepdim=True) + a["eps"])
    off = 2.0 ** -18 * m.norm(dim=1, keepdim=True) / o.norm(dim=1, keepdim=True).clamp(min=1e-300) + 2.0 ** -19
    got["rstd_next"] = r[:, 0], (off * r)[:, 0]
    got["u"] = o * r * d["w_next"], (2.0 ** -18 * m + (off + 2.0 ** -23) * o.abs()) * r * d["w_next"].abs()
    return got


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,H,gate,post,y", [(1, 2048, "channel", True, True), (3, 32, "none", True, True), (7, 96, "token", True, True),
                                             (333, 2080, "token", False, True), (65, 4128, "full", True, True), (129, 7168, "channel", True, True),
                                             (5, 16384, "channel", True, True), (400, 64, "none", False, False), (2000, 1056, "full", True, True),
                                             (3, 8224, "channel", True, True), (37, 14336, "none", False, False), (900, 7168, "channel", True, True),
                                             (700, 4096, "channel", False, True), (1500, 1024, "token", True, True), (320, 16384, "full", True, True),
                                             (310, 3104, "none", True, True), (1300, 2048, "none", False, False),
                                             (650, 16384, "full", True, True), (640, 9248, "channel", True, True)])
def test_norm(T, H, gate, post, y, dtype):
    """out, u and the statistics are within the roundings of fp32 (and a half step of their type) of the formula in
    64 bits; the rows are u's unrounded values in 8 bits: u itself quantised in 32 bits, and for 16-bit types
    within the roundings of u."""
    require_cuda()
    dt = DT[dtype]
    a = norm_inputs(T, H, dt, gate, post, y, T + H)
    got = binding.moe_residual_norm_mx8(**a)
    want = norm64(a)
    assert set(got) == set(want) | {"q", "sf"}
    for name, (v, off) in want.items():
        half = torch.finfo(got[name].dtype).eps / 2
        low = torch.finfo(got[name].dtype).smallest_normal * half
        assert got[name].dtype == (torch.float32 if name.startswith("rstd") else dt)
        assert ((got[name].double() - v).abs() <= off + half * (v.abs() + off) + low).all(), name
    q, sf = got["q"], got["sf"]
    alone = binding.moe_residual_norm_mx8(**a, with_u=False)
    assert "u" not in alone
    for name in alone:
        assert torch.equal(alone[name].view(torch.uint8), got[name].view(torch.uint8)), name
    if dtype == "f32":
        eq, es = binding.moe_quantize_mx8(got["u"])
        assert torch.equal(q.view(torch.uint8), eq.view(torch.uint8)) and torch.equal(sf, es)
        return
    u, off = want["u"]
    unit = power(sf.long() - 127).repeat_interleave(32, 1)
    assert ((values64(q, sf) - u).abs() <= 2.0 ** -4 * (u.abs() + off) + 2.0 ** -10 * unit + off).all()
    top, most = u.abs().view(T, -1, 32).amax(2), off.view(T, -1, 32).amax(2)
    unit = unit.view(T, -1, 32)[:, :, 0]
    assert (top - most <= 448 * unit).all() and ((top + most > 224 * unit) | (sf == 0)).all()


def test_norm_odd_values():
    """A row of zeros, a NaN, an infinity: each stays in its row, and in 8 bits in its block of 32 where the
    statistics allow (a NaN in the weight)."""
    require_cuda()
    H = 128
    x = torch.randn((5, H), device="cuda")
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 70] = float("inf")
    w = torch.ones(H, device="cuda")
    w[33] = float("nan")
    got = binding.moe_residual_norm_mx8(None, x, w_next=w)
    assert same(values64(got["q"], got["sf"])[:, 32:64], torch.full((5, 32), float("nan"), dtype=torch.float64, device="cuda"))
    assert (got["sf"][1] == 255).all() and (got["q"].view(torch.uint8)[1] == 0).all()
    assert (got["sf"][0, [0, 2, 3]] == 0).all()
    assert (got["sf"][2, 2] == 255).all()  # inf * rstd 0
    assert (got["sf"][3:, [0, 2, 3]] != 255).all()
    assert binding.moe_residual_norm_mx8(None, x[:0], w_next=w)["q"].shape == (0, H)
    # statistics without a finite root: a row of zeros without eps, rows too long for fp32 and too short
    x = torch.stack([torch.zeros(H, device="cuda"), torch.full((H,), 1e25, device="cuda"), torch.full((H,), 1e-18, device="cuda")])
    got = binding.moe_residual_norm_mx8(None, x, w_next=torch.ones(H, device="cuda"), eps=0.0)
    assert got["rstd_next"][0] == float("inf") and got["rstd_next"][1] == 0
    assert (got["sf"][0] == 255).all() and (got["q"].view(torch.uint8)[:2] == 0).all() and (got["sf"][1] == 0).all()
    assert ((values64(got["q"], got["sf"])[2] - 1).abs() <= 2.0 ** -4).all()


def test_norm_in_place_and_its_gradient():
    """out may be res; the gradient is moe_residual_norm_backward of the same saved values."""
    require_cuda()
    a = norm_inputs(50, 512, torch.bfloat16, "channel", True, True, 1)
    want = binding.moe_residual_norm_mx8(**a)
    res = a["res"].clone()
    got = binding.moe_residual_norm_mx8(**{**a, "res": res}, out=res)
    assert got["out"] is res and all(torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)) for n in want)
    d_out, d_u = torch.randn_like(res), torch.randn_like(res)
    g = binding.moe_residual_norm_backward(d_out, d_u, a["y"], want["out"], a["w_post"], a["gate"], a["alpha"], a["w_next"],
                                           want["rstd_post"], want["rstd_next"])
    # the formula's gradient in 64 bits, by autograd of the forward in 64 bits at the stored statistics' own precision:
    # bf16's half step (2^-9 of the value, d_res and d_y) and the stored out's (another one) bound both
    d = {n: v.double().requires_grad_() if isinstance(v, torch.Tensor) else v for n, v in a.items()}
    z = d["y"] * torch.rsqrt(d["y"].square().mean(1, keepdim=True) + a["eps"]) * d["w_post"] * d["gate"]
    o = d["res"] + a["alpha"] * z
    u = o * torch.rsqrt(o.square().mean(1, keepdim=True) + a["eps"]) * d["w_next"]
    ((d_out.double() * o).sum() + (d_u.double() * u).sum()).backward()
    for name, ref in (("d_res", d["res"]), ("d_y", d["y"]), ("d_w_post", d["w_post"]), ("d_w_next", d["w_next"]), ("d_gate", d["gate"])):
        assert (g[name].double() - ref.grad).norm() <= 2 * 2.0 ** -8 * ref.grad.norm(), name


# ----------------------------------------------------------------------------- the sort

@pytest.mark.parametrize("T,K,k", [(1, 32, 1), (1, 7168, 8), (64, 2048, 6), (333, 1056, 5), (7, 96, 32), (1000, 160, 3), (50, 16384, 2)])
def test_sort(T, K, k):
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(T)
    q, sf = rows8(T, K, g)
    n, more = T * k, 5
    pos = torch.randperm(n + more, generator=g, device="cuda")[:n].to(torch.int32).view(T, k)
    gone = torch.rand((T, k), generator=g, device="cuda") < 0.1
    pos = torch.where(gone, torch.tensor([-1, n + more, -7, 2 ** 31 - 1], device="cuda", dtype=torch.int32)[torch.randint(0, 4, (T, k), generator=g, device="cuda")], pos)
    out, osf = torch.full((n + more, K), 0x5a, dtype=torch.uint8, device="cuda"), torch.full((n + more, K // 32), 0xa5, dtype=torch.uint8, device="cuda")
    want, wsf = out.clone(), osf.clone()
    here = ~gone
    t = torch.arange(T, device="cuda").view(T, 1).expand(T, k)[here]
    want[pos[here].long()], wsf[pos[here].long()] = q.view(torch.uint8)[t], sf[t]
    got = binding.moe_sort_rows_mx8(q, sf, pos, n + more, out.view(E4M3), osf)
    assert torch.equal(got[0].view(torch.uint8), want) and torch.equal(got[1], wsf)


def test_sort_unaligned_scales():
    """The scales' bytes may start anywhere."""
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    q, sf = rows8(20, 256, g)
    pos = torch.randperm(40, generator=g, device="cuda").to(torch.int32).view(20, 2)
    want = binding.moe_sort_rows_mx8(q, sf, pos)
    room, place = torch.empty(20 * 8 + 3, dtype=torch.uint8, device="cuda"), torch.empty(40 * 8 + 1, dtype=torch.uint8, device="cuda")
    odd = room[3:].view(20, 8).copy_(sf)
    got = binding.moe_sort_rows_mx8(q, odd, pos, sf_out=place[1:].view(40, 8))
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])


def test_sort_past_2_31_bytes():
    require_cuda()
    T, K, k = 40000, 7168, 8  # 2.3e9 bytes of rows
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randint(0, 127, (T, K), generator=g, device="cuda", dtype=torch.uint8).view(E4M3)
    sf = torch.randint(0, 255, (T, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    pos = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    out, osf = binding.moe_sort_rows_mx8(q, sf, pos)
    for j in range(k):
        p = pos[:, j].long()
        assert torch.equal(out.view(torch.uint8)[p], q.view(torch.uint8)) and torch.equal(osf[p], sf)


# ----------------------------------------------------------------------------- the products

def routed(T, k, E, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    score = torch.randn((T, E), generator=g, device="cuda") + spread * torch.randn((E,), generator=g, device="cuda")
    idx = score.topk(k, dim=1).indices.to(torch.int32).contiguous()
    return binding.moe_build_dispatch(idx, None, E), g


def by_group(t):
    first = 0
    for e, n in enumerate(t["group_sizes"].tolist()):
        if n:
            yield e, slice(first, first + n)
        first += n


def product_and_size(a, b, t):
    """A_r B[g]^T in 64 bits, and the sum of the terms' magnitudes."""
    out = torch.empty((a.shape[0], b.shape[1]), dtype=torch.float64, device="cuda")
    mag = torch.empty_like(out)
    for e, at in by_group(t):
        out[at], mag[at] = a[at] @ b[e].t(), a[at].abs() @ b[e].abs().t()
    return out, mag


SHAPES = [(1, 1, 1, 32, 1), (1, 8, 8, 256, 128), (5, 2, 3, 64, 33), (64, 6, 64, 2048, 768), (301, 3, 5, 1056, 333), (130, 1, 1, 96, 257),
          (700, 2, 3, 288, 200), (257, 4, 7, 1024, 512), (96, 2, 6, 7168, 160), (40, 2, 600, 160, 64), (128, 1, 1, 512, 300), (129, 1, 1, 544, 256)]
# more units of rows than a CTA lists: of up to 128 rows, and of up to 256; several rounds of tiles of up to 256
SHAPES += [(1100, 2, 900, 96, 40), (10000, 4, 600, 32, 40), (20000, 4, 600, 32, 300), (5000, 2, 7, 288, 4100), (3000, 2, 7, 4128, 700),
           (2000, 1, 3, 4096, 2000)]


@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,k,E,K,N", SHAPES)
def test_product(T, k, E, K, N, out):
    require_cuda()
    t, g = routed(T, k, E, T + K)
    qa, sa = rows8(T * k, K, g)
    qb, sb = (x.view(E, N, -1) for x in rows8(E * N, K, g))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.moe_grouped_gemm_mx8(qa, sa, qb, sb, t, DT[out], err=err)
    want, mag = product_and_size(values64(qa, sa), values64(qb, sb), t)
    assert int(err.item()) == 0
    top = torch.finfo(DT[out]).max
    fits = want.abs() + sum_off(K) * mag < top
    step = torch.finfo(DT[out]).eps / 2
    bad = (got.double() - want).abs() > sum_off(K) * mag + step * want.abs() + torch.finfo(DT[out]).smallest_normal * step
    assert not (bad & fits).any(), int((bad & fits).sum())


@pytest.mark.parametrize("T,k,E,K,N", SHAPES + [(300, 2, 3, 7168, 300), (1000, 2, 5, 2080, 130)])
def test_product_of_whole_numbers(T, k, E, K, N):
    """Elements of up to 4, scales of 1, 2 and 4: every partial sum is a whole number of at most 7168 * 256 <
    2^24, and the result is exact in fp32."""
    require_cuda()
    t, g = routed(T, k, E, T + K)

    def whole(rows):
        q = torch.randint(-4, 5, (rows, K), generator=g, device="cuda").float()
        q *= torch.rand((rows, K), generator=g, device="cuda") < 0.5
        return q.to(E4M3), torch.randint(127, 130, (rows, K // 32), generator=g, device="cuda").to(torch.uint8)
    (qa, sa), (qb, sb) = whole(T * k), whole(E * N)
    qb, sb = qb.view(E, N, K), sb.view(E, N, K // 32)
    want, mag = product_and_size(values64(qa, sa), values64(qb, sb), t)
    assert float(mag.max()) < 2 ** 24
    assert torch.equal(binding.moe_grouped_gemm_mx8(qa, sa, qb, sb, t, torch.float32).double(), want)


def silu_products(t, qa, sa, gate, up):
    """h in 64 bits and how far the kernel's fp32 h may be: from the two sums, each product's derivative, and
    2^-20 of h for the exponential (2 + 1.2 |g| units), the quotient (2) and the product."""
    a, off = values64(qa, sa), sum_off(qa.shape[1])
    g, mg = product_and_size(a, values64(*gate), t)
    u, mu = product_and_size(a, values64(*up), t)
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.1 * off * mg * (u.abs() + off * mu) + off * mu * s.abs() + (2.0 ** -20 + 2.0 ** -22 * g.abs()) * h.abs()


@pytest.mark.parametrize("T,k,E,K,N", [(1, 1, 1, 32, 32), (1, 8, 8, 256, 128), (5, 2, 3, 64, 96), (64, 6, 64, 2048, 768), (301, 3, 5, 1056, 352),
                                       (700, 2, 3, 288, 224), (257, 4, 7, 1024, 512), (40, 2, 600, 160, 64), (129, 1, 1, 544, 256), (33, 1, 2, 7168, 160),
                                       (1100, 2, 900, 96, 64), (400, 2, 3, 4128, 96), (600, 1, 2, 4096, 160), (39000, 1, 600, 4096, 32),
                                       (4000, 1, 3, 4128, 512), (2000, 2, 5, 4096, 1056)])
def test_gate_up(T, k, E, K, N):
    require_cuda()
    t, g = routed(T, k, E, T + K)
    qa, sa = binding.moe_quantize_mx8(torch.randn((T * k, K), generator=g, device="cuda"))
    w = [binding.moe_quantize_mx8(torch.randn((E * n, m), generator=g, device="cuda") * m ** -0.5) for n, m in ((N, K), (N, K), (K, N))]
    parts = [x.view(E, n, -1) for (q, s), n in zip(w, (N, N, K)) for x in (q, s)]
    e = binding.Mx8Experts(*parts)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, sf = binding.moe_grouped_gate_up_silu_mx8(qa, sa, e, t, err=err)
    assert int(err.item()) == 0
    h, off = silu_products(t, qa, sa, parts[0:2], parts[2:4])
    unit = power(sf.long() - 127)
    wide = unit.repeat_interleave(32, 1)
    assert ((values64(q, sf) - h).abs() <= 2.0 ** -4 * (h.abs() + off) + 2.0 ** -10 * wide + off).all()
    top, most = h.abs().view(T * k, -1, 32).amax(2), off.view(T * k, -1, 32).amax(2)
    assert (top - most <= 448 * unit).all() and ((top + most > 224 * unit) | (sf == 0)).all()


def test_gate_up_of_many_rows_over_short_sums():
    """Tiles of 256 rows below 4096 features: many rows an expert and several rounds of tiles, none of them whole."""
    test_gate_up(4100, 1, 2, 2080, 2336)


def test_products_of_odd_values():
    """NaN scales, infinities in the sums and zeros stay in their rows and columns; rows of h in their blocks."""
    require_cuda()
    T, E, K, N = 200, 2, 320, 96
    t, g = routed(T, 1, E, 3)
    qa, sa = rows8(T, K, g)
    qb, sb = (x.view(E, N, -1).clone() for x in rows8(E * N, K, g))
    want, mag = product_and_size(values64(qa, sa), values64(qb, sb), t)
    sa[3, 9] = 255
    sa[150] = 255
    sb[0, 40, 0] = 255
    qa.view(torch.uint8)[10] = 0
    got = binding.moe_grouped_gemm_mx8(qa, sa, qb, sb, t, torch.float32)
    expert = torch.zeros(T, dtype=torch.long, device="cuda")
    expert[int(t["group_sizes"][0]):] = 1
    nan = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    nan[3] = nan[150] = True
    nan[expert == 0, 40] = True
    assert torch.equal(got.isnan(), nan)
    assert (got[10][~nan[10]] == 0).all()
    ok = ~nan
    ok[10] = False
    assert ((got.double() - want).abs() <= sum_off(K) * mag + 2.0 ** -24 * want.abs())[ok].all()
    e = binding.Mx8Experts(qb, sb, qb, torch.full_like(sb, 127), *(x.view(E, K, -1) for x in rows8(E * K, N, g)))
    q, sf = binding.moe_grouped_gate_up_silu_mx8(qa, sa, e, t)
    bad = torch.zeros((T, N // 32), dtype=torch.bool, device="cuda")
    bad[3] = bad[150] = True
    bad[expert == 0, 1] = True  # feature 40's block
    assert torch.equal(sf == 255, bad) and (q.view(torch.uint8).view(T, -1, 32)[bad] == 0).all()


def test_gate_up_of_large_gates():
    """Gates from -448 to 448: silu where exp(-g) leaves fp32, down to its least numbers, times an up of 2^80.  Each sum is
    one product, exact; exp's and the quotient's errors are far below half a step of 8 bits, but exp's result loses
    bits below 2^-126, where a gate counts with an error of 2^-149."""
    require_cuda()
    values = torch.tensor([0.0, 0.5, 1, 4, 16, 30, 60, 80, 88, 96, 104, 112, 256, 448], device="cuda")
    values = torch.cat((values, -values, values[:4]))
    K, N = 32, 32
    t, _ = routed(1, 1, 1, 0)
    qa = torch.zeros((1, K), device="cuda")
    qa[0, 0] = 1
    gate, up = torch.zeros((1, N, K), device="cuda"), torch.zeros((1, N, K), device="cuda")
    gate[0, :, 0], up[0, :, 0] = values, 1
    one = torch.full((1, N, 1), 127, dtype=torch.uint8, device="cuda")
    for pick in range(N):  # one feature at a time: the others' magnitudes would set the block's scale
        only = up.clone()
        only[0, :pick] = 0
        only[0, pick + 1:] = 0
        e = binding.Mx8Experts(gate.to(E4M3), one, only.to(E4M3), one + 80, torch.zeros((1, K, N), device="cuda").to(E4M3), one)
        q, sf = binding.moe_grouped_gate_up_silu_mx8(qa.to(E4M3), one[0, :1, 0].view(1, 1), e, t)
        g = float(values[pick])
        want = torch.tensor(g, dtype=torch.float64)
        want = float(want * torch.sigmoid(want)) * 2.0 ** 80
        got = float(values64(q, sf)[0, pick])
        assert abs(got - want) <= 2.0 ** -4 * abs(want) * 1.001 + abs(g) * 2.0 ** -149 * 2.0 ** 80 + 2.0 ** -136, (g, got, want)


def test_nothing_to_do():
    """No tokens, no rows: empty results, at every entry point."""
    require_cuda()
    t, g = routed(3, 2, 4, 0)
    q, sf = torch.empty((0, 64), device="cuda").to(E4M3), torch.empty((0, 2), dtype=torch.uint8, device="cuda")
    w = [x.view(4, n, -1) for n, m in ((96, 64), (96, 64), (64, 96)) for x in rows8(4 * n, m, g)]
    e = binding.Mx8Experts(*w)
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert binding.moe_quantize_mx8(torch.empty((0, 64), device="cuda"))[0].shape == (0, 64)
    assert binding.moe_dequantize_mx8(q, sf).shape == (0, 64)
    assert binding.moe_sort_rows_mx8(q, sf, none)[0].shape == (0, 64)
    assert binding.moe_grouped_gate_up_silu_mx8(q, sf, e, t)[0].shape == (0, 96)
    assert binding.moe_grouped_gemm_mx8(q, sf, w[0], w[1], t).shape == (0, 96)
    x, w_g, bias, w = layer(2, 256, 64, 4, 2, "f16")
    assert binding.moe_forward_mx8(x[:0], w_g, bias, binding.Mx8Experts.from_weights(*w), 2).shape == (0, 256)


def test_rows_behind_the_last_group_are_left():
    require_cuda()
    T, E, K, N, more = 50, 3, 128, 96, 30
    t, g = routed(T, 2, E, 4)
    qa, sa = rows8(2 * T + more, K, g)
    w = [x.view(E, n, -1) for n, m in ((N, K), (N, K), (K, N)) for x in rows8(E * n, m, g)]
    for dt in (torch.float32, torch.float16):
        out = torch.full((2 * T + more, N), 7.0, device="cuda", dtype=dt)
        binding.moe_grouped_gemm_mx8(qa, sa, w[0], w[1], t, dt, out=out)
        assert (out[2 * T:] == 7).all() and not (out[:2 * T] == 7).all()
    q, s = torch.full((2 * T + more, N), 3, dtype=torch.uint8, device="cuda"), torch.full((2 * T + more, N // 32), 3, dtype=torch.uint8, device="cuda")
    binding.moe_grouped_gate_up_silu_mx8(qa, sa, binding.Mx8Experts(*w), t, q.view(E4M3), s)
    assert (q[2 * T:] == 3).all() and (s[2 * T:] == 3).all() and not (s[:2 * T] == 3).all()


def test_past_2_31_elements():
    """Weights of more than 2^31 bytes and a result of more than 2^31 elements, at places on both sides of it."""
    require_cuda()
    T, k, E, K, N = 64, 4, 300, 4096, 2048
    t, g = routed(T, k, E, 1)
    qa, sa = rows8(T * k, K, g)
    qb = torch.randint(0, 100, (E, N, K), generator=g, device="cuda", dtype=torch.uint8).view(E4M3)
    sb = torch.randint(120, 130, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    got = binding.moe_grouped_gemm_mx8(qa, sa, qb, sb, t, torch.float32)
    for e, at in by_group(t):
        if e < 5 or e > E - 5:
            a, b = values64(qa[at], sa[at]), values64(qb[e], sb[e])
            off = sum_off(K) * (a.abs() @ b.abs().t()) + 2.0 ** -24 * (a @ b.t()).abs()
            assert ((got[at].double() - a @ b.t()).abs() <= off).all(), e
    del qb, sb
    T, E, K, N = 90000, 3, 32, 24001
    t, g = routed(T, 1, E, 2)
    (qa, sa), (qb, sb) = rows8(T, K, g), (x.view(E, N, -1) for x in rows8(E * N, K, g))
    got = binding.moe_grouped_gemm_mx8(qa, sa, qb, sb, t, torch.bfloat16)
    for e, at in by_group(t):
        for r in (at.start, at.stop - 1):
            a, b = values64(qa[r:r + 1], sa[r:r + 1]), values64(qb[e], sb[e])
            want = (a @ b.t())[0]
            off = sum_off(K) * (a.abs() @ b.abs().t())[0] + 2.0 ** -8 * want.abs() + 2.0 ** -134
            assert ((got[r].double() - want).abs() <= off).all(), r


def test_two_streams_at_once():
    """No call keeps state: products of different sizes on two streams, in turn and together, give the same bits."""
    require_cuda()
    calls = []
    for T, k, E, K, N in ((700, 2, 3, 1024, 512), (64, 6, 64, 512, 256)):
        t, g = routed(T, k, E, T)
        a, b = rows8(T * k, K, g), [x.view(E, N, -1) for x in rows8(E * N, K, g)]
        calls.append(lambda a=a, b=b, t=t: binding.moe_grouped_gemm_mx8(*a, *b, t, torch.float32))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(c())
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for g, w in zip(got, want) for x in g)


def test_unaligned_scales_and_results():
    """Scale bytes and results may start where their types do."""
    require_cuda()
    T, E, K, N = 77, 3, 512, 130
    t, g = routed(T, 2, E, 6)
    qa, sa = rows8(2 * T, K, g)
    qb, sb = (x.view(E, N, -1) for x in rows8(E * N, K, g))
    want = binding.moe_grouped_gemm_mx8(qa, sa, qb, sb, t, torch.bfloat16)
    for shift in (1, 2, 4):
        def moved(s):
            room = torch.empty(s.numel() + shift, dtype=torch.uint8, device="cuda")[shift:].view(s.shape)
            return room.copy_(s)
        assert torch.equal(binding.moe_grouped_gemm_mx8(qa, moved(sa), qb, moved(sb), t, torch.bfloat16), want)


# ----------------------------------------------------------------------------- the layer and the block

def layer(T, d_h, d_e, E, k, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dt = DT[dtype]
    x, w_g = n(T, d_h).to(dt), (n(E, d_h) * d_h ** -0.5).to(dt)
    w = [(n(E, a, b) * b ** -0.5).to(dt) for a, b in ((d_e, d_h), (d_e, d_h), (d_h, d_e))]
    return x, w_g, 0.2 * n(E), w


@pytest.mark.parametrize("T,d_h,d_e,E,k,dtype", [(1, 256, 64, 4, 2, "f16"), (64, 512, 192, 16, 4, "bf16"), (300, 256, 320, 7, 3, "f16"),
                                                 (1100, 512, 128, 24, 2, "bf16")])
def test_forward_is_its_parts(T, d_h, d_e, E, k, dtype):
    require_cuda()
    x, w_g, bias, w = layer(T, d_h, d_e, E, k, dtype)
    e = binding.Mx8Experts.from_weights(*w)
    q, sf = binding.moe_quantize_mx8(x)
    idx, tw = binding.moe_gate_topk(x, w_g, bias, k)
    t = binding.moe_build_dispatch(idx, tw, E)
    sq, ss = binding.moe_sort_rows_mx8(q, sf, t["token_topk_to_pos"])
    y = binding.moe_grouped_gemm_mx8(*binding.moe_grouped_gate_up_silu_mx8(sq, ss, e, t), e.q_down, e.sf_down, t, DT[dtype])
    want = binding.moe_reduce_fused(y, t["token_topk_to_pos"], tw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(binding.moe_forward_mx8(x, w_g, bias, e, k, err=err), want)
    assert torch.equal(binding.moe_forward_mx8(x, w_g, bias, e, k, (q, sf), err=err), want)
    assert int(err.item()) == 0
    # a replayed graph on other tokens
    graph, ws = torch.cuda.CUDAGraph(), torch.empty(binding.forward_mx8_workspace_bytes(T, d_h, d_e, E, k, DT[dtype]), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    with torch.cuda.graph(graph):
        binding.moe_forward_mx8(x, w_g, bias, e, k, ws=ws, out=out)
    x.copy_(x.flip(0))
    graph.replay()
    assert torch.equal(out, binding.moe_forward_mx8(x, w_g, bias, e, k))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = binding.moe_forward_mx8(x, w_g, bias, e, k)
    side.synchronize()
    assert torch.equal(other, out)


def test_blocks_of_all_kinds():
    """16-bit, 8-bit and 4-bit blocks in turn: each is the entry points' calls in order."""
    require_cuda()
    T, d_h, d_e, E, k = 70, 512, 128, 8, 2
    x, w_g, bias, w = layer(T, d_h, d_e, E, k, "bf16")
    one = torch.ones(d_h, dtype=torch.bfloat16, device="cuda")
    e8, e4 = binding.Mx8Experts.from_weights(*w), binding.Mx4Experts.from_weights(*w)
    make = lambda experts, last=False: MoEBlock(w_g, bias, experts, k, w_post=one, alpha=0.5, w_next=None if last else one * 0.9)  # noqa: E731
    u, res = run_blocks(iter([make(e8), make(tuple(w)), make(e8), make(e8), make(e4, True)]), x, one)
    assert u is None
    r = x.clone()
    f = binding.moe_residual_norm_mx8(None, r, w_next=one)
    for kind, nxt in (("8", "16"), ("16", "8"), ("8", "8"), ("8", "4"), ("4", None)):
        if kind == "8":
            y = binding.moe_forward_mx8(f["u"], w_g, bias, e8, k, (f["q"], f["sf"]))
        else:
            y = binding.moe_forward(f["u"], w_g, bias, *w, k) if kind == "16" else binding.moe_forward_mx4(f["u"], w_g, bias, e4, k)
        norm = binding.moe_residual_norm_mx8 if nxt == "8" else binding.moe_residual_norm
        f = norm(y, r, one, None, 0.5, None if nxt is None else one * 0.9)
        r = f["out"]
    assert torch.equal(res, r)
    rows = make(e8)(torch.zeros_like(x), x.clone(), rows8=True)[0]
    assert isinstance(rows, Rows8) and rows.q.dtype == E4M3


def test_refusals():
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(0)
    q, sf = rows8(8, 64, g)
    pos = torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    x = torch.randn((8, 64), device="cuda")
    for call in (lambda: binding.moe_quantize_mx8(x[:, :40].contiguous()), lambda: binding.moe_quantize_mx8(x.t()),
                 lambda: binding.moe_dequantize_mx8(q, sf[:4]), lambda: binding.moe_sort_rows_mx8(q[:4], sf[:4], pos),
                 lambda: binding.moe_sort_rows_mx8(q, sf[:, :1].contiguous(), pos), lambda: binding.moe_residual_norm_mx8(x, x, w_next=None),
                 lambda: binding.moe_residual_norm_mx8(None, x, w_post=x[0], w_next=x[0]), lambda: binding.moe_residual_norm_mx8(x, x, w_next=x[0, :32]),
                 lambda: binding.moe_residual_norm_mx8(None, x[:, :40].contiguous(), w_next=x[0, :40]),
                 lambda: binding.Mx8Experts(q[None], sf[None], q[None], sf[None], q[None], sf[None]),
                 lambda: binding.moe_grouped_gemm_mx8(q, sf, q[None], sf[None], binding.moe_build_dispatch(pos, None, 2)),
                 lambda: binding.moe_grouped_gemm_mx8(q, sf, q[None, :, :32].contiguous(), sf[None, :, :1].contiguous(), {})):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: binding.moe_dequantize_mx8(q.view(torch.uint8), sf), lambda: binding.moe_sort_rows_mx8(q, sf.int(), pos),
                 lambda: binding.moe_sort_rows_mx8(q, sf, pos.long()), lambda: binding.moe_quantize_mx8(x.double())):
        with pytest.raises(TypeError):
            call()


def test_the_extension_makes_the_same_calls(monkeypatch):
    """With the extension of the short calls and without it: the same bits, the same refusals."""
    require_cuda()
    binding.lib()
    host = binding._host
    assert host is not None
    T, k, E, K, N = 70, 3, 5, 256, 96
    t, g = routed(T, k, E, 9)
    (q, sf), w = rows8(T, K, g), [x.view(E, n, -1) for n, m in ((N, K), (N, K), (K, N)) for x in rows8(E * n, m, g)]
    x, d_out, tw = torch.randn((T * k, K), device="cuda").half(), torch.randn((T, K), device="cuda").half(), torch.rand((T, k), device="cuda")
    pos, token = t["token_topk_to_pos"], t["sorted_token_idx"]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    made = []

    def calls():
        out = []
        for gate in ("none", "channel", "token", "full"):
            for post, y in ((True, True), (False, True), (False, False)):
                if y or gate == "none":
                    a = norm_inputs(T, K, torch.bfloat16, gate, post, y, 5)
                    for with_u in (True, False):
                        out.append(binding.moe_residual_norm_mx8(**a, with_u=with_u))
        a = norm_inputs(T, K, torch.float16, "channel", True, True, 6)
        res = a["res"].clone()
        out.append(binding.moe_residual_norm_mx8(**{**a, "res": res}, out=res))
        assert out[-1]["out"] is res or out[-1]["out"].data_ptr() == res.data_ptr()
        out.append(binding.moe_sort_rows_mx8(q, sf, pos))
        for weights, e in ((tw, err), (None, None)):
            out.append(binding.moe_reduce_fused_backward(d_out, x, pos, weights, token, e))
        e = binding.Mx8Experts(*w)
        out.append((e.E, e.d_e, e.d_h))
        rows = binding.moe_sort_rows_mx8(q, sf, pos)
        h = binding.moe_grouped_gate_up_silu_mx8(*rows, e, t, err=err)
        out += [h] + [binding.moe_grouped_gemm_mx8(*h, e.q_down, e.sf_down, t, d) for d in DT.values()]
        return out

    def bits(v):
        if isinstance(v, dict):
            return {n: bits(x) for n, x in v.items()}
        if isinstance(v, (tuple, list)):
            return [bits(x) for x in v]
        return (v.dtype, v.shape, v.view(torch.uint8).tolist()) if isinstance(v, torch.Tensor) else v

    class Counted:
        def __getattr__(self, name):
            def f(*a):
                r = getattr(host, name)(*a)
                made.append((name, r is not None))
                return r
            return f
    monkeypatch.setattr(binding, "_host", Counted())
    fast = bits(calls())
    assert all(yes for _, yes in made) and {n for n, _ in made} == {"norm_mx8", "sort_rows_mx8", "reduce_fused_backward", "experts_mx8",
                                                                    "grouped_gemm_mx8", "grouped_gate_up_silu_mx8"}
    with torch.inference_mode():
        assert bits(calls()) == fast and binding.moe_sort_rows_mx8(q, sf, pos)[0].is_inference()
    monkeypatch.setattr(binding, "_host", None)
    assert bits(calls()) == fast
    e = binding.Mx8Experts(*w)
    wrong = [lambda: binding.moe_sort_rows_mx8(q, sf, pos.long()), lambda: binding.moe_sort_rows_mx8(q, sf[:, :4], pos),
             lambda: binding.moe_sort_rows_mx8(q.view(torch.uint8), sf, pos), lambda: binding.moe_sort_rows_mx8(q, sf, pos[:5]),
             lambda: binding.moe_reduce_fused_backward(d_out.float(), x, pos, tw, token), lambda: binding.moe_reduce_fused_backward(d_out, x, pos, tw, token[:4]),
             lambda: binding.moe_reduce_fused_backward(d_out, x, pos, tw.half(), token), lambda: binding.moe_reduce_fused_backward(d_out.t(), x, pos, tw, token),
             lambda: binding.moe_grouped_gemm_mx8(q, sf, *w[4:], t), lambda: binding.moe_grouped_gemm_mx8(q, sf, w[0], w[1], {}),
             lambda: binding.moe_grouped_gemm_mx8(q, sf, w[0], w[1], t, torch.float64), lambda: binding.moe_grouped_gemm_mx8(q, sf, w[0], w[1], t, err=tw),
             lambda: binding.moe_grouped_gate_up_silu_mx8(*rows8(4, 64, g), e, t), lambda: binding.Mx8Experts(*w[2:], *w[:2]),
             lambda: binding.moe_residual_norm_mx8(d_out, x, w_next=x[0]), lambda: binding.moe_residual_norm_mx8(None, x, w_next=x[0].float()),
             lambda: binding.moe_residual_norm_mx8(None, x, w_next=x[0], alpha="1"), lambda: binding.moe_residual_norm_mx8(None, x, w_next=x[0], eps=-1.0),
             lambda: binding.moe_residual_norm_mx8(x, x, gate=x[0, :32], w_next=x[0]), lambda: binding.moe_residual_norm_mx8(None, x, None, x[0], w_next=x[0])]
    told = []
    for h in (None, host):
        monkeypatch.setattr(binding, "_host", h)
        for f in wrong:
            with pytest.raises(Exception) as caught:
                f()
            told.append((type(caught.value), str(caught.value)))
    assert told[:len(wrong)] == told[len(wrong):]
