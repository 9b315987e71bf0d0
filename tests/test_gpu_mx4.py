"""Microscaled 4-bit rows and their grouped product.

Quantisation and dequantisation are held bit for bit to a list of what 4 bits
can hold.  The product's terms are exact, so its error is that of fp32 sums:
2^-20 of the sum of the terms' magnitudes (the tensor cores add 64 products at
a time, each aligned to the largest and cut at 24 bits or more, then up to 512
such sums in fp32), plus one unit in the last place of the output's type."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding, workloads

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ULP = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7, "f32": 2.0 ** -23}
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantize64(x):
    """Values and scale exponents of x [R, K] in 64 bits; NaN where the block has a NaN or an infinity."""
    grid = GRID.to(x.device)
    b = x.double().view(x.shape[0], -1, 32)
    a = b.abs()
    bad = ~a.isfinite().all(2, keepdim=True)
    top = torch.where(bad, torch.zeros_like(a[:, :, :1]), a.amax(2, keepdim=True))
    e = torch.where(top > 0, ((top.view(torch.int64) >> 52) & 2047) - 1023 - 2, -127).clamp(-127, 127)
    unit = ((e + 1023) << 52).view(torch.float64)
    near = (a / unit)[..., None] - grid
    d = near.abs()
    best = d.amin(3, keepdim=True)
    ok = d == best  # one, or two at a tie: then the even code
    code = torch.arange(8, device=x.device)
    ok = ok & ((code % 2 == 0) | (ok.sum(3, keepdim=True) == 1))
    v = torch.sign(b) * (ok.to(torch.float64) * grid).sum(3) * unit
    return torch.where(bad, torch.full_like(v, float("nan")), v).view(x.shape), torch.where(bad, torch.full_like(e, 128), e)[:, :, 0]


def values64(q, sf):
    """What elements and scale bytes stand for, from the format."""
    held = torch.cat((GRID, -GRID)).to(q.device)
    v = torch.stack((held[(q % 16).long()], held[(q // 16).long()]), -1).view(*q.shape[:-1], -1, 32)
    unit = ((sf.long() + 896) << 52).view(torch.float64)
    return torch.where(sf == 255, torch.full_like(unit, float("nan")), unit)[..., None].mul(v).view(*q.shape[:-1], -1)


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (64, 2048), (5, 1056), (130, 288), (2, 7168), (33, 64)])
def test_quantize(R, K, dtype):
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(R * 17 + K)
    x = torch.randn((R, K), generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-6, 6, (R, K // 32), generator=g, device="cuda").float()).repeat_interleave(32, 1)
    x = x.to(DT[dtype])
    q, sf = binding.moe_quantize_mx4(x)
    want, e = quantize64(x)
    assert torch.equal(sf.long(), e + 127)
    assert same(values64(q, sf), want)
    for out in ("bf16", "f32"):
        assert torch.equal(binding.moe_dequantize_mx4(q, sf, DT[out]).double(), want), out


def test_quantize_ties_and_edges():
    require_cuda()
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, 4.0, 0.1, 0.2500001, 0.2499999, 5.0000005, 4.9999995],
                        device="cuda")
    rows = [torch.cat((ties, -ties)) * s for s in (1.0, 2.0 ** -20, 2.0 ** 100, 2.0 ** -140, 2.0 ** -147)]
    rows += [torch.zeros(32, device="cuda"), -torch.zeros(32, device="cuda"), torch.full((32,), 2.0 ** -149, device="cuda"),
             torch.full((32,), torch.finfo(torch.float32).max, device="cuda")]
    for bad in (float("nan"), float("inf"), float("-inf")):
        r = torch.randn(32, device="cuda")
        r[31] = bad
        rows.append(r)
    x = torch.stack(rows)
    q, sf = binding.moe_quantize_mx4(x)
    want, e = quantize64(x)
    assert torch.equal(sf.long(), e + 127)
    assert same(values64(q, sf), want)
    assert same(binding.moe_dequantize_mx4(q, sf, torch.float32).double(), want)
    # every code with every scale byte, through the values' own types
    q = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(1, 16, 16).expand(256, 16, 16).reshape(256, 256).contiguous()
    sf = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(256, 1).expand(256, 16).contiguous()
    for dtype in ("f32", "bf16", "f16"):
        assert same(binding.moe_dequantize_mx4(q, sf, DT[dtype]), values64(q, sf).to(DT[dtype])), dtype


def test_quantize_gathers_rows():
    require_cuda()
    x = torch.randn((40, 160), device="cuda").bfloat16()
    idx = torch.tensor([3, 3, 39, 0, 17, 5, 3], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, sf = binding.moe_quantize_mx4(x, idx, err=err)
    want, _ = quantize64(x[idx.long()])
    assert torch.equal(values64(q, sf), want) and int(err.item()) == 0
    idx[2], idx[5] = 40, -1
    q, sf = binding.moe_quantize_mx4(x, idx, err=err)
    want = quantize64(x[idx.long().clamp(0, 39)])[0]
    want[2] = 0
    want[5] = 0
    assert torch.equal(values64(q, sf), want) and int(err.item()) == 5


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("T,K,rows", [(700, 1024, 1400), (1300, 1056, 5000), (617, 9216, 1301)])
def test_quantize_gathers_repeated_rows(T, K, rows, dtype):
    """Many rows of few tokens: some tokens have no row, one has thousands, some
    indexes are out of range."""
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, K), generator=g, device="cuda").to(DT[dtype])
    idx = torch.randint(0, T, (rows,), generator=g, device="cuda", dtype=torch.int32)
    idx[100:rows - 300] = torch.where(idx[100:rows - 300] % 3 == 0, torch.full_like(idx[100:rows - 300], 5), idx[100:rows - 300])
    idx[3], idx[rows - 1], idx[77] = T, -7, 2 ** 31 - 1
    raw_q = torch.full((4096 + rows * K // 2 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    raw_s = torch.full((4096 + rows * K // 32 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, sf = binding.moe_quantize_mx4(x, idx, q=raw_q[4096:-4096].view(rows, K // 2), sf=raw_s[4096:-4096].view(rows, K // 32), err=err)
    good = (idx >= 0) & (idx < T)
    want = quantize64(x)[0][idx.long().clamp(0, T - 1)]
    want[~good] = 0
    assert torch.equal(values64(q, sf), want) and int(err.item()) == 5
    one_q, one_sf = binding.moe_quantize_mx4(x)  # the scale bytes too
    assert torch.equal(q[good], one_q[idx[good].long()]) and torch.equal(sf[good], one_sf[idx[good].long()])
    for r in (raw_q, raw_s):
        assert bool((r[:4096] == 0xA5).all()) and bool((r[-4096:] == 0xA5).all())


def tables_for(sizes):
    """Dispatch tables of groups of these sizes (top-1 routing)."""
    idx = torch.cat([torch.full((n,), e, dtype=torch.int32) for e, n in enumerate(sizes)]).cuda().view(-1, 1)
    return binding.moe_build_dispatch(idx, None, len(sizes))


def operands(rows, E, N, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows * 13 + N * 7 + K)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)  # noqa: E731
    return (u8(0, 256, rows, K // 2), u8(120, 132, rows, K // 32), u8(0, 256, E, N, K // 2), u8(118, 126, E, N, K // 32))


def product64(qa, sa, qb, sb, sizes):
    a, first, parts, mags = values64(qa, sa), 0, [], []
    for e, n in enumerate(sizes):
        w = values64(qb[e], sb[e])
        parts.append(a[first:first + n] @ w.t())
        mags.append(a[first:first + n].abs() @ w.abs().t())
        first += n
    return torch.cat(parts), torch.cat(mags)


def check(got, want, mag, dtype):
    limit = torch.finfo(DT[dtype]).max
    bound = ULP[dtype] * want.abs() + 2.0 ** -20 * mag + (2.0 ** -24 if dtype == "f16" else 0.0)
    g = got.double()
    bad = ~((g - want).abs() <= bound) & (want.abs() < 0.99 * limit)
    assert not bad.any(), (int(bad.sum()), float(((g - want).abs() / bound.clamp_min(1e-300)).max()))


GROUPS = [[1], [128], [129], [0, 1, 0, 127, 128, 129, 3, 300], [64, 65, 16, 17, 0, 0, 700], [2, 0, 5, 1, 1, 9, 0, 33, 8, 1]]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("N,K", [(1, 32), (128, 256), (333, 1056), (256, 64), (130, 512), (72, 288), (768, 2048), (17, 7168)])
def test_grouped_product(N, K, dtype):
    require_cuda()
    for i, sizes in enumerate(GROUPS):
        qa, sa, qb, sb = operands(sum(sizes), len(sizes), N, K, seed=i)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = binding.moe_grouped_gemm_mx4(qa, sa, qb, sb, tables_for(sizes), DT[dtype], err=err)
        want, mag = product64(qa, sa, qb, sb, sizes)
        assert int(err.item()) == 0
        check(got, want, mag, dtype)


def test_grouped_product_scales_at_their_ends():
    """Products of the largest and the smallest scales that fp32 holds, and a
    NaN scale that stays in its row and its column."""
    require_cuda()
    sizes, N, K = [40, 5], 48, 128
    qa, sa, qb, sb = operands(45, 2, N, K, seed=3)
    for a, b in ((250, 5), (3, 250), (100, 150), (127, 127)):
        sa.fill_(a)
        sb.fill_(b)
        want, mag = product64(qa, sa, qb, sb, sizes)
        check(binding.moe_grouped_gemm_mx4(qa, sa, qb, sb, tables_for(sizes), torch.float32), want, mag, "f32")
    sa[7, 2] = 255
    sb[1, 11, 0] = 255
    got = binding.moe_grouped_gemm_mx4(qa, sa, qb, sb, tables_for(sizes), torch.float32)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[7] = True
    nan[40:, 11] = True
    assert torch.equal(got.isnan(), nan)
    check(got[~nan], want[~nan], mag[~nan], "f32")


def test_grouped_product_stays_inside_repeats_and_streams():
    require_cuda()
    sizes, N, K = [3, 130, 0, 61], 201, 320
    rows = sum(sizes)
    ops = operands(rows, 4, N, K, seed=4)
    tab = tables_for(sizes)
    want, mag = product64(*ops, sizes)
    for dtype in ("f16", "f32"):
        n = rows * N * (2 if dtype == "f16" else 4)
        raw = torch.full((4096 + n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        out = raw[4096:4096 + n].view(DT[dtype]).view(rows, N)
        ref = binding.moe_grouped_gemm_mx4(*ops, tab, DT[dtype], out=out).clone()
        check(ref, want, mag, dtype)
        assert bool((raw[:4096] == 0xA5).all()) and bool((raw[4096 + n:] == 0xA5).all())
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                assert torch.equal(binding.moe_grouped_gemm_mx4(*ops, tab, DT[dtype]), ref)
        stream.synchronize()


@pytest.mark.parametrize("d_h,d_e,sizes", [(64, 32, [3]), (256, 128, [130, 0, 5]), (1056, 96, [1, 64, 65, 129]), (512, 320, [17, 200])])
def test_gate_up_silu(d_h, d_e, sizes):
    """The quantised h lies between the quantised ends of what fp32 sums allow:
    silu's slope is at most 1.1, a sum is off by 2^-20 of its magnitudes,
    the exponential, the division and the product by 2^-20 of h."""
    require_cuda()
    rows, E = sum(sizes), len(sizes)
    qa, sa, qg, sg = operands(rows, E, d_e, d_h, seed=1)
    _, _, qu, su = operands(rows, E, d_e, d_h, seed=2)
    e = binding.Mx4Experts(qg, sg, qu, su, torch.zeros((E, d_h, d_e // 2), dtype=torch.uint8, device="cuda"),
                           torch.zeros((E, d_h, d_e // 32), dtype=torch.uint8, device="cuda"))
    raw = torch.full((2 * 4096 + rows * d_e // 2,), 0xA5, dtype=torch.uint8, device="cuda")
    qh, sh = binding.moe_grouped_gate_up_silu_mx4(qa, sa, e, tables_for(sizes), q_h=raw[4096:-4096].view(rows, d_e // 2))
    assert bool((raw[:4096] == 0xA5).all()) and bool((raw[-4096:] == 0xA5).all())
    got = values64(qh, sh)
    g, mg = product64(qa, sa, qg, sg, sizes)
    u, mu = product64(qa, sa, qu, su, sizes)
    silu = g * torch.sigmoid(g)
    h = silu * u
    off = 2.0 ** -20 * (1.1 * mg * u.abs() + silu.abs() * mu + h.abs()) + 1e-30
    lo, el = quantize64(h - off)
    hi, eh = quantize64(h + off)
    steady = ((el == eh) & (sh.long() - 127 == el)).repeat_interleave(32, 1)
    assert float(steady.double().mean()) > 0.9
    inside = (got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))
    assert bool(inside[steady].all())


@pytest.mark.parametrize("T,d_h,d_e,E,k,dtype", [(1, 256, 64, 4, 2, "f16"), (64, 2048, 768, 64, 6, "f16"), (300, 512, 320, 9, 3, "bf16"),
                                                 (1030, 256, 128, 16, 4, "bf16")])
def test_forward(T, d_h, d_e, E, k, dtype):
    """The 4-bit forward is its parts, called one by one, to the last bit."""
    require_cuda()
    cfg = workloads.MoEConfig("mx4", 1, T, d_h, d_e, E, k, dtype, 5)
    d = workloads.make_moe_inputs(cfg, device="cuda")
    ex = binding.Mx4Experts.from_weights(d["w_gate"], d["w_up"], d["w_down"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.moe_forward_mx4(d["x"], d["wg"], None, ex, k, err=err)
    idx, w = binding.moe_gate_topk(d["x"], d["wg"], None, k)
    tab = binding.moe_build_dispatch(idx, w, E)
    qa, sa = binding.moe_quantize_mx4(d["x"], tab["sorted_token_idx"])
    qh, sh = binding.moe_grouped_gate_up_silu_mx4(qa, sa, ex, tab)
    y = binding.moe_grouped_gemm_mx4(qh, sh, ex.q_down, ex.sf_down, tab, d["x"].dtype)
    assert torch.equal(out, binding.moe_reduce_fused(y, tab["token_topk_to_pos"], w))
    assert int(err.item()) == 0
    # and near the 16-bit layer: 4-bit rows and weights are off by about a tenth each
    ref = binding.moe_forward(d["x"], d["wg"], None, d["w_gate"], d["w_up"], d["w_down"], k)
    assert float((out.float() - ref.float()).norm() / ref.float().norm()) < 0.4


def test_refusals():
    require_cuda()
    x = torch.randn((4, 64), device="cuda")
    q, sf = binding.moe_quantize_mx4(x)
    with pytest.raises(ValueError):
        binding.moe_quantize_mx4(torch.randn((4, 48), device="cuda"))
    with pytest.raises(ValueError):
        binding.moe_quantize_mx4(x, sf=sf[:2])
    with pytest.raises(TypeError):
        binding.moe_quantize_mx4(x.double())
    with pytest.raises(TypeError):
        binding.moe_quantize_mx4(x, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        binding.moe_dequantize_mx4(q, sf[:, :1])
    with pytest.raises(binding.MoEError, match="INVALID_ARG"):
        binding.moe_quantize_mx4(torch.randn(4 * 64 + 1, device="cuda")[1:].view(4, 64))
    tab = tables_for([4])
    qb, sb = q.view(1, 4, 32), sf.view(1, 4, 2)
    with pytest.raises(ValueError):
        binding.moe_grouped_gemm_mx4(q, sf, qb[:, :, :16].contiguous(), sb[:, :, :1].contiguous(), tab)
    with pytest.raises(binding.MoEError, match="INVALID_ARG"):
        binding.moe_grouped_gemm_mx4(q, sf, qb, sb, {**tab, "group_idx_for_bx": torch.zeros(9, dtype=torch.int32, device="cuda")})
    with pytest.raises(binding.MoEError, match="UNSUPPORTED"):
        binding.moe_grouped_gemm_mx4(q, sf, qb, sb, tab, torch.float8_e4m3fn)
    none = torch.empty((0, 64), device="cuda")
    assert binding.moe_quantize_mx4(none)[0].shape == (0, 32)
    ex = binding.Mx4Experts.from_weights(*(torch.randn(n, device="cuda") for n in ((2, 64, 256), (2, 64, 256), (2, 256, 64))))
    with pytest.raises(ValueError):
        binding.Mx4Experts(ex.q_gate, ex.sf_gate, ex.q_up, ex.sf_up, ex.q_gate, ex.sf_gate)
    with pytest.raises(ValueError):
        binding.moe_forward_mx4(x.half(), torch.zeros((2, 64), dtype=torch.float16, device="cuda"), None, ex, 1)
    rows = torch.zeros((3, 256), dtype=torch.float16, device="cuda")
    with pytest.raises(binding.MoEError, match="INVALID_ARG"):
        binding.moe_forward_mx4(rows, rows[:2].contiguous(), None, ex, 3)
    with pytest.raises(binding.MoEError, match="WORKSPACE"):
        binding.moe_forward_mx4(rows, rows[:2].contiguous(), None, ex, 1, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
