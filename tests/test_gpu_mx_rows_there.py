"""Tables of a larger batch than the call's rows: the grouped products of 8-bit and 4-bit
rows neither read nor write a row past their own, and say so.  All rows that the tables name
lie in the test's own tensors, the call's rows being the first part of them."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
DEVICE_FLAG = 5


class Eight:
    quantize, experts = staticmethod(binding.moe_quantize_mx8), binding.Mx8Experts
    product, gate_up = staticmethod(binding.moe_grouped_gemm_mx8), staticmethod(binding.moe_grouped_gate_up_silu_mx8)
    per, dtype = 1, E4M3


class Four:
    quantize, experts = staticmethod(binding.moe_quantize_mx4), binding.Mx4Experts
    product, gate_up = staticmethod(binding.moe_grouped_gemm_mx4), staticmethod(binding.moe_grouped_gate_up_silu_mx4)
    per, dtype = 2, torch.uint8


# few units of rows; more than a CTA lists; tiles of up to 256 rows; those, more than a CTA lists
SHAPES = [(60, 3, 5, 256, 96), (1100, 2, 900, 96, 64), (5000, 2, 7, 288, 4128), (3000, 2, 7, 4128, 704), (60000, 1, 600, 4096, 32)]


@pytest.mark.parametrize("there", [0.0, 0.4, 0.97])
@pytest.mark.parametrize("T,k,E,K,N", SHAPES)
@pytest.mark.parametrize("form", [Eight, Four])
def test_tables_of_a_larger_batch(form, T, k, E, K, N, there):
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(T + K)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32).contiguous()
    t = binding.moe_build_dispatch(idx, None, E)
    rows, n = T * k, max(1, int(T * k * there))
    t["group_idx_for_bx"] = t["group_idx_for_bx"][:-(-n // 128) + E].contiguous()  # as many blocks as so many rows can have
    qa, sa = form.quantize(torch.randn((rows, K), generator=g, device="cuda"))
    w = [form.quantize(torch.randn((E * a, b), generator=g, device="cuda") * b ** -0.5) for a, b in ((N, K), (N, K), (K, N))]
    e = form.experts(*(x.view(E, a, -1) for (q, s), a in zip(w, (N, N, K)) for x in (q, s)))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # the same call with all rows, and the tables' sizes cut to those that there are
    ends = t["group_offsets"].long() + t["group_sizes"].long()
    cut = dict(t, group_sizes=(ends.clamp(max=n) - t["group_offsets"].long()).clamp(min=0).to(torch.int32))
    out = torch.full((rows, N), 7.0, device="cuda")
    form.product(qa, sa, e.q_gate, e.sf_gate, cut, torch.float32, out=out, err=err)
    q, s = torch.full((rows, N // form.per), 3, dtype=torch.uint8, device="cuda"), torch.full((rows, N // 32), 3, dtype=torch.uint8, device="cuda")
    form.gate_up(qa, sa, e, cut, q.view(form.dtype), s, err=err)
    assert int(err.item()) == 0 and (out[n:] == 7).all() and (s[n:] == 3).all() and not (out[:n] == 7).all()
    # the first n rows alone
    got = torch.full((rows, N), 7.0, device="cuda")
    form.product(qa[:n], sa[:n], e.q_gate, e.sf_gate, t, torch.float32, out=got[:n], err=err)
    assert int(err.item()) == DEVICE_FLAG and torch.equal(got, out)
    err.zero_()
    gq, gs = torch.full_like(q, 3), torch.full_like(s, 3)
    form.gate_up(qa[:n], sa[:n], e, t, gq.view(form.dtype)[:n], gs[:n], err=err)
    assert int(err.item()) == DEVICE_FLAG and torch.equal(gq, q) and torch.equal(gs, s)
    form.product(qa[:n], sa[:n], e.q_gate, e.sf_gate, t, torch.float32, out=got[:n])  # no word to say it in
    assert torch.equal(got, out)


@pytest.mark.parametrize("form", [Eight, Four])
def test_tables_that_name_no_row(form):
    """First rows below 0 and experts that there are not: nothing is read or written for them."""
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(0)
    E, K, N, n = 3, 64, 64, 40
    a, b = form.quantize(torch.randn((n, K), generator=g, device="cuda")), form.quantize(torch.randn((E * N, K), generator=g, device="cuda"))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dict(group_sizes=i32(20, 10, 30), group_offsets=i32(0, -10, 20), group_padded_offsets=i32(0, 128, 256), group_idx_for_bx=i32(0, 1, 2, 77))
    ok = dict(t, group_sizes=i32(20, 0, 20), group_idx_for_bx=i32(0, 1, 2, 2))
    err, out = torch.zeros(1, dtype=torch.int32, device="cuda"), []
    for tables in (ok, t):
        out.append(torch.full((n, N), float("nan"), device="cuda"))
        form.product(*a, *(x.view(E, N, -1) for x in b), tables, torch.float32, out=out[-1], err=err)
        assert int(err.item()) == (0 if tables is ok else DEVICE_FLAG)
    assert torch.equal(*out)  # every row is written: a NaN is not equal to itself


@pytest.mark.parametrize("form", [Eight, Four])
def test_as_many_rows_as_there_may_be(form):
    """2^31 - 256 rows of 32 elements, and blocks up to row 2^31: the products of the first rows and the last."""
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    E, K, N, n, last, some = 3, 32, 1, 2 ** 31 - 256, 1000, 700
    sizes = torch.tensor([n - last, 0, last])
    padded = torch.tensor([0, 0, 0])
    for i in (1, 2):
        padded[i] = padded[i - 1] + (sizes[i - 1] + 128) // 128 * 128
    blocks = -(-n // 128) + E
    assert blocks * 128 > 2 ** 31 and int(padded[2]) + last < 2 ** 31
    t = dict(group_sizes=sizes, group_offsets=torch.tensor([0, n - last, n - last]), group_padded_offsets=padded)
    t = {name: v.to(torch.int32).cuda() for name, v in t.items()}
    gidx = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    gidx[int(padded[1]) // 128:] = 1
    gidx[int(padded[2]) // 128:] = 2
    t["group_idx_for_bx"] = gidx
    qa, sa = torch.zeros((n, K // form.per), dtype=torch.uint8, device="cuda"), torch.full((n, 1), 127, dtype=torch.uint8, device="cuda")
    ends = [slice(0, some), slice(n - last - some, n - last), slice(n - last, n)]
    parts = [form.quantize(torch.randn((at.stop - at.start, K), generator=g, device="cuda")) for at in ends]
    for at, (q, s) in zip(ends, parts):
        qa[at], sa[at] = q.view(torch.uint8), s
    qb, sb = form.quantize(torch.randn((E * N, K), generator=g, device="cuda"))
    qb, sb = qb.view(E, N, -1), sb.view(E, N, -1)
    out, err = torch.full((n, N), 7.0, dtype=torch.float16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    form.product(qa.view(form.dtype), sa, qb, sb, t, torch.float16, out=out, err=err)
    assert int(err.item()) == 0
    for at, e, (q, s) in zip(ends, (0, 0, 2), parts):
        r = at.stop - at.start
        one = dict(group_sizes=[r], group_offsets=[0], group_padded_offsets=[0], group_idx_for_bx=[0] * (r // 128 + 1))
        one = {name: torch.tensor(v, dtype=torch.int32, device="cuda") for name, v in one.items()}
        assert torch.equal(out[at], form.product(q, s, qb[e:e + 1], sb[e:e + 1], one, torch.float16)), (at, e)
    assert not (out[some:some + 2 ** 20]).any() and not out[-last - some - 2 ** 20:-last - some].any()


@pytest.mark.parametrize("form", [Eight, Four])
def test_more_units_than_a_list_holds_and_experts_without_rows(form):
    """First rows below 0 and past the end among more units of rows than a CTA lists."""
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    E, K, N, n = 700, 64, 32, 700 * 2
    a, b = form.quantize(torch.randn((n, K), generator=g, device="cuda")), form.quantize(torch.randn((E * N, K), generator=g, device="cuda"))
    sizes, offsets = torch.full((E,), 2), torch.arange(E) * 2
    t = dict(group_sizes=sizes, group_offsets=offsets, group_padded_offsets=torch.arange(E) * 128, group_idx_for_bx=torch.arange(E))
    gone = torch.tensor([0, 5, 350, 698])
    ok = dict(t, group_sizes=sizes.index_fill(0, gone, 0))
    bad = dict(t, group_offsets=offsets.index_copy(0, gone, torch.tensor([-2, -(2 ** 31), n, 2 ** 31 - 1])))
    err, out = torch.zeros(1, dtype=torch.int32, device="cuda"), []
    for tables in (ok, bad):
        out.append(torch.full((n, N), -1000.5, device="cuda"))
        form.product(*a, *(x.view(E, N, -1) for x in b), {i: v.to(torch.int32).cuda() for i, v in tables.items()}, torch.float32, out=out[-1], err=err)
        assert int(err.item()) == (0 if tables is ok else DEVICE_FLAG)
    left = torch.zeros(n, dtype=torch.bool, device="cuda")
    left.view(E, 2)[gone.cuda()] = True
    assert torch.equal(*out) and (out[0][left] == -1000.5).all() and not (out[0][~left] == -1000.5).any()


def test_tables_of_fewer_experts_than_the_weights():
    """4-bit rows whose tables have no entry for the last experts, which no block names: what lies behind the
    tables (here entries that would name rows past the call's) is not looked at."""
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(4)
    E, more, K, N, n = 3, 40, 64, 64, 40
    a, b = Four.quantize(torch.randn((n, K), generator=g, device="cuda")), Four.quantize(torch.randn(((E + more) * N, K), generator=g, device="cuda"))
    b = [x.view(E + more, N, -1) for x in b]
    behind = [2 ** 30] * more
    t = dict(group_sizes=[20, 0, 20], group_offsets=[0, 20, 20], group_padded_offsets=[0, 128, 256], group_idx_for_bx=[0, 1, 2, 2])
    t = {name: torch.tensor(v + behind, dtype=torch.int32, device="cuda")[:len(v)] for name, v in t.items()}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = Four.product(*a, *b, t, torch.float32, err=err)
    assert int(err.item()) == 0
    assert torch.equal(got, Four.product(*a, *(x[:E].contiguous() for x in b), t, torch.float32))
