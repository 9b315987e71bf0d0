"""The combine's gradient against its formula in 64 bits, against differences, and
at the positions where it can go wrong.

d_x is one product, rounded once: fp32's w * d_out, then the type.  d_topk_w is an
fp32 sum; an element takes part in at most 64 additions (its thread's, its warp's, the
warps'), so it is within 64 * 2^-24 of the sum of the terms' magnitudes."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
PAIRS = [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "f16"), ("f32", "bf16")]


def routed(T, K, E, seed, device="cuda"):
    """Positions [T, K] and the rows' tokens, as the dispatch gives them."""
    g = torch.Generator(device=device).manual_seed(seed)
    idx = torch.rand((T, E), generator=g, device=device).topk(K, dim=1).indices.to(torch.int32)
    t = binding.moe_build_dispatch(idx.contiguous(), None, E)
    return t["token_topk_to_pos"], t["sorted_token_idx"]


def formula(d_out, x, pos, w, token):
    """Both gradients in 64 bits, pair by pair, and the sum of the magnitudes of d_topk_w's terms."""
    n, (T, K) = x.shape[0], pos.shape
    d_x = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    d_w = torch.zeros((T, K), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(d_w)
    f = torch.zeros(n, dtype=torch.float64, device=x.device)
    for j in range(K):
        p = pos[:, j].long()
        here = (p >= 0) & (p < n)
        t = torch.nonzero(here)[:, 0]
        terms = x[p[t]].double() * d_out[t].double()
        d_w[t, j], mag[t, j] = terms.sum(1), terms.abs().sum(1)
        t = t[token[p[t]].long() == t]
        f.index_put_((p[t],), torch.ones(len(t), dtype=torch.float64, device=x.device) if w is None else w[t, j].double(), accumulate=True)
    owner = token.long()
    ok = (owner >= 0) & (owner < T)
    d_x[ok] = f[ok, None] * d_out[owner[ok]].double()
    d_x[f == 0] = 0.0
    return d_x, d_w, mag


def check(got, want, dtype):
    d_x, d_w = got
    w_x, w_w, mag = want
    assert ((d_w.double() - w_w).abs() <= 64 * 2.0 ** -24 * mag).all()
    # a sum of weights and the product: two roundings of fp32 each at most, then one of the type (its least normal number's half step below that)
    step = torch.finfo(dtype).eps / 2
    assert ((d_x.double() - w_x).abs() <= (step + 2.0 ** -22) * w_x.abs() + torch.finfo(dtype).smallest_normal * step).all()


@pytest.mark.parametrize("types", PAIRS)
@pytest.mark.parametrize("T,K,E,H", [(1, 1, 1, 256), (1, 8, 8, 256), (3, 2, 5, 512), (64, 6, 64, 2048), (333, 5, 40, 2304), (130, 32, 40, 256),
                                     (37, 3, 9, 7168), (500, 1, 3, 1024), (5, 4, 16, 16640)])
def test_against_the_formula(T, K, E, H, types):
    require_cuda()
    tx, td = (DT[t] for t in types)
    pos, token = routed(T, K, E, T * 31 + K)
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn((T * K, H), generator=g, device="cuda").to(tx)
    d_out = torch.randn((T, H), generator=g, device="cuda").to(td)
    w = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for weights in (w, None):
        got = binding.moe_reduce_fused_backward(d_out, x, pos, weights, token, err=err)
        check(got, formula(d_out, x, pos, weights, token), tx)
        t = token.long()
        at = torch.zeros(T * K, device="cuda")
        at[pos.long().view(-1)] = torch.ones(T * K, device="cuda") if weights is None else weights.view(-1)
        assert torch.equal(got[0], (at[:, None] * d_out[t].float()).to(tx))
    assert int(err.item()) == 0


def test_dropped_pairs_and_rows_of_nobody():
    require_cuda()
    T, K, H, extra = 70, 4, 512, 13
    pos, token = routed(T, K, 12, 5)
    token = torch.cat((token, torch.tensor([-1, T, 2 ** 31 - 1, 0, 5, 69, -2 ** 31, 3, 3, 3, 3, 3, 3], dtype=torch.int32, device="cuda")))
    pos = pos.clone()
    pos[::3, 1] = -1
    pos[7] = -1  # a token without any row
    x = torch.randn((T * K + extra, H), device="cuda").bfloat16()
    gone = torch.ones(T * K + extra, dtype=torch.bool, device="cuda")
    gone[pos[pos >= 0].long()] = False
    x[gone] = float("nan")  # rows that no position names are not read
    d_out = torch.randn((T, H), device="cuda").bfloat16()
    d_out[7] = float("inf")  # nor is this token's gradient put anywhere
    w = torch.rand((T, K), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d_x, d_w = binding.moe_reduce_fused_backward(d_out, x, pos, w, token, err=err)
    assert (d_x[gone] == 0).all() and (d_w[pos < 0] == 0).all() and int(err.item()) == 0
    clean, d = torch.nan_to_num(x), torch.nan_to_num(d_out, posinf=0.0)
    check((d_x, d_w), formula(d, clean, pos, w, token), torch.bfloat16)


def test_positions_that_are_wrong():
    """Out of range: as -1.  The same row twice in one token: both weights' gradients, the row's factor their
    sum.  Another token's row: read, and given nothing.  Each but the second is told."""
    require_cuda()
    T, K, H = 9, 3, 256
    pos, token = routed(T, K, 6, 8)
    x, d_out, w = torch.randn((T * K, H), device="cuda"), torch.randn((T, H), device="cuda"), torch.rand((T, K), device="cuda")
    for change, flag in (((0, 1, T * K), 5), ((2, 0, -2), 5), ((3, 2, 2 ** 31 - 1), 5), ((4, 1, int(pos[4, 0])), 0), ((5, 2, int(pos[1, 1])), 5)):
        p = pos.clone()
        p[change[0], change[1]] = change[2]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = binding.moe_reduce_fused_backward(d_out, x, p, w, token, err=err)
        check(got, formula(d_out, x, p, w, token), torch.float32)
        again = binding.moe_reduce_fused_backward(d_out, x, p, w, token)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        assert int(err.item()) == flag, change


def test_no_tokens_and_no_rows():
    require_cuda()
    token = torch.zeros(5, dtype=torch.int32, device="cuda")
    x = torch.randn((5, 256), device="cuda")
    d_x, d_w = binding.moe_reduce_fused_backward(torch.empty((0, 256), device="cuda"), x, torch.empty((0, 2), dtype=torch.int32, device="cuda"), None, token)
    assert (d_x == 0).all() and d_w.shape == (0, 2)
    pos = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    d_x, d_w = binding.moe_reduce_fused_backward(torch.randn((3, 256), device="cuda"), x[:0], pos, None, token[:0])
    assert d_x.shape == (0, 256) and (d_w == 0).all()


def test_without_the_weights_gradient():
    """d_topk_w NULL: x is not needed."""
    require_cuda()
    T, K, H = 20, 3, 512
    pos, token = routed(T, K, 7, 1)
    d_out, w = torch.randn((T, H), device="cuda").half(), torch.rand((T, K), device="cuda")
    d_x = torch.empty((T * K, H), dtype=torch.float16, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    st = binding.lib().moe_reduce_fused_backward(p(d_out), None, T * K, p(pos), p(w), p(token), T, K, H, 0, 0, p(d_x), None, None,
                                                 torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(d_x, binding.moe_reduce_fused_backward(d_out, torch.zeros_like(d_x), pos, w, token)[0])


def test_chain_against_differences():
    """loss = <v, combine(gather(x) * c, w)>: the rows' way there and back, with their gradients, against
    differences of the loss.  It is linear in x and in w, so a central difference is exact but for the
    rounding of the loss: its terms are summed in 64 bits, each output element off by at most 9 roundings of fp32."""
    require_cuda()
    T, K, E, H = 40, 4, 10, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    pos, token = routed(T, K, E, 11)
    x, c, v, w = n(T, H), n(T * K, H), n(T, H), torch.softmax(n(T, K), 1)

    def out(x, w):
        rows = binding.moe_gather_rows_by_token(x, pos, T * K)
        return binding.moe_reduce_fused(rows * c, pos, w)
    rows = binding.moe_gather_rows_by_token(x, pos, T * K)
    d_rows, d_w = binding.moe_reduce_fused_backward(v, rows * c, pos, w, token)
    d_x = binding.moe_reduce_fused(d_rows * c, pos)
    for which, grad in ((0, d_x), (1, d_w)):
        dirn = n(*grad.shape)
        hi, lo = (out(x + s * dirn, w) if which == 0 else out(x, w + s * dirn) for s in (0.5, -0.5))
        got = (v.double() * (hi.double() - lo.double())).sum()
        want = (grad.double() * dirn.double()).sum()
        most = (x.abs() + (0.5 * dirn.abs() if which == 0 else 0)).max() * c.abs().max() * (w.abs() + (0.5 * dirn.abs() if which else 0)).max()
        assert abs(got - want) <= 9 * 2.0 ** -24 * 2 * K * float(most) * float(v.double().abs().sum())


def test_on_a_stream_and_in_a_graph():
    require_cuda()
    T, K, H = 150, 4, 1024
    pos, token = routed(T, K, 9, 2)
    x, d_out, w = torch.randn((T * K, H), device="cuda").half(), torch.randn((T, H), device="cuda").half(), torch.rand((T, K), device="cuda")
    want = binding.moe_reduce_fused_backward(d_out, x, pos, w, token)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = binding.moe_reduce_fused_backward(d_out, x, pos, w, token)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = binding.moe_reduce_fused_backward(d_out, x, pos, w, token)
    d_out.copy_(torch.randn((T, H), device="cuda"))
    graph.replay()
    want = binding.moe_reduce_fused_backward(d_out, x, pos, w, token)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_more_than_2_31_elements():
    require_cuda()
    T, K, H = 38000, 8, 7168  # 2.18e9 elements of x
    pos, token = routed(T, K, 64, 4)
    x = torch.empty((T * K, H), dtype=torch.bfloat16, device="cuda").normal_()
    d_out, w = torch.randn((T, H), device="cuda").bfloat16(), torch.rand((T, K), device="cuda")
    d_x, d_w = binding.moe_reduce_fused_backward(d_out, x, pos, w, token)
    for t in (0, 1, T // 2, T - 1):
        r = pos[t].long()
        assert torch.equal(d_x[r], (w[t][:, None] * d_out[t].float()).bfloat16())
        terms = x[r].double() * d_out[t].double()
        assert ((d_w[t].double() - terms.sum(1)).abs() <= 64 * 2.0 ** -24 * terms.abs().sum(1)).all()


def test_refusals():
    require_cuda()
    T, K, H = 4, 2, 256
    pos, token = routed(T, K, 4, 0)
    x, d, w = torch.randn((8, H), device="cuda"), torch.randn((T, H), device="cuda"), torch.rand((T, K), device="cuda")
    f = binding.moe_reduce_fused_backward
    for args in ((d, x.t(), pos, w, token), (d[:3], x, pos, w, token), (d, x, pos, w[:, :1], token), (d, x, pos, w, token[:7]),
                 (d, x, pos.t(), w, token), (d, torch.randn((16, H), device="cuda")[::2], pos, w, token)):
        with pytest.raises(ValueError):
            f(*args)
    for args in ((d, x, pos.long(), w, token), (d, x, pos, w.double(), token), (d, x, pos, w, token.long()), (d, x.double(), pos, w, token)):
        with pytest.raises(TypeError):
            f(*args)
    with pytest.raises(binding.MoEError):
        f(d, x.half(), pos, w, token)  # 16-bit rows with an fp32 output are not the combine's
    with pytest.raises(binding.MoEError):
        f(d[:, :128].contiguous(), x[:, :128].contiguous(), pos, w, token)
