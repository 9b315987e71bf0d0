"""Tokens and experts whose logits are NaN or infinite: the gate names k
distinct experts for every token whatever the logits hold (NaN first, ties to
the lower id), so such a token's results are its own and no other's."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding, workloads

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
NAN, INF = float("nan"), float("inf")


# every form of the selection: one token and four tokens a CTA with all experts,
# a warp a token (few and many tokens, up to 1024 experts), candidates after the
# tensor cores' logits
SHAPES = [(5, 256, 8, 8), (9, 512, 64, 6), (1, 256, 1, 1), (33, 256, 40, 32), (700, 256, 64, 8), (11, 256, 72, 8), (6, 256, 1000, 32),
          (600, 256, 100, 12), (1024, 256, 64, 8), (1030, 512, 8, 2), (1024, 256, 300, 32)]


def gate(x, w_g, bias, k):
    idx = torch.full((x.shape[0], k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((x.shape[0], k), 7.0, device="cuda")
    binding.moe_gate_topk(x, w_g, bias, k, topk_idx=idx, topk_w=w)
    return idx, w


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,d_h,E,k", SHAPES)
def test_every_slot_names_an_expert(T, d_h, E, k, dtype):
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn((T, d_h), generator=g, device="cuda").to(DT[dtype])
    w_g = (torch.randn((E, d_h), generator=g, device="cuda") / d_h ** 0.5).to(DT[dtype])
    clean = gate(x, w_g, None, k)
    bad = sorted({0, T // 2, T - 1})
    for value in (NAN, INF, -INF):
        xb = x.clone()
        xb[bad, 17] = value
        idx, w = gate(xb, w_g, None, k)
        assert int(idx.min()) >= 0 and int(idx.max()) < E
        assert bool((idx.sort(1).values.diff(dim=1) > 0).all())
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[bad] = False
        assert torch.equal(idx[rest], clean[0][rest]) and torch.equal(w[rest], clean[1][rest])
        if value != value:  # all logits equal: the lowest ids
            assert torch.equal(idx[bad].long(), torch.arange(k, device="cuda").expand(len(bad), k))
            assert bool(w[bad].isnan().all())


@pytest.mark.parametrize("T,d_h,E,k", [s for s in SHAPES if s[2] > 5])
def test_experts_with_nan_logits_come_first(T, d_h, E, k):
    require_cuda()
    g = torch.Generator(device="cuda").manual_seed(T + 2 * E)
    x = torch.randn((T, d_h), generator=g, device="cuda").bfloat16()
    w_g = (torch.randn((E, d_h), generator=g, device="cuda") / d_h ** 0.5).bfloat16()
    order, _ = gate(x, w_g, None, min(k + 2, E, 32))
    bias = torch.zeros(E, device="cuda")
    bias[5], bias[3] = NAN, NAN
    idx, w = gate(x, w_g, bias, k)
    want = torch.empty_like(idx)
    for t in range(T):
        rest = [e for e in order[t].tolist() if e not in (3, 5)]
        want[t] = torch.tensor(([3, 5] + rest + [-1] * k)[:k])
    sure = want >= 0  # the order holds at most 32 experts
    assert torch.equal(idx[sure], want[sure])
    assert int(idx.min()) >= 0 and int(idx.max()) < E and bool((idx.sort(1).values.diff(dim=1) > 0).all())
    assert bool(w.isnan().all())


@pytest.mark.parametrize("T,d_h,d_e,E,k,dtype", [(40, 512, 128, 16, 4, "bf16"), (20, 256, 64, 72, 8, "f16"), (1024, 256, 64, 64, 8, "bf16")])
def test_a_bad_token_stays_alone_in_the_forwards(T, d_h, d_e, E, k, dtype):
    """On workspaces that hold other bytes: no slot of a table is left as it was."""
    require_cuda()
    d = workloads.make_moe_inputs(workloads.MoEConfig("nan", 1, T, d_h, d_e, E, k, dtype, 5), device="cuda")
    x, wg, w = d["x"], d["wg"], (d["w_gate"], d["w_up"], d["w_down"])
    experts = binding.Mx4Experts.from_weights(*w)
    code = DT[dtype]
    forwards = [(lambda v, ws, err: binding.moe_forward_mx4(v, wg, None, experts, k, ws=ws, err=err),
                 binding.forward_mx4_workspace_bytes(T, d_h, d_e, E, k, code)),
                (lambda v, ws, err: binding.moe_forward(v, wg, None, *w, k, ws=ws, err=err),
                 binding.forward_workspace_bytes(T, d_h, d_e, E, k, code))]
    bad = [1, 7, T - 1]
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[bad] = False
    xb = x.clone()
    xb[1, 5], xb[7, 100], xb[T - 1, 3] = NAN, INF, -INF
    for forward, n in forwards:
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ref = forward(x, torch.zeros(n, dtype=torch.uint8, device="cuda"), err).clone()
        for fill in (0xFF, 0x7F, 0x00, 0x01):
            ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
            got = forward(xb, ws, err)
            torch.cuda.synchronize()
            assert int(err.item()) == 0
            assert torch.equal(got[rest], ref[rest])
            assert not bool(got[1].isfinite().any())
