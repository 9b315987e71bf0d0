"""Every tensor of a call lies on one device: a call that mixes devices is refused before the library
sees an address.  The tensors are stand-ins that say they are on a GPU; no call reaches the library."""
import pytest
import torch

from mixture_experts_routed_gate_gb300 import _build, binding

E4M3, U8, I32, F32, BF16 = torch.float8_e4m3fn, torch.uint8, torch.int32, torch.float32, torch.bfloat16
HERE, THERE = torch.device("cuda:0"), torch.device("cuda:1")
T, H, D, E, K = 4, 256, 64, 3, 2
R = T * K


class On(torch.Tensor):
    """A tensor of the host that says it is on a GPU."""

    @staticmethod
    def __new__(cls, shape, dtype, device):
        t = torch.Tensor._make_subclass(cls, torch.zeros(shape, dtype=dtype))
        t.on = torch.device(device)
        return t

    is_cuda = property(lambda self: True)
    device = property(lambda self: self.on)


# every argument that is a tensor: shape and type
ROWS = dict(y=((T, H), BF16), res=((T, H), BF16), w_post=((H,), BF16), gate=((H,), BF16), w_next=((H,), BF16), out=((T, H), BF16))
TABLES = dict(group_sizes=((E,), I32), group_offsets=((E,), I32), group_padded_offsets=((E,), I32), group_idx_for_bx=((4,), I32))
ERR = dict(err=((1,), I32))


def experts(per, dtype):
    parts = dict(q_gate=((E, D, H // per), dtype), sf_gate=((E, D, H // 32), U8), q_up=((E, D, H // per), dtype), sf_up=((E, D, H // 32), U8),
                 q_down=((E, H, D // per), dtype), sf_down=((E, H, D // 32), U8))
    return parts, list(parts)


def split(a, names):
    return {n: a.pop(n) for n in names}


def with_tables(f):
    return lambda **a: f(tables=split(a, TABLES), **a)


def with_experts(cls, names, f):
    return lambda **a: f(experts=cls(**split(a, names)), **a)


def forward(f):
    def call(q=None, sf=None, **a):
        return f(k=K, **({} if q is None else {"rows": (q, sf)}), **a)
    return call


LAYER = dict(x=((T, H), BF16), w_g=((E, H), BF16), bias=((E,), F32), ws=((1 << 20,), U8), out=((T, H), BF16), **ERR)
E8, N8 = experts(1, E4M3)
E4, N4 = experts(2, U8)
CALLS = {
    "residual_norm": (binding.moe_residual_norm, dict(ROWS, u=((T, H), BF16))),
    "residual_norm_mx8": (binding.moe_residual_norm_mx8, dict(ROWS, q=((T, H), E4M3), sf=((T, H // 32), U8))),
    "residual_norm_mx8 of res": (binding.moe_residual_norm_mx8, dict(y=None, res=((T, H), BF16), w_next=((H,), BF16))),
    "residual_norm_backward": (binding.moe_residual_norm_backward, dict(
        {n: v for n, v in ROWS.items() if n != "res"}, d_out=((T, H), BF16), d_u=((T, H), BF16), rstd_post=((T,), F32), rstd_next=((T,), F32),
        ws=((1 << 20,), U8))),
    "reduce_fused_backward": (binding.moe_reduce_fused_backward, dict(
        d_out=((T, H), BF16), x=((R, H), BF16), token_topk_to_pos=((T, K), I32), topk_weights=((T, K), F32), sorted_token_idx=((R,), I32), **ERR)),
    "quantize_mx8": (binding.moe_quantize_mx8, dict(x=((T, H), BF16), q=((T, H), E4M3), sf=((T, H // 32), U8))),
    "dequantize_mx8": (binding.moe_dequantize_mx8, dict(q=((T, H), E4M3), sf=((T, H // 32), U8), out=((T, H), BF16))),
    "sort_rows_mx8": (binding.moe_sort_rows_mx8, dict(
        q=((T, H), E4M3), sf=((T, H // 32), U8), token_topk_to_pos=((T, K), I32), q_out=((R, H), E4M3), sf_out=((R, H // 32), U8))),
    "grouped_gemm_mx8": (with_tables(binding.moe_grouped_gemm_mx8), dict(
        TABLES, q_a=((R, H), E4M3), sf_a=((R, H // 32), U8), q_b=((E, D, H), E4M3), sf_b=((E, D, H // 32), U8), out=((R, D), BF16), **ERR)),
    "grouped_gate_up_silu_mx8": (with_experts(binding.Mx8Experts, N8, with_tables(binding.moe_grouped_gate_up_silu_mx8)), dict(
        TABLES, **E8, q_a=((R, H), E4M3), sf_a=((R, H // 32), U8), q_h=((R, D), E4M3), sf_h=((R, D // 32), U8), **ERR)),
    "forward_mx8": (with_experts(binding.Mx8Experts, N8, forward(binding.moe_forward_mx8)),
                    dict(LAYER, **E8, q=((T, H), E4M3), sf=((T, H // 32), U8))),
    "quantize_mx4": (binding.moe_quantize_mx4, dict(x=((T, H), BF16), row_idx=((R,), I32), q=((R, H // 2), U8), sf=((R, H // 32), U8), **ERR)),
    "dequantize_mx4": (binding.moe_dequantize_mx4, dict(q=((T, H // 2), U8), sf=((T, H // 32), U8), out=((T, H), BF16))),
    "grouped_gemm_mx4": (with_tables(binding.moe_grouped_gemm_mx4), dict(
        TABLES, q_a=((R, H // 2), U8), sf_a=((R, H // 32), U8), q_b=((E, D, H // 2), U8), sf_b=((E, D, H // 32), U8), out=((R, D), BF16), **ERR)),
    "grouped_gate_up_silu_mx4": (with_experts(binding.Mx4Experts, N4, with_tables(binding.moe_grouped_gate_up_silu_mx4)), dict(
        TABLES, **E4, q_a=((R, H // 2), U8), sf_a=((R, H // 32), U8), q_h=((R, D // 2), U8), sf_h=((R, D // 32), U8), **ERR)),
    "forward_mx4": (with_experts(binding.Mx4Experts, N4, forward(binding.moe_forward_mx4)), dict(LAYER, **E4)),
    "forward_few": (lambda **a: binding.moe_forward_few(k=K, **a), dict(
        LAYER, w_gate=((E, D, H), BF16), w_up=((E, D, H), BF16), w_down=((E, H, D), BF16))),
}


@pytest.fixture(scope="module")
def built():
    _build.build()
    return binding.lib()


@pytest.fixture
def reached(built, monkeypatch):
    calls = []
    monkeypatch.setattr(binding, "_call", lambda what, dev, *args: calls.append((what, dev)))
    monkeypatch.setattr(binding, "_host", None)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=F32, device=None: On(shape, dtype, device))
    return calls


def made(form, device, other=None):
    return {n: None if v is None else On(*v, THERE if n == other else device) for n, v in form.items()}


@pytest.mark.parametrize("name", CALLS)
def test_one_device(reached, name):
    call, form = CALLS[name]
    for device in (HERE, THERE):
        call(**made(form, device))
        assert reached.pop() == ("moe_" + name.split()[0], device) and not reached
    tensors = [n for n, v in form.items() if v is not None]
    for other in tensors if len(tensors) > 1 else ():
        with pytest.raises(ValueError, match="must be on cuda:"):
            call(**made(form, HERE, other))
        assert not reached, other


@pytest.mark.parametrize("cls,names,parts", [(binding.Mx8Experts, N8, E8), (binding.Mx4Experts, N4, E4)])
def test_experts_of_another_device(reached, cls, names, parts):
    """Experts that are whole, on a device that is not the rows'."""
    e = cls(**made(parts, THERE))
    eight = cls is binding.Mx8Experts
    form = CALLS["grouped_gate_up_silu_mx8" if eight else "grouped_gate_up_silu_mx4"][1]
    a = made({n: v for n, v in form.items() if n not in names}, HERE)
    gate_up, layer = (binding.moe_grouped_gate_up_silu_mx8, binding.moe_forward_mx8) if eight else (
        binding.moe_grouped_gate_up_silu_mx4, binding.moe_forward_mx4)
    with pytest.raises(ValueError, match="the experts must be on cuda:0"):
        with_tables(gate_up)(experts=e, **a)
    with pytest.raises(ValueError, match="the experts must be on cuda:0"):
        layer(experts=e, k=K, **made(LAYER, HERE))
    assert not reached
