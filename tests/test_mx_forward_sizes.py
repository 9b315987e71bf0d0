"""The 8-bit and the 4-bit forward refuse sizes that one of their parts would refuse, before any part is launched."""
import ctypes

import pytest

from mixture_experts_routed_gate_gb300 import _build, binding

UNSUPPORTED, WORKSPACE = 2, 3
F16 = 0
NONE = ctypes.c_size_t(-1).value
A = 0x1000  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.lib()


def forward(lib, bits, T=4, d_h=256, d_e=64, E=8, k=2, n=1 << 62):
    if bits == 8:
        return lib.moe_forward_mx8(A, None, None, A, None, A, A, A, A, A, A, T, d_h, d_e, E, k, F16, 0x100000, n, A, None, None)
    return lib.moe_forward_mx4(A, A, None, A, A, A, A, A, A, T, d_h, d_e, E, k, F16, 0x100000, n, A, None, None)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("change", [dict(T=1 << 31), dict(T=1 << 40), dict(T=1 << 62, k=8), dict(T=1 << 28, k=8), dict(T=(1 << 31) - 255, k=1),
                                    dict(d_h=(1 << 20) + 256), dict(d_e=(1 << 20) + 64)])
def test_sizes_that_a_part_refuses(lib, bits, change):
    assert forward(lib, bits, **change) == UNSUPPORTED
    sizes = dict(dict(T=4, d_h=256, d_e=64, E=8, k=2), **change)
    assert getattr(lib, f"moe_forward_mx{bits}_workspace_bytes")(*sizes.values(), F16) == NONE


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("change", [dict(T=(1 << 31) - 256, k=1), dict(d_h=1 << 20), dict(d_e=1 << 20)])
def test_the_largest_sizes_are_taken(lib, bits, change):
    sizes = dict(dict(T=4, d_h=256, d_e=64, E=8, k=2), **change)
    need = getattr(lib, f"moe_forward_mx{bits}_workspace_bytes")(*sizes.values(), F16)
    assert sizes["T"] * sizes["k"] * sizes["d_h"] * 2 < need < 1 << 62
    assert forward(lib, bits, **change, n=need - 1) == WORKSPACE
