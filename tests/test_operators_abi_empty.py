"""Host side of the norms' gradients: with no rows, whose tensors may all be null,
nothing is launched and the process lives; the workspace is what the grid can
use."""
import subprocess
import sys

import pytest

from mixture_experts_routed_gate_gb300 import _build

CALL = """
from mixture_experts_routed_gate_gb300 import binding
lib, A = binding.lib(), 0x1000  # an address that is never read
w_post, gate, kind, w_next = {args}
print(lib.moe_residual_norm_backward(None, None, None, None, w_post, gate, kind, 1.0, w_next, None, None, 0, 64, {dtype},
                                     None, None, None, None, None, A, 1 << 20, None))
"""


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("args", ["A, None, 0, None", "None, None, 2, None", "None, A, 1, None", "None, None, 3, None", "None, None, 0, A",
                                  "A, A, 1, A"])
def test_gradients_of_no_rows(args, dtype):
    _build.build()
    r = subprocess.run([sys.executable, "-c", CALL.format(args=args, dtype=dtype)], cwd=_build.ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split()[-1] == "0", (r.returncode, r.stdout, r.stderr[-500:])


@pytest.mark.parametrize("T,H,ctas_per_sm", [(4096, 7168, 1), (4096, 16384, 1), (100000, 2048, 3), (100000, 64, 16), (100000, 1, 16), (3, 7168, 1)])
def test_workspace_of_the_gradients(T, H, ctas_per_sm):
    """Three fp32 rows of column sums a CTA: 896 threads an SM, 8 elements each,
    or one CTA, on a GPU of at most 160 SMs."""
    _build.build()
    from mixture_experts_routed_gate_gb300 import binding
    n = binding.lib().moe_residual_norm_backward_workspace_bytes(T, H)
    row = 3 * H * 4
    assert min(T, ctas_per_sm) * row <= n <= min(T, 160 * ctas_per_sm) * row + 16
