"""The extension of the short calls: what is unusual is left to the Python code."""
import pytest
import torch

from gpu_helpers import require_cuda
from mixture_experts_routed_gate_gb300 import binding

pytestmark = pytest.mark.gpu


def test_a_flag_without_a_truth_value(monkeypatch):
    """with_u of two elements: the same error with the extension and without it, and no call."""
    require_cuda()
    binding.lib()
    host, told = binding._host, []
    assert host is not None
    x, out = torch.randn((2, 3, 64), device="cuda").unbind(0)
    before = out.clone()
    w = torch.ones(64, device="cuda")
    for h in (None, host):
        monkeypatch.setattr(binding, "_host", h)
        with pytest.raises(Exception) as caught:
            binding.moe_residual_norm_mx8(x, out, w_next=w, with_u=torch.ones(2), out=out)
        told.append((type(caught.value), str(caught.value)))
        assert torch.equal(out, before)
    assert told[0] == told[1] and told[0][0] is not SystemError
    assert host.norm_mx8(x, out, None, None, 1.0, w, 1e-6, torch.ones(2), None) is None
    # what has one counts as it does in Python
    for flag, has in ((1, True), ([], False), (torch.ones(1), True), ("", False)):
        assert ("u" in binding.moe_residual_norm_mx8(x, out, w_next=w, with_u=flag)) == has
