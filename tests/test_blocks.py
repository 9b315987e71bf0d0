"""run_blocks on the host: which blocks it holds and what it asks of them.  The norms and the blocks are
stand-ins; their arithmetic is tested with a GPU."""
import gc
import weakref

import pytest
import torch

from mixture_experts_routed_gate_gb300 import binding
from mixture_experts_routed_gate_gb300.block import MoEBlock, Rows8, run_blocks


@pytest.fixture
def norms(monkeypatch):
    def norm(y, res, w_post=None, gate=None, alpha=1.0, w_next=None, eps=None, out=None):
        return dict(out=res) if w_next is None else dict(u=res, q=res, sf=res, out=res)
    monkeypatch.setattr(binding, "moe_residual_norm", norm)
    monkeypatch.setattr(binding, "moe_residual_norm_mx8", norm)
    monkeypatch.setattr(MoEBlock, "layer", lambda self, u, err=None: u.u if isinstance(u, Rows8) else u)


def make(eight=False, last=False):
    experts = object.__new__(binding.Mx8Experts) if eight else ()
    return MoEBlock(None, None, experts, 1, w_next=None if last else 1)


def test_blocks_are_made_as_they_are_needed(norms):
    """Of a generator's blocks no more than two are there at a time: the one that runs and the next."""
    there, most = weakref.WeakSet(), []

    class Counted(MoEBlock):
        __hash__ = object.__hash__

        def __call__(self, u, res, err=None, rows8=False):
            gc.collect()
            most.append(len(there))
            return super().__call__(u, res, err, rows8)

    def loaded():
        for i in range(6):
            b = Counted(None, None, object.__new__(binding.Mx8Experts) if i % 2 else (), 1, w_next=1)
            there.add(b)
            yield b
            del b
    run_blocks(loaded(), torch.zeros(2, 4), 1)
    assert len(most) == 6 and max(most) == 2 and most[-1] == 1


def test_what_each_block_gets_and_is_asked_for(norms, monkeypatch):
    seen, call = [], MoEBlock.__call__

    def watched(self, u, res, err=None, rows8=False):
        seen.append((isinstance(u, Rows8), rows8))
        return call(self, u, res, err, rows8)
    monkeypatch.setattr(MoEBlock, "__call__", watched)
    run_blocks(iter([make(True), make(), make(True), make(True), make(last=True)]), torch.zeros(2, 4), 1)
    assert seen == [(True, False), (False, True), (True, True), (True, False), (False, False)]
    x = torch.zeros(2, 4)
    u, res = run_blocks([], x, 1)
    assert u is x and res is not x
    with pytest.raises(ValueError, match="only the last block"):
        run_blocks([make(last=True), make()], x, 1)
    assert run_blocks((make(last=True),), x, 1)[0] is None


def test_a_callable_before_an_8_bit_block(norms):
    """A program's own (u, res, err) -> (u, res) among the blocks: it is asked for no 8-bit rows."""
    seen = []

    def own(u, res, err):
        seen.append(u)
        return u + 1, res
    x = torch.zeros(2, 4)
    u, _ = run_blocks([own, make(True), own], x, 1)
    assert len(seen) == 2 and seen[0] is x and torch.equal(u, torch.ones(2, 4))
