"""A pre-norm MoE block from the library's entry points: the routed layer with
the norms on its two sides.

    y    = experts(u)                       u: the residual stream, normalised
    res' = res + alpha * gate * norm(y)
    u'   = norm(res') * w_next              the next block's input

Serving walks blocks of it: :func:`run_blocks` normalises the first block's
input and hands each block's (u', res') to the next.  The layer itself takes
one of four paths, by what the block holds and how many tokens come: 4-bit or
8-bit experts (:class:`.binding.Mx4Experts`, :class:`.binding.Mx8Experts`),
``moe_forward_few`` for at most :data:`FEW_TOKENS` tokens, ``moe_forward``
otherwise.  8-bit experts read u in 8 bits, which the norm before them writes
beside u itself (the gate reads that one): a :class:`Rows8`.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import NamedTuple

import torch

from . import binding

# Up to here moe_forward_few is the faster one at both layer sizes measured
# (T = 8: 68 against 78 us at 2048 / 768, 64 experts, top-6, fp16, and 726
# against 778 us at 7168 / 2048, 256 experts, top-8, bf16; at T = 12 it is 91
# against 87 and 956 against 1022 us).  4-bit experts take moe_forward_mx4 at any
# T: at T = 8 48 and 263 us, at T = 1 34 (16-bit experts: 27) and 81 (122).
FEW_TOKENS = 8


class Rows8(NamedTuple):
    """The norm's result u [T, H] with the same rows in 8 bits: elements q, scales sf."""

    u: torch.Tensor
    q: torch.Tensor
    sf: torch.Tensor


@dataclass
class MoEBlock:
    """Weights of one block.  ``experts``: (w_gate, w_up, w_down) in the gate's
    16-bit type, :class:`.binding.Mx4Experts` or :class:`.binding.Mx8Experts`.  ``w_post``: weight of the norm
    on the layer's output (None: no such norm); ``gate``: per channel [H], per
    token [T, 1] or None; ``w_next``: weight of the norm before the next block
    (None: the block is the last, and returns no u)."""

    w_g: torch.Tensor
    bias: torch.Tensor | None
    experts: object
    k: int
    w_post: torch.Tensor | None = None
    gate: torch.Tensor | None = None
    alpha: float = 1.0
    w_next: torch.Tensor | None = None
    eps: float = 1e-6

    def layer(self, u, err=None):
        """The routed layer alone: u [T, d_hidden], or its :class:`Rows8`, to [T, d_hidden]."""
        rows = None
        if isinstance(u, Rows8):
            u, rows = u.u, (u.q, u.sf)
        if isinstance(self.experts, binding.Mx8Experts):
            return binding.moe_forward_mx8(u, self.w_g, self.bias, self.experts, self.k, rows, err=err)
        if isinstance(self.experts, binding.Mx4Experts):
            return binding.moe_forward_mx4(u, self.w_g, self.bias, self.experts, self.k, err=err)
        forward = binding.moe_forward_few if u.shape[0] <= FEW_TOKENS else binding.moe_forward
        return forward(u, self.w_g, self.bias, *self.experts, self.k, err=err)

    def __call__(self, u, res, err=None, rows8=False):
        """(u', res'); res is updated in place.  u' is None for the last block, and
        a :class:`Rows8` with ``rows8`` (the next block's experts are 8-bit)."""
        args = (self.layer(u, err), res, self.w_post, self.gate, self.alpha, self.w_next, self.eps)
        if rows8 and self.w_next is not None:
            got = binding.moe_residual_norm_mx8(*args, out=res)
            return Rows8(got["u"], got["q"], got["sf"]), got["out"]
        got = binding.moe_residual_norm(*args, out=res)
        return got.get("u"), got["out"]


def _reads_rows8(block) -> bool:
    return isinstance(getattr(block, "experts", None), binding.Mx8Experts)


def run_blocks(blocks, x, w_first, eps: float = 1e-6, err=None):
    """x [T, d_hidden], the residual stream, through the blocks; w_first: weight
    of the norm before the first one.  Returns (u, res): the last block's u' (or
    None) and the residual stream; x is left as it was.  ``blocks`` may make them
    as they are needed: the next one is asked for when one runs, whose norm writes
    what the next one reads, and none is held behind that."""
    blocks = iter(blocks)
    block = next(blocks, None)
    if _reads_rows8(block):
        got = binding.moe_residual_norm_mx8(None, x, w_next=w_first, eps=eps)
        u = Rows8(got["u"], got["q"], got["sf"])
    else:
        u = binding.moe_residual_norm(None, x, w_next=w_first, eps=eps)["u"]
    res = x.clone()
    while block is not None:
        if u is None:
            raise ValueError("only the last block may have no w_next")
        following = next(blocks, None)
        # what is no MoEBlock gives u alone, which an 8-bit layer quantises for itself
        u, res = block(u, res, err, rows8=True) if isinstance(block, MoEBlock) and _reads_rows8(following) else block(u, res, err)
        block = following
    return u, res
