"""The join of a block with the residual stream, and dropout, for torch programs:
callables that take part in autograd (first derivatives; a second one is an
error).

    join = BlockJoin(make_block_config(768, dropout=0.1))
    h = join.norm(x, gain)                                  # the first block's input
    x, h = join(x, block(h), y_gain, gain, seed=seed, call=layer, step=step)

A program gives each dropout of a step its own `call`, and each step its own
`step`: an integer, or, for a captured step, an int64 tensor on the device that
every replay reads (and that stays as it is until the backward pass is done).
A call counts its rows from 0: micro-batches of one step, and ranks that have a
shard of the batch or of the sequence, drop the same places unless each is given
a `seed` (or `call`) of its own, as seed + rank.

For a step captured in a CUDA graph hold to what torch asks of any captured
backward pass: no autograd graph of the same leaves, made outside the capture,
may be alive during it.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (GATE_NONE, GATE_PLAIN, GATE_SIGMOID, make_block_config, zero_block_create,
               zero_block_destroy, zero_block_join, zero_block_join_backward, zero_dropout)

__all__ = ["BlockJoin", "GATE_NONE", "GATE_PLAIN", "GATE_SIGMOID", "dropout", "make_block_config"]


def _rows(t):
    """`t` with contiguous rows."""
    return t if t is None or t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class _Join(torch.autograd.Function):
    @staticmethod
    def forward(ctx, owner, x, y, y_gain, gain, gate, mask, seed, call, step):
        x_out = None if y is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        h = torch.empty(x.shape, dtype=owner._dtype, device=x.device) if owner._norm_out else None
        zero_block_join(owner._handle, x, y, x_out, h, y_gain, gain, gate=gate, mask=mask, seed=seed,
                        call=call, step=step)
        ctx.owner = owner          # the handle is there for the backward pass
        ctx.rng = seed, call, None if isinstance(step, torch.Tensor) else step
        ctx.save_for_backward(x if y is None else x_out, y, y_gain, gain, gate, mask,
                              step if isinstance(step, torch.Tensor) else None)
        ctx.set_materialize_grads(False)
        return x_out, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dx_out, dh):
        x_out, y, y_gain, gain, gate, mask, step = ctx.saved_tensors
        nothing = (None,) * 10
        if dx_out is None and dh is None:
            return nothing
        want = ctx.needs_input_grad
        owner = ctx.owner

        def like(t, wanted):
            return torch.empty(t.shape, dtype=t.dtype, device=t.device) if t is not None and wanted else None
        dx, dy, dgate = like(x_out, want[1]), like(y, want[2]), like(gate, want[5])
        dyg, dg = like(y_gain, want[3]), like(gain, want[4])
        if y is None and dyg is not None:
            dyg.zero_()
        seed, call, number = ctx.rng
        zero_block_join_backward(owner._handle, _rows(dx_out), _rows(dh), x_out, y, dx, dy,
                                 None if y is None else dyg, dg, y_gain, gain, gate=gate, dgate=dgate,
                                 mask=mask, seed=seed, call=call, step=number if step is None else step)
        return None, dx, dy, dyg, dg, dgate, None, None, None, None


class BlockJoin:
    """Owns a handle of `cfg`; calls are ordered as the handle's are: on one
    stream, or synchronized by the caller.  The handle lives until `close()`, or
    until neither this object nor a graph that came from it is left."""

    def __init__(self, cfg):
        self._handle = None
        self._dtype = (torch.float16, torch.bfloat16, torch.float32)[cfg.dtype]
        self._norm_out, self._gated = bool(cfg.norm_out), cfg.gate != GATE_NONE
        self._handle = zero_block_create(cfg)

    def __call__(self, x, y, y_gain=None, gain=None, gate=None, mask=None, seed=0, call=0, step=0):
        """(x', h) of the stream `x` [tokens, D] and the block's output `y`; h is
        None without norm_out.  Gains are binary32 [D] or None (ones), `mask` bool
        [tokens] or None, `gate` as `y`, and given where the configuration has one."""
        if y is None:
            raise ValueError("y is None: norm() normalises the stream alone")
        if self._gated != (gate is not None):
            raise ValueError("a gate is given " + ("to a join without one" if gate is not None
                                                   else "where the configuration has one"))
        return _Join.apply(self, x, y, y_gain, gain, gate, mask, seed, call, step)

    def norm(self, x, gain=None, mask=None):
        """h of the stream alone."""
        if not self._norm_out:
            raise ValueError("a join without norm_out has no norm")
        return _Join.apply(self, x, None, None, gain, None, mask, 0, 0, 0)[1]

    def close(self):
        if self._handle is not None:
            zero_block_destroy(self._handle)
            self._handle = None

    def __del__(self):
        if getattr(self, "_handle", None) is not None:
            self.close()


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, call, step):
        x = x.contiguous()
        out = torch.empty_like(x)
        zero_dropout(x, out, p, seed=seed, call=call, step=step)
        ctx.rng = p, seed, call, None if isinstance(step, torch.Tensor) else step
        ctx.save_for_backward(step if isinstance(step, torch.Tensor) else None)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d):
        p, seed, call, number = ctx.rng
        (step,) = ctx.saved_tensors
        d = d.contiguous()
        dx = torch.empty_like(d)
        zero_dropout(d, dx, p, seed=seed, call=call, step=number if step is None else step)
        return dx, None, None, None, None


def dropout(x, p, seed=0, call=0, step=0):
    """`x` with numbers dropped, the others scaled by 1 / (1 - p), by the rule of
    zero_dropout; rows are of the last dimension."""
    return _Dropout.apply(x, p, seed, call, step)
