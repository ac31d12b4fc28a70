"""The query/key norm with rotation for torch programs: a callable that keeps
the handle and takes part in autograd (first derivatives; a second one is an
error).

    norm = QkNormRope(make_qk_config(q_heads=8, k_heads=2, head_dim=64))
    q, k = norm(q, k, q_gain, k_gain, cos, sin, positions)

With positions on several axes (time, height and width of a video's patches):

    axis = axis_of_pairs((16, 24, 24))
    norm = QkNormRope(make_qk_config(q_heads=8, k_heads=2, head_dim=128), make_qk_axes(axis))
    q, k = norm(q, k, q_gain, k_gain, cos, sin, positions)          # positions [3, tokens]
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (make_qk_axes, make_qk_config, zero_qk_create, zero_qk_destroy, zero_qk_norm_rope,
               zero_qk_norm_rope_backward)

__all__ = ["QkNormRope", "axis_of_pairs", "make_qk_axes", "make_qk_config", "rotation_tables"]


def axis_of_pairs(sections, alternate=False):
    """The axis of each rotated pair: `sections[a]` pairs of axis a, one section
    after another, or (`alternate`) the axes in turn while they have pairs left."""
    if not alternate:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                left[a] -= 1
                out.append(a)
    return out


def rotation_tables(n_pos: int, rotary_dim: int, base: float = 10000.0, device="cuda", axis=None):
    """cos and sin of position * base^(-2j / rotary_dim), binary32
    [n_pos, rotary_dim / 2] (angles in binary64).  With `axis` (of each pair)
    every axis has frequencies from 1 down of its own: base^(-i / n) for the
    i-th of its n pairs."""
    j = torch.arange(0, rotary_dim, 2, device=device, dtype=torch.float64)
    power = j / max(rotary_dim, 1)
    if axis is not None:
        if len(axis) != rotary_dim // 2:
            raise ValueError(f"axis must name {rotary_dim // 2} pairs")
        seen = [axis[:i].count(a) / axis.count(a) for i, a in enumerate(axis)]
        power = torch.tensor(seen, device=device, dtype=torch.float64)
    angle = torch.arange(n_pos, device=device, dtype=torch.float64)[:, None] * base ** -power
    return angle.cos().float(), angle.sin().float()


class _Apply(torch.autograd.Function):
    @staticmethod
    def forward(ctx, owner, q, k, q_gain, k_gain, cos, sin, positions):
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        zero_qk_norm_rope(owner._handle, q, k, q_out, k_out, q_gain, k_gain, cos, sin, positions)
        ctx.owner = owner          # the handle is there for the backward pass
        # a rotation back needs neither queries nor keys
        rows = (q, k) if owner._normalise else (None, None)
        ctx.save_for_backward(*rows, q_gain, k_gain, cos, sin, positions)
        return q_out, k_out

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_gain, k_gain, cos, sin, positions = ctx.saved_tensors
        dq, dk = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (dq_out, dk_out))
        dqg, dkg = (torch.empty_like(gain) if wanted else None
                    for gain, wanted in zip((q_gain, k_gain), ctx.needs_input_grad[3:5]))
        zero_qk_norm_rope_backward(ctx.owner._handle, dq_out.contiguous(), dk_out.contiguous(), q, k, dq,
                                   dk, dqg, dkg, q_gain, k_gain, cos, sin, positions)
        return None, dq, dk, dqg, dkg, None, None, None


class QkNormRope:
    """Owns a handle of `cfg` (with at least one key head) and, for positions on
    several axes, `axes` of make_qk_axes; calls are ordered as
    the handle's are: on one stream, or synchronized by the caller.  The handle
    lives until `close()`, or until neither this object nor a graph that came
    from it is left."""

    def __init__(self, cfg, axes=None):
        if cfg.k_heads < 1:
            raise ValueError("QkNormRope takes queries and keys")
        self._normalise = axes is None or bool(axes.normalise)
        self._handle = zero_qk_create(cfg) if axes is None else zero_qk_create(cfg, axes)

    def __call__(self, q, k, q_gain, k_gain, cos, sin, positions):
        """q [tokens, q_heads, D] and k [tokens, k_heads, D] (heads contiguous),
        binary32 gains (None: ones), tables and positions as `zero_qk_norm_rope`
        takes them.  A gain that requires no gradient costs no sums.  Without the
        norm the backward pass keeps neither q nor k, which may be overwritten."""
        return _Apply.apply(self, q, k, q_gain, k_gain, cos, sin, positions)

    def close(self):
        if self._handle is not None:
            zero_qk_destroy(self._handle)
            self._handle = None

    def __del__(self):
        if getattr(self, "_handle", None) is not None:
            self.close()
