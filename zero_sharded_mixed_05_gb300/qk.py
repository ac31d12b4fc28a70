"""The query/key norm with rotation for torch programs: a callable that keeps
the handle and takes part in autograd (first derivatives; a second one is an
error).

    norm = QkNormRope(make_qk_config(q_heads=8, k_heads=2, head_dim=64))
    q, k = norm(q, k, q_gain, k_gain, cos, sin, positions)
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (make_qk_config, zero_qk_create, zero_qk_destroy, zero_qk_norm_rope,
               zero_qk_norm_rope_backward)

__all__ = ["QkNormRope", "make_qk_config", "rotation_tables"]


def rotation_tables(n_pos: int, rotary_dim: int, base: float = 10000.0, device="cuda"):
    """cos and sin of position * base^(-2j / rotary_dim), binary32
    [n_pos, rotary_dim / 2] (angles in binary64)."""
    j = torch.arange(0, rotary_dim, 2, device=device, dtype=torch.float64)
    angle = torch.arange(n_pos, device=device, dtype=torch.float64)[:, None] * \
        base ** (-j / max(rotary_dim, 1))
    return angle.cos().float(), angle.sin().float()


class _Apply(torch.autograd.Function):
    @staticmethod
    def forward(ctx, owner, q, k, q_gain, k_gain, cos, sin, positions):
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        zero_qk_norm_rope(owner._handle, q, k, q_out, k_out, q_gain, k_gain, cos, sin, positions)
        ctx.owner = owner          # the handle is there for the backward pass
        ctx.save_for_backward(q, k, q_gain, k_gain, cos, sin, positions)
        return q_out, k_out

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_gain, k_gain, cos, sin, positions = ctx.saved_tensors
        dq, dk = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k))
        dqg, dkg = (torch.empty_like(gain) if wanted else None
                    for gain, wanted in zip((q_gain, k_gain), ctx.needs_input_grad[3:5]))
        zero_qk_norm_rope_backward(ctx.owner._handle, dq_out.contiguous(), dk_out.contiguous(), q, k, dq,
                                   dk, dqg, dkg, q_gain, k_gain, cos, sin, positions)
        return None, dq, dk, dqg, dkg, None, None, None


class QkNormRope:
    """Owns a handle of `cfg` (with at least one key head); calls are ordered as
    the handle's are: on one stream, or synchronized by the caller.  The handle
    lives until `close()`, or until neither this object nor a graph that came
    from it is left."""

    def __init__(self, cfg):
        if cfg.k_heads < 1:
            raise ValueError("QkNormRope takes queries and keys")
        self._handle = zero_qk_create(cfg)

    def __call__(self, q, k, q_gain, k_gain, cos, sin, positions):
        """q [tokens, q_heads, D] and k [tokens, k_heads, D] (heads contiguous),
        binary32 gains (None: ones), tables and positions as `zero_qk_norm_rope`
        takes them.  A gain that requires no gradient costs no sums."""
        return _Apply.apply(self, q, k, q_gain, k_gain, cos, sin, positions)

    def close(self):
        if self._handle is not None:
            zero_qk_destroy(self._handle)
            self._handle = None

    def __del__(self):
        if getattr(self, "_handle", None) is not None:
            self.close()
