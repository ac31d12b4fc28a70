"""The operators together: gradients through the autograd wrapper, and the
example's training loop."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_autograd_gradients_are_the_formulas():
    """Against torch's autograd on the plain formula in 64 bits; the wrapper
    adds nothing to the kernels' own error: binary32 throughout, sums of 64 and
    of 30 tokens x 4 heads, (64 + 120 + 16) 2^-24 of the largest terms, which
    are below 8 here."""
    import torch
    import zero_sharded_mixed_05_gb300 as z
    from zero_sharded_mixed_05_gb300.qk import QkNormRope, rotation_tables
    g = torch.Generator(device="cuda").manual_seed(1)
    T, hq, hk, D = 30, 4, 2, 64
    q, k, wq, wk = (torch.randn(T, h, D, device="cuda", generator=g) for h in (hq, hk, hq, hk))
    qg, kg = (1 + 0.1 * torch.randn(D, device="cuda", generator=g) for _ in range(2))
    cos, sin = rotation_tables(64, D)
    pos = torch.randint(0, 64, (T,), device="cuda", generator=g)
    norm = QkNormRope(z.make_qk_config(hq, hk, D, dtype=z.FP32))
    got = [t.clone().requires_grad_() for t in (q, k, qg, kg)]
    qo, ko = norm(*got, cos, sin, pos)
    ((qo * wq).sum() + (ko * wk).sum()).backward()
    ref = [t.double().requires_grad_() for t in (q, k, qg, kg)]

    def plain(x, gain):
        y = x * (x.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * gain
        c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
        u, v = y[..., :D // 2], y[..., D // 2:]
        return torch.cat((u * c - v * s, v * c + u * s), -1)
    ((plain(ref[0], ref[2]) * wq).sum() + (plain(ref[1], ref[3]) * wk).sum()).backward()
    for a, b in zip(got, ref):
        terms = 1 if a.dim() == 3 else T * hq
        assert ((a.grad.double() - b.grad).abs() <= 200 * 2.0 ** -24 * 8 * terms).all()
    norm.close()
    with pytest.raises(ValueError):
        QkNormRope(z.make_qk_config(2, 0, D))


def test_the_example_learns():
    """log(64) = 4.16 at the start; a fixed function of two tokens is learnt to
    well below half of that in a hundred steps."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_muon
    finally:
        sys.path.pop(0)
    losses = train_muon.train(steps=100, width=128, layers=2, quiet=True)
    assert 3.9 < losses[0] < 5.5
    assert sum(losses[-5:]) / 5 < 2.0, losses[::10]
