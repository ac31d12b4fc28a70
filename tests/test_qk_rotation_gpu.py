"""Rotation without the norm, on the GPU: its gradient needs the results' gradients
and the angles alone."""
import pytest

from test_qk_axes_gpu import CASES, Case, z  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rotation_alone_keeps_no_rows(z):  # noqa: F811
    """Queries and keys may be overwritten before the backward pass, which does not
    look at them, and what is not needed elsewhere is freed."""
    import torch
    from zero_sharded_mixed_05_gb300.qk import QkNormRope, axis_of_pairs, make_qk_axes, rotation_tables
    g = torch.Generator(device="cuda").manual_seed(31)
    T, hq, hk, D = 40, 4, 2, 64
    axis = axis_of_pairs((16, 16))
    cos, sin = rotation_tables(50, D, axis=axis)
    pos = torch.randint(0, 50, (2, T), device="cuda", generator=g)
    norm = QkNormRope(z.make_qk_config(hq, hk, D, dtype=z.FP32), make_qk_axes(axis, normalise=False))
    leaves = [torch.randn(T, h, D, device="cuda", generator=g).requires_grad_() for h in (hq, hk)]
    w = [torch.randn(T, h, D, device="cuda", generator=g) for h in (hq, hk)]
    grads = []
    for change in (False, True):
        q, k = (t.clone() for t in leaves)
        qo, ko = norm(q, k, None, None, cos, sin, pos)
        if change:
            with torch.no_grad():
                q.fill_(float("nan"))
                k.fill_(float("nan"))
        grads.append(torch.autograd.grad((qo * w[0]).sum() + (ko * w[1]).sum(), leaves))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    # the gradients of the results alone, through the call itself
    dq, dk = torch.empty_like(w[0]), torch.empty_like(w[1])
    z.zero_qk_norm_rope_backward(norm._handle, *w, None, None, dq, dk, None, None, None, None, cos, sin, pos)
    assert torch.equal(dq, grads[0][0]) and torch.equal(dk, grads[0][1])
    with pytest.raises(ValueError):            # a norm's gradient needs them
        full = QkNormRope(z.make_qk_config(hq, hk, D, dtype=z.FP32), make_qk_axes(axis))
        z.zero_qk_norm_rope_backward(full._handle, *w, None, None, dq, dk, None, None, None, None, cos, sin, pos)
    norm.close()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotation_back_does_not_see_queries_or_keys(z, case):  # noqa: F811
    import torch
    c = Case(z, case, normalise=False, seed=6)
    want = c.backward(c.many, *c.many_at())
    c.q.fill_(float("nan"))
    c.k.fill_(float("nan"))
    assert all(torch.equal(a, b) for a, b in zip(c.backward(c.many, *c.many_at()), want))
    c.close()
