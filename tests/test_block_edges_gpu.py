"""Calls of the join at the edges of what its documentation allows, on the GPU
against the formulas in 64 bits.  Tolerances are test_block_gpu.py's where none
is given."""
import pytest

import block_ref as R
from test_block_gpu import Case, blank, rows, z  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [512, 517])
@pytest.mark.parametrize("fill", ["nan", "inf"])
def test_the_norm_alone_does_not_see_the_branch_s_gain(z, D, fill):  # noqa: F811
    import torch
    c = Case(z, (300, D, "bf16", "fp32", False, True, "none", 0.0, 0.2, "own", 1.0, 1.0, False), 20)
    c.y_gain = None
    want = (c.forward()[1], *c.backward(c.x).values())
    c.y_gain = torch.full((D,), float(fill), device="cuda")
    got = (c.forward()[1], *c.backward(c.x).values())
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    c.close()


@pytest.mark.parametrize("D,dtype,layout", [(640, "fp32", "own"), (517, "fp32", "own"), (640, "bf16", "own"),
                                            (333, "bf16", "odd"), (4104, "bf16", "own"), (4103, "fp32", "own"),
                                            (8200, "bf16", "own"), (8201, "bf16", "odd")])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_a_gradient_of_rows_of_extreme_sizes(z, monkeypatch, D, dtype, layout, p):  # noqa: F811
    """x' and y of 2^-56, 1 and 2^56 together, the branch scaled by 2^-10 to 2^10
    behind its norm: squares are within binary32's range, products of x', dx' and y
    are not.  dy goes down to 2^-56 2^-56 2^-10 of numbers below one: into bf16's
    subnormals (below 2^-126), whose half step is 2^-134 whatever the number."""
    import torch
    monkeypatch.setattr(R, "EPS", 0.0)
    sizes = [(a, b, e) for a in (-56, 0, 56) for b in (-56, 0, 56) for e in (-10, 0, 10)]
    T = len(sizes)
    c = Case(z, (T, D, dtype, "fp32", True, True, "plain", p, 0.0, layout, 1.0, 1.0, True), 21)
    z.zero_block_destroy(c.h)
    cfg = z.make_block_config(D, dtype=z.FP32 if dtype == "fp32" else z.BF16, stream_dtype=z.FP32, norm_branch=True,
                              gate=z.GATE_PLAIN, eps=0.0, dropout=p)
    c.h = z.zero_block_create(cfg)
    sx, sy, sg = (2.0 ** torch.tensor(s, device="cuda", dtype=torch.float32)[:, None] for s in zip(*sizes))
    c.x.mul_(sx)                   # powers of two: nothing is rounded
    c.y.mul_(sy.to(c.y.dtype))
    c.gate.mul_(sg.to(c.gate.dtype))
    c.dxo.div_(sx)
    got = c.backward(c.x)
    out, tol = c.ref().backward(c.x, c.dxo, c.dh)
    assert all(v.isfinite().all() for v in out.values())
    if dtype == "bf16":
        tol["dy"] = tol["dy"] + 2.0 ** -134
    c.check(got, out, tol)
    c.close()


@pytest.mark.parametrize("D,layout", [(64, "own"), (61, "odd"), (4104, "own")])
def test_a_gate_beside_a_binary32_stream(z, D, layout):  # noqa: F811
    """The branch alone (x = 0) as the stream has it.  With e = exp(-|g|), in halves of
    a unit in the last place (2^-24): e within four, 1 + e one, its reciprocal four, the
    product of both one; the product with y y_gain one and that one itself one: 12 2^-24
    of the branch, to first order."""
    import torch
    T = 500
    c = Case(z, (T, D, "fp16", "fp32", False, True, "sigmoid", 0.0, 0.0, layout, 1.0, 1.0, True), 22)
    c.x.zero_()
    g = torch.Generator(device="cuda").manual_seed(22)
    c.gate.copy_(14 * (2 * torch.rand(T, D, device="cuda", generator=g) - 1))
    xo, _ = c.forward()
    ref = c.y.double() * c.y_gain.double() * torch.sigmoid(c.gate.double())
    assert ((xo.double() - ref).abs() <= 12.1 * R.E32 * ref.abs()).all()
    c.close()


@pytest.mark.parametrize("eps", [1e-12, 1e-30, 1e-44, 1e-50, 1e-300])
@pytest.mark.parametrize("D", [64, 61])
def test_rows_of_zeros_by_any_eps(z, D, eps):  # noqa: F811
    """Zero over the root of any eps that is not zero is zero, of both norms; and
    the gradient of such rows is dx' for the stream, as no term of the norm's is
    with dh = 0."""
    import torch
    h = z.zero_block_create(z.make_block_config(D, dtype=z.FP32, norm_branch=True, eps=eps))
    x = torch.zeros(9, D, device="cuda")
    xo, ho = torch.ones_like(x), torch.ones_like(x)
    z.zero_block_join(h, x, x, xo, ho, None, None)
    assert not xo.any() and not ho.any()
    dx, dxo, dh = torch.zeros_like(x), torch.randn_like(x), torch.zeros_like(x)
    z.zero_block_join_backward(h, dxo, dh, xo, x, dx, None, None, None, None, None)
    assert torch.equal(dx, dxo)
    z.zero_block_destroy(h)


@pytest.mark.parametrize("D", [512, 517])
@pytest.mark.parametrize("norm_out", [False, True])
def test_a_gain_that_nothing_is_scaled_by_is_not_seen(z, D, norm_out):  # noqa: F811
    """Without norm_out there is no h for it, and without a gradient of h it has no
    part in those of x and y."""
    import torch
    c = Case(z, (300, D, "bf16", "bf16", True, norm_out, "none", 0.1, 0.2, "own", 1.5, 1.0, True), 23)
    results = []
    for c.gain in (None, torch.full((D,), float("nan"), device="cuda")):
        xo = c.like("bf16")
        if not norm_out:
            z.zero_block_join(c.h, c.x, c.y, xo, None, c.y_gain, c.gain, **c.kw)
        results.append((xo, *c.backward(c.x, dh=None).values()))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    c.close()
