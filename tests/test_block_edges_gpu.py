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


@pytest.mark.parametrize("D,dtype,stream", [(520, "bf16", "fp32"), (517, "bf16", "bf16"), (4104, "fp16", "fp16"),
                                            (61, "fp32", "fp32")])
def test_rows_in_reverse(z, D, dtype, stream):  # noqa: F811
    """Negative strides, from the last row up, of every tensor: the same numbers, in
    the same places of the results.  The mask and the dropout go by the token, so
    that they are left out."""
    import ctypes
    import torch
    T = 333
    c = Case(z, (T, D, dtype, stream, True, True, "sigmoid", 0.0, 0.0, "own", 1.0, 1.0, True), 24)

    def back(t):
        return z.zero_block_rows(t.data_ptr() + (T - 1) * t.stride(0) * t.element_size(), -t.stride(0))
    c.kw.update(mask=None)
    xo, h = c.forward()
    want = c.backward(c.x)
    names = dict(x=c.x, y=c.y, gate=c.gate, x_out=torch.full_like(c.x, 7), h=torch.full_like(c.y, 7))
    b = z.zero_block_buffers()
    b.tokens = T
    for k, t in names.items():
        setattr(b, k, back(t))
    b.y_gain, b.gain = c.y_gain.data_ptr(), c.gain.data_ptr()
    stream_now = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert z.lib().zero_block_join(c.h, ctypes.byref(b), stream_now) == z.ZERO_OK
    assert torch.equal(names["x_out"], xo) and torch.equal(names["h"], h)
    res = dict(dx=torch.full_like(c.x, 7), dy=torch.full_like(c.y, 7), dgate=torch.full_like(c.y, 7))
    for k, t in dict(x_out=c.x, dx_out=c.dxo, dh=c.dh, **res).items():
        setattr(b, k, back(t))
    dyg, dg = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    b.dy_gain, b.dgain = dyg.data_ptr(), dg.data_ptr()
    assert z.lib().zero_block_join_backward(c.h, ctypes.byref(b), stream_now) == z.ZERO_OK
    assert all(torch.equal(res[k], want[k]) for k in res)
    out, tol = c.ref().backward(c.x, c.dxo, c.dh)
    R.near(dyg, out["dy_gain"], tol["dy_gain"], "fp32", "dy_gain")       # summed in another order
    R.near(dg, out["dgain"], tol["dgain"], "fp32", "dgain")
    c.close()


def test_dropout_of_rows_in_reverse(z):  # noqa: F811
    import ctypes
    import torch
    for D in (64, 61):
        T = 70
        x, out = torch.randn(T, D, device="cuda"), torch.full((T, D), 7.0, device="cuda")
        b = z.zero_drop_buffers()
        b.in_, b.out = (t.data_ptr() + (T - 1) * D * 4 for t in (x, out))
        b.rows, b.cols, b.in_stride, b.out_stride, b.dtype, b.p = T, D, -D, -D, z.FP32, 0.5
        b.rng.seed = 9
        assert z.lib().zero_dropout(ctypes.byref(b), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == z.ZERO_OK
        keep = torch.from_numpy(R.kept(T, D, 0.5, 9)).cuda().flip(0)
        assert torch.equal(out, torch.where(keep, x * 2, torch.zeros_like(x)))


@pytest.mark.parametrize("D,T", [(4096, 540000), (777, 2800000)])
def test_more_than_32_bits_of_numbers_in_many_rows(z, D, T):  # noqa: F811
    """2.2e9 numbers a tensor, in place: rows at both ends and where the numbers and
    the bytes pass 2^31 and 2^32, and dgain, which no dropout changes, as a whole."""
    import torch
    assert T * D > 2 ** 31 and T * D * 2 > 2 ** 32
    p, rng = 0.1, (3, 4, 5)
    g = torch.Generator(device="cuda").manual_seed(25)

    def fill():
        return torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    x, y = fill(), fill()
    h = z.zero_block_create(z.make_block_config(D, norm_branch=True, dropout=p))
    kw = dict(seed=rng[0], call=rng[1], step=rng[2])
    places = [0, 2 ** 30 // D - 4, 2 ** 31 // D - 4, T - 8]

    def ref(at, xs, ys):
        r = R.Ref(xs, ys, None, None, post=True, p=p, rng=rng)
        r.keep = torch.from_numpy(R.kept(8, D, p, *rng, first_row=at)).cuda()
        return r
    before = [(x[a:a + 8].clone(), y[a:a + 8].clone()) for a in places]
    z.zero_block_join(h, x, y, x, y, None, None, **kw)
    for a, (xs, ys) in zip(places, before):
        x64, h64, tx, th = ref(a, xs, ys).forward()
        R.near(x[a:a + 8], x64, tx, "bf16", a)
        R.near(y[a:a + 8], h64, th, "bf16", a)
    y.normal_(generator=g)
    dxo, dh = fill(), fill()
    want, bound = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2))
    for a in range(0, T, 20000):
        xs = x[a:a + 20000].double()
        terms = dh[a:a + 20000].double() * xs * (xs.square().mean(-1, keepdim=True) + R.EPS) ** -0.5
        want += terms.sum(0)
        bound += terms.abs().sum(0)
    before = [tuple(t[a:a + 8].clone() for t in (x, y, dxo, dh)) for a in places]
    dg = torch.empty(D, device="cuda")
    z.zero_block_join_backward(h, dxo, dh, x, y, dxo, dh, None, dg, None, None, **kw)
    for a, (xs, ys, os, hs) in zip(places, before):
        out, tol = ref(a, xs, ys).backward(xs, os, hs)
        R.near(dxo[a:a + 8], out["dx"], tol["dx"], "bf16", a)
        R.near(dh[a:a + 8], out["dy"], tol["dy"], "bf16", a)
    # a CTA sums at most T / 152 rows of one team, then 600 parts and fewer
    assert ((dg.double() - want).abs() <= (T / 152 + 600 + D + 48) * R.E32 * bound).all()
    z.zero_block_destroy(h)
