"""The join of a block with the residual stream, and dropout, on the GPU
against the formulas in 64 bits.

Tolerances.  A result is computed in binary32 and rounded once to its type: half
a step (2^-11 fp16, 2^-8 bf16, 2^-24 fp32, and fp16's subnormal spacing 2^-25),
plus the binary32 arithmetic, (D + 32) 2^-24 of the largest terms for what comes
of a sum of D numbers in any order; block_ref.py carries the terms.  Gains'
gradients add T such terms in some order.
"""
import pytest

import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import zero_sharded_mixed_05_gb300 as z
    z.lib()
    return z


def code(z, name):
    return dict(fp16=z.FP16, bf16=z.BF16, fp32=z.FP32)[name]


# tokens, D, dtype, stream, post, pre, gate, p, masked share, layout, alpha, beta, with y
CASES = [
    (1, 1, "fp32", "fp32", True, True, "none", 0.0, 0.0, "own", 1.0, 1.0, True),
    (1, 4096, "bf16", "bf16", True, True, "none", 0.0, 0.0, "own", 1.0, 1.0, True),
    (2, 7, "fp16", "fp32", False, True, "plain", 0.3, 0.0, "own", 1.5, 0.5, True),
    (3, 8, "bf16", "bf16", False, True, "sigmoid", 0.1, 0.0, "own", 1.0, 1.0, True),
    (5, 255, "bf16", "fp32", True, True, "sigmoid", 0.1, 0.0, "odd", 1.0, 1.0, True),
    (64, 256, "fp16", "fp16", False, True, "none", 0.1, 0.3, "own", 1.0, 1.0, True),
    (65, 264, "bf16", "bf16", True, False, "plain", 0.5, 0.3, "padded", -1.0, 2.0, True),
    (515, 777, "fp16", "fp16", True, True, "sigmoid", 0.1, 0.2, "own", 1.0, 1.0, True),
    (515, 777, "bf16", "bf16", False, True, "plain", 0.0, 0.2, "padded", 1.0, 1.0, True),
    (700, 768, "fp16", "fp32", False, True, "none", 0.1, 0.0, "own", 1.0, 1.0, True),
    (1500, 1000, "fp32", "fp32", True, True, "none", 0.0, 0.1, "own", 1.0, 1.0, True),
    (900, 2048, "bf16", "bf16", False, True, "sigmoid", 0.0, 0.0, "broadcast", 1.0, 1.0, True),
    (2000, 4096, "bf16", "bf16", True, True, "none", 0.1, 0.0, "own", 1.0, 1.0, True),
    (700, 4097, "bf16", "fp32", True, True, "none", 0.0, 0.0, "own", 1.0, 1.0, True),
    (900, 5000, "fp16", "fp16", True, True, "plain", 0.1, 0.1, "padded", 1.0, 1.0, True),
    (400, 8192, "fp32", "fp32", True, True, "sigmoid", 0.1, 0.0, "own", 1.0, 1.0, True),
    (333, 12288, "bf16", "fp32", True, True, "plain", 0.1, 0.0, "own", 1.0, 1.0, True),
    (310, 12287, "bf16", "fp32", True, True, "sigmoid", 0.1, 0.1, "own", 1.0, 1.0, True),
    (320, 16384, "bf16", "fp32", True, True, "none", 0.1, 0.0, "own", 1.0, 1.0, True),
    (315, 8191, "fp32", "fp32", True, True, "plain", 0.1, 0.0, "odd", 1.0, 1.0, True),
    (700, 2050, "fp32", "fp32", False, True, "sigmoid", 0.0, 0.1, "odd", 1.0, 1.0, True),
    (2500, 100, "bf16", "fp32", True, True, "none", 0.1, 0.1, "own", 1.0, 1.0, True),
    (3000, 12, "fp16", "fp16", True, True, "plain", 0.1, 0.1, "odd", 1.0, 1.0, True),
    (320, 16383, "fp16", "fp16", True, True, "plain", 0.1, 0.0, "odd", 1.0, 1.0, True),
    (3, 12345, "bf16", "bf16", False, True, "none", 0.1, 0.0, "own", 1.0, 1.0, True),
    (300, 1024, "bf16", "bf16", False, True, "none", 0.0, 0.2, "own", 1.0, 1.0, False),
    (301, 333, "fp16", "fp32", False, True, "none", 0.0, 0.2, "odd", 2.0, 1.0, False),
    (40, 128, "bf16", "bf16", False, False, "none", 1.0, 0.0, "own", 1.0, 1.0, True),
]
IDS = ["x".join(map(str, c[:2])) + "-" + "-".join(map(str, c[2:10])) + ("" if c[12] else "-norm") for c in CASES]


def blank(T, D, name, layout):
    """A [T, D] tensor of sevens in a layout."""
    import torch
    kw = dict(device="cuda", dtype=R.dt(name))
    if layout == "own":
        return torch.full((T, D), 7.0, **kw)
    if layout == "odd":            # an odd base address and an odd stride
        out = torch.full((T * (D + 3) + 1,), float("nan"), **kw)[1:].as_strided((T, D), (D + 3 - D % 2, 1))
    else:                          # rows on 16-byte boundaries
        out = torch.full((T, -(-D // 8) * 8 + 16), float("nan"), **kw)[:, :D]
    return out.fill_(7.0)


def rows(g, T, D, name, layout, big=1.0):
    import torch
    t = (torch.randn(T, D, device="cuda", generator=g) * big).to(R.dt(name))
    if layout == "broadcast":
        return t[:1].expand(T, D)
    return blank(T, D, name, layout).copy_(t)


class Case:
    def __init__(self, z, case, seed=0):
        import torch
        (self.T, self.D, self.dtype, self.stream, self.post, self.pre, self.kind, self.p, masked, layout,
         self.alpha, self.beta, with_y) = case
        g = torch.Generator(device="cuda").manual_seed(seed)
        T, D, plain = self.T, self.D, "own" if layout == "broadcast" else layout
        self.x = rows(g, T, D, self.stream, plain)
        self.y = rows(g, T, D, self.dtype, plain, 0.7) if with_y else None
        self.gate = rows(g, T, D, self.dtype, layout, 2.0) if self.kind != "none" else None
        self.dxo, self.dh = rows(g, T, D, self.stream, plain), rows(g, T, D, self.dtype, plain)
        self.y_gain = 1 + 0.2 * torch.randn(D, device="cuda", generator=g)
        self.gain = 1 + 0.2 * torch.randn(D + 1, device="cuda", generator=g)[1:].clone()
        self.mask = torch.rand(T, device="cuda", generator=g) >= masked if masked else None
        self.rng = (0xABCDEF0123456789, 0xFFFFFFFE, 2 ** 33 + 5)
        self.kw = dict(gate=self.gate, mask=self.mask, seed=self.rng[0], call=self.rng[1], step=self.rng[2])
        self.layout = plain
        cfg = z.make_block_config(D, dtype=code(z, self.dtype), stream_dtype=code(z, self.stream),
                                  norm_branch=self.post, norm_out=self.pre, alpha=self.alpha, beta=self.beta,
                                  gate=dict(none=z.GATE_NONE, plain=z.GATE_PLAIN, sigmoid=z.GATE_SIGMOID)[self.kind],
                                  dropout=self.p)
        self.z, self.h = z, z.zero_block_create(cfg)

    def like(self, name):
        """A result's buffer in the case's layout."""
        return blank(self.T, self.D, name, self.layout)

    def ref(self):
        return R.Ref(self.x, self.y, self.y_gain, self.gain, self.gate, self.kind, self.post, self.pre,
                     self.alpha, self.beta, self.p, self.mask, self.rng)

    def forward(self, gains=True):
        xo, h = self.like(self.stream), self.like(self.dtype)
        self.z.zero_block_join(self.h, self.x, self.y, xo if self.y is not None else None,
                               h if self.pre else None, self.y_gain, self.gain, **self.kw)
        return xo, h

    def backward(self, x_out, **override):
        import torch
        dx, dy, dg = (self.like(n) for n in (self.stream, self.dtype, self.dtype))
        dyg, dgain = (torch.full((self.D,), 7.0, device="cuda") for _ in range(2))
        a = dict(dx_out=self.dxo, dh=self.dh if self.pre else None, dx=dx, dy=dy if self.y is not None else None,
                 dy_gain=dyg, dgain=dgain)
        a.update(override)
        self.z.zero_block_join_backward(self.h, a["dx_out"], a["dh"], x_out, self.y, a["dx"], a["dy"],
                                        a["dy_gain"], a["dgain"], self.y_gain, self.gain,
                                        dgate=dg if self.gate is not None else None, **self.kw)
        return dict(dx=dx, dy=dy, dgate=dg, dy_gain=dyg, dgain=dgain)

    def check(self, got, out, tol):
        names = dict(dx=self.stream, dgain="fp32")
        if self.y is not None:
            names.update(dy=self.dtype, dy_gain="fp32")
        if self.gate is not None:
            names["dgate"] = self.dtype
        for k, name in names.items():
            R.near(got[k], out[k], tol[k], name, k)

    def close(self):
        self.z.zero_block_destroy(self.h)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(z, case):
    c = Case(z, case)
    xo, h = c.forward()
    x64, h64, tx, th = c.ref().forward()
    if c.y is not None:
        R.near(xo, x64, tx, c.stream, "x_out")
    if c.pre:
        R.near(h, h64, th, c.dtype, "h")
    assert z.zero_block_launch_count(c.h) == 1
    c.close()


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(z, case):
    c = Case(z, case, 1)
    got = c.backward(c.x)
    c.check(got, *c.ref().backward(c.x, c.dxo, c.dh if c.pre else None))
    if c.layout == "padded":           # what lies between the rows is left as it was
        buf = got["dx"]._base
        assert buf[:, c.D:].isnan().all()
    again = c.backward(c.x)            # equal bits
    import torch
    assert all(torch.equal(got[k], again[k]) for k in got)
    c.close()


PART = (300, 777, "bf16", "bf16", True, True, "plain", 0.1, 0.1, "own", 1.5, 0.5, True)


@pytest.mark.parametrize("layout", ["own", "padded"])
@pytest.mark.parametrize("without", ["dx_out", "dh", "dx", "dy", "gains", "one gain"])
def test_what_is_not_given_or_wanted(z, without, layout):
    """A gradient that is not given counts as zero; a result that is not wanted
    changes no other."""
    c = Case(z, PART[:9] + (layout,) + PART[10:], 2)
    dxo, dh = c.dxo, c.dh
    over = {}
    if without in ("dx_out", "dh"):
        over = {without: None}
        dxo, dh = (None, dh) if without == "dx_out" else (dxo, None)
    elif without == "gains":
        over = dict(dy_gain=None, dgain=None)
    elif without == "one gain":
        over = dict(dy_gain=None)
    else:
        over = {without: None}
    got = c.backward(c.x, **over)
    out, tol = c.ref().backward(c.x, dxo, dh)
    for k in over:
        if k in got and k not in ("dx_out", "dh"):
            assert (got[k] == 7.0).all()       # not written
    for k, name in dict(dx="bf16", dy="bf16", dgate="bf16", dy_gain="fp32", dgain="fp32").items():
        if without not in (k, "gains") and not (without == "one gain" and k == "dy_gain"):
            R.near(got[k], out[k], tol[k], name, k)
    c.close()


@pytest.mark.parametrize("layout", ["own", "padded"])
def test_gains_of_ones_and_x_out_alone(z, layout):
    import torch
    for pre in (True, False):
        c = Case(z, (100, 520, "fp16", "fp16", True, pre, "none", 0.0, 0.0, layout, 1.0, 1.0, True), 3)
        xo, h = c.like("fp16"), c.like("fp16")
        z.zero_block_join(c.h, c.x, c.y, xo, h if pre else None, None, None)
        c.y_gain = c.gain = None
        x64, h64, tx, th = c.ref().forward()
        R.near(xo, x64, tx, "fp16")
        if pre:
            R.near(h, h64, th, "fp16")
            h2 = c.like("fp16")
            z.zero_block_join(c.h, c.x, c.y, None, h2, None, None)      # h alone
            assert torch.equal(h, h2)
        c.close()


@pytest.mark.parametrize("D", [512, 517, 4096])
def test_in_place(z, D):
    """x' over x, h over y; dx over dx', dy over dh: the same bits."""
    import torch
    c = Case(z, (400, D, "bf16", "bf16", True, True, "sigmoid", 0.1, 0.1, "own", 1.0, 1.0, True), 4)
    xo, h = c.forward()
    x, y = c.x.clone(), c.y.clone()
    z.zero_block_join(c.h, x, y, x, y, c.y_gain, c.gain, **c.kw)
    assert torch.equal(x, xo) and torch.equal(y, h)
    want = c.backward(xo)
    dxo, dh, gate = c.dxo.clone(), c.dh.clone(), c.gate.clone()
    z.zero_block_join_backward(c.h, dxo, dh, xo, c.y, dxo, dh, None, None, c.y_gain, c.gain, dgate=gate,
                               **dict(c.kw, gate=gate))
    assert torch.equal(dxo, want["dx"]) and torch.equal(dh, want["dy"]) and torch.equal(gate, want["dgate"])
    c.close()


@pytest.mark.parametrize("D", [512, 517])
@pytest.mark.parametrize("fill", ["nan", "inf"])
def test_what_padding_holds_does_not_count(z, D, fill):
    import torch
    c = Case(z, (300, D, "fp16", "fp16", True, True, "plain", 0.1, 0.3, "own", 1.0, 1.0, True), 5)
    xo, h = c.forward()
    want = c.backward(c.x)
    for t in (c.x, c.y, c.gate, c.dxo, c.dh):
        t[~c.mask] = float(fill)
    xo2, h2 = c.forward()
    got = c.backward(c.x)
    assert torch.equal(xo, xo2) and torch.equal(h, h2)
    assert all(torch.equal(want[k], got[k]) for k in want)
    assert not xo2[~c.mask].any() and not h2[~c.mask].any() and not got["dx"][~c.mask].any()
    c.mask.fill_(False)                # a batch of nothing but padding
    xo, h = c.forward()
    got = c.backward(c.x)
    assert not any(t.any() for t in (xo, h, *got.values()))
    c.close()


def test_what_is_dropped_does_not_count(z):
    """A dropped number is zero, and so is its gradient, whatever it held."""
    import torch
    for D in (512, 517):
        c = Case(z, (200, D, "bf16", "bf16", False, False, "plain", 0.5, 0.0, "own", 1.0, 1.0, True), 6)
        keep = torch.from_numpy(R.kept(200, D, 0.5, *c.rng)).cuda()
        xo, _ = c.forward()
        got = c.backward(c.x)
        assert torch.equal(xo[~keep], c.x[~keep]) and not got["dy"][~keep].any() and not got["dgate"][~keep].any()
        c.y[~keep] = c.gate[~keep] = float("nan")
        assert torch.equal(c.forward()[0], xo)
        c.dxo[~keep] = float("inf")
        again = c.backward(c.x)
        assert all(torch.equal(again[k], got[k]) for k in ("dy", "dgate", "dy_gain"))
        c.close()


@pytest.mark.parametrize("D", [1, 3, 8, 13])
def test_a_row_of_which_all_is_dropped(z, D):
    """It is the stream's, though the branch's norm be NaN; also of rows that are not
    whole chunks."""
    import torch
    c = Case(z, (4000, D, "fp32", "fp32", True, True, "none", 0.6, 0.0, "own", 1.0, 1.0, True), 14)
    keep = torch.from_numpy(R.kept(4000, D, 0.6, *c.rng)).cuda()
    gone = ~keep.any(-1)
    assert gone.any()
    c.y[:, 0] = float("nan")
    xo, h = c.forward()
    assert torch.equal(xo[gone], c.x[gone]) and h[gone].isfinite().all()
    c.y.zero_()
    c.y[:, 0] = 1.0
    want = c.forward()
    assert torch.equal(want[1][gone], h[gone])
    c.close()


@pytest.mark.parametrize("D", [520, 521])
def test_in_place_on_a_binary32_stream(z, D):
    """As test_in_place, with results that change places with other inputs."""
    import torch
    c = Case(z, (333, D, "bf16", "fp32", True, True, "plain", 0.1, 0.1, "own", 1.0, 1.0, True), 15)
    xo, h = c.forward()
    want = c.backward(xo)
    x, gate = c.x.clone(), c.gate.clone()
    z.zero_block_join(c.h, x, c.y, x, gate, c.y_gain, c.gain, **dict(c.kw, gate=gate))
    assert torch.equal(x, xo) and torch.equal(gate, h)
    y, dh, xo2 = c.y.clone(), c.dh.clone(), xo.clone()       # dgate over dh, dy over y, dx over x'
    z.zero_block_join_backward(c.h, c.dxo, dh, xo2, y, xo2, y, None, None, c.y_gain, c.gain, dgate=dh, **c.kw)
    assert torch.equal(xo2, want["dx"]) and torch.equal(y, want["dy"]) and torch.equal(dh, want["dgate"])
    c.close()


def test_rows_of_zeros_and_of_extreme_sizes(z):
    """1e-17 to 1e17 in binary32 with eps 0 is exact in its scale; zero rows are
    normalised to zero."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(7)
    T, D = 36, 640
    base = torch.randn(1, D, device="cuda", generator=g)
    size = 2.0 ** torch.linspace(-56, 56, T, device="cuda").round()[:, None]
    y, x = base * size, torch.zeros(T, D, device="cuda")
    cfg = z.make_block_config(D, dtype=z.FP32, norm_branch=True, eps=0.0)
    h = z.zero_block_create(cfg)
    xo, out = torch.empty_like(x), torch.empty_like(x)
    z.zero_block_join(h, x, y, xo, out, None, None)
    # powers of two scale everything without rounding; rsqrt of an even power differs in nothing
    ref = base.double() / base.double().square().mean().sqrt()
    assert ((xo - ref).abs() <= (D + 32) * R.E32 * ref.abs()).all()
    dx, dy = torch.empty_like(x), torch.empty_like(x)
    d = torch.randn(1, D, device="cuda", generator=g).expand(T, D).contiguous()
    z.zero_block_join_backward(h, d, None, xo, y, dx, dy, None, None, None, None)
    b, u = base.double(), d[:1].double()
    r = b.square().mean().sqrt() ** -1
    want = r * (u - b * r * (u * b * r).mean())
    mag = r * (u.abs() + (b * r).abs() * (u * b * r).abs().mean())
    assert ((dy * size - want).abs() <= 2 * (D + 48) * R.E32 * mag).all()
    z.zero_block_destroy(h)
    c = Case(z, (5, 640, "fp32", "fp32", True, True, "none", 0.0, 0.0, "own", 1.0, 1.0, True), 8)
    c.x.zero_()
    c.y.zero_()
    xo, hh = c.forward()
    assert not xo.any() and not hh.any()
    got = c.backward(c.x)
    c.check(got, *c.ref().backward(c.x, c.dxo, c.dh))
    c.close()


def test_gradients_by_differences(z):
    """The derivative along a direction, by two forward calls a step 2e-3 apart:
    the difference's own error is the third derivative (below 60 for rows of
    order one) times step^2 / 6, and 2^-24 of the sum's terms over the step."""
    import torch
    for D in (96, 100):
        c = Case(z, (24, D, "fp32", "fp32", True, True, "sigmoid", 0.2, 0.2, "own", 1.3, 0.7, True), 9)
        g = torch.Generator(device="cuda").manual_seed(10)
        v = {k: torch.randn(getattr(c, k).shape, device="cuda", generator=g) for k in ("x", "y", "gate", "y_gain", "gain")}
        base = {k: getattr(c, k).clone() for k in v}

        def f(s):
            for k in v:
                getattr(c, k).copy_(base[k] + s * v[k])
            xo, h = c.forward()
            return (xo.double() * c.dxo.double() * c.mask[:, None]).sum() + (h.double() * c.dh.double() * c.mask[:, None]).sum()
        e = 1e-3
        num = (f(e) - f(-e)) / (2 * e)
        f(0.0)
        xo, _ = c.forward()
        got = c.backward(xo)
        an = sum((got[k].double() * v[n].double()).sum() for k, n in
                 (("dx", "x"), ("dy", "y"), ("dgate", "gate"), ("dy_gain", "y_gain"), ("dgain", "gain")))
        n = 24 * D
        bound = 60 * e * e / 6 * n + 8 * R.E32 * n ** 0.5 * 30 / e
        assert abs(num - an) <= bound, (num, an, bound)
        c.close()


def test_no_tokens(z):
    import torch
    h = z.zero_block_create(z.make_block_config(64, dtype=z.FP32, norm_branch=True))
    e, dg = torch.empty(0, 64, device="cuda"), torch.full((2, 64), 7.0, device="cuda")
    z.zero_block_join(h, e, e, e, e, None, None)
    z.zero_block_join_backward(h, e, e, e, e, e, e, dg[0], dg[1], None, None)
    assert not dg.any() and z.zero_block_launch_count(h) == 0
    z.zero_block_destroy(h)


@pytest.mark.parametrize("D", [1, 9, 64, 777, 4096])
def test_dropout(z, D):
    import torch
    for name in R.U:
        for T, p in ((1, 0.1), (33, 0.5), (300, 0.9), (5, 0.0), (5, 1.0)):
            g = torch.Generator(device="cuda").manual_seed(D)
            for layout in ("own", "odd", "padded"):
                x = rows(g, T, D, name, layout)
                out = blank(T, D, name, layout)
                z.zero_dropout(x, out, p, seed=2 ** 64 - 3, call=7, step=-2)
                keep = torch.from_numpy(R.kept(T, D, p, 2 ** 64 - 3, 7, -2)).cuda()
                ref = torch.where(keep, x.double() * R.factor(p), 0.0)
                R.near(out, ref, ref.abs() * 2 * R.E32, name)
                assert not out[~keep].any()
                z.zero_dropout(x, x, p, seed=2 ** 64 - 3, call=7, step=-2)        # in place
                assert torch.equal(x, out)


def test_dropout_shapes(z):
    """One dimension is one row; further ones are rows of the last."""
    import torch
    x = torch.randn(2, 3, 40, device="cuda")
    a, b, f = torch.empty_like(x), torch.empty(6, 40, device="cuda"), torch.empty(240, device="cuda")
    z.zero_dropout(x, a, 0.5, seed=1)
    z.zero_dropout(x.view(6, 40), b, 0.5, seed=1)
    assert torch.equal(a.view(6, 40), b)
    z.zero_dropout(x.view(240), f, 0.5, seed=1)      # 40 is whole blocks of eight
    assert torch.equal(f.view(6, 40), b)
    for shape in ((0, 40), (40, 0), (0,), ()):
        e = torch.ones(shape, device="cuda")
        z.zero_dropout(e, e, 0.5)
    for bad in (x[..., ::2], x.transpose(1, 2)):
        with pytest.raises(ValueError):
            z.zero_dropout(bad, torch.empty_like(bad), 0.5)
    with pytest.raises(ValueError):
        z.zero_dropout(x, a.half(), 0.5)
    with pytest.raises(ValueError):
        z.zero_dropout(x.cpu(), a.cpu(), 0.5)
    with pytest.raises(ValueError):
        z.zero_dropout(x, a, 0.5, step=torch.zeros(1, dtype=torch.int64))


def test_how_often_numbers_stay(z):
    """Of 2^24 numbers those kept are within five standard deviations of their
    share, over the eight places of a block and for neighbouring calls, steps and
    seeds, which agree as independent choices do."""
    import torch
    n, p = 2 ** 24, 0.3
    x, a, b = (torch.ones(n, device="cuda") for _ in range(3))
    q = 1 - R.cut_of(p) / 65536
    z.zero_dropout(x, a, p, seed=5, call=1, step=1)
    for i in range(8):
        k = (a[i::8] != 0).double().sum().item()
        assert abs(k - q * n / 8) <= 5 * (n / 8 * q * (1 - q)) ** 0.5
    same = q * q + (1 - q) ** 2
    for kw in (dict(seed=6, call=1, step=1), dict(seed=5, call=2, step=1), dict(seed=5, call=1, step=2)):
        z.zero_dropout(x, b, p, **kw)
        k = ((a != 0) == (b != 0)).double().sum().item()
        assert abs(k - same * n) <= 5 * (n * same * (1 - same)) ** 0.5


def test_graph_with_a_step_on_the_device(z):
    """A captured call drops by the step that the device holds when it is
    replayed; the join's two passes agree."""
    import torch
    c = Case(z, (300, 512, "bf16", "bf16", True, True, "none", 0.2, 0.0, "own", 1.0, 1.0, True), 11)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    c.kw["step"] = step
    drop = torch.empty_like(c.y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.forward(), c.backward(c.x)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xo, h = c.forward()
        got = c.backward(c.x)
        z.zero_dropout(c.y, drop, 0.2, seed=3, call=4, step=step)
    for v in (1, 2 ** 32 + 9, -1):
        step.fill_(v)
        graph.replay()
        torch.cuda.synchronize()
        c.rng = (c.rng[0], c.rng[1], v)
        r = c.ref()
        x64, h64, tx, th = r.forward()
        R.near(xo, x64, tx, "bf16")
        R.near(h, h64, th, "bf16")
        c.check(got, *r.backward(c.x, c.dxo, c.dh))
        keep = torch.from_numpy(R.kept(300, 512, 0.2, 3, 4, v)).cuda()
        assert torch.equal(drop != 0, keep & (c.y != 0))
    c.close()


def test_another_stream(z):
    import torch
    c = Case(z, (2000, 1024, "bf16", "bf16", True, True, "none", 0.1, 0.0, "own", 1.0, 1.0, True), 12)
    xo, h = c.forward()
    want = c.backward(c.x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        xo2, h2 = c.forward()
        got = c.backward(c.x)
    s.synchronize()
    assert torch.equal(xo, xo2) and torch.equal(h, h2) and all(torch.equal(want[k], got[k]) for k in want)
    c.close()


def test_strides_past_32_bits(z):
    """Two rows whose second begins 2^31 + 24 numbers behind the first (and an
    odd number more), of the join and of dropout."""
    import torch
    D = 520
    for far in (2 ** 31 + 24, 2 ** 31 + 25):
        buf = torch.empty(far + D, dtype=torch.bfloat16, device="cuda")
        t = buf.as_strided((2, D), (far, 1))
        c = Case(z, (2, D, "bf16", "bf16", True, True, "none", 0.1, 0.0, "own", 1.0, 1.0, True), 13)
        xo, h = c.forward()
        want = c.backward(c.x)
        t.copy_(c.x)
        h2 = torch.empty_like(h)
        z.zero_block_join(c.h, t, c.y, t, h2, c.y_gain, c.gain, **c.kw)
        assert torch.equal(t, xo) and torch.equal(h, h2)
        t.copy_(c.dxo)
        dy = torch.empty_like(h)
        z.zero_block_join_backward(c.h, t, c.dh, c.x, c.y, t, dy, None, None, c.y_gain, c.gain, **c.kw)
        assert torch.equal(t, want["dx"]) and torch.equal(dy, want["dy"])
        t.copy_(c.x)
        z.zero_dropout(t, t, 0.5, seed=9)
        keep = torch.from_numpy(R.kept(2, D, 0.5, 9)).cuda()
        assert torch.equal(t, torch.where(keep, c.x * 2, torch.zeros_like(c.x)))
        c.close()
        del t, buf
        torch.cuda.empty_cache()


def test_a_long_flat_dropout(z):
    """More than 2^32 numbers: the counter's second word, checked at both ends."""
    import torch
    n = 2 ** 35 + 2 ** 12 + 5      # blocks of eight past 2^32
    x = torch.ones(n, dtype=torch.float16, device="cuda")
    z.zero_dropout(x, x, 0.5, seed=11, call=3, step=4)
    for at in (0, 2 ** 31 - 2 ** 10, 2 ** 32, 2 ** 35 - 2 ** 10):
        keep = R.kept(2 ** 8, 8, 0.5, 11, 3, 4, first_row=at // 8)
        assert torch.equal((x[at:at + 2 ** 11] != 0).cpu(), torch.from_numpy(keep.reshape(-1)))
    tail = R.kept(1, n - n // 8 * 8, 0.5, 11, 3, 4, first_row=n // 8)
    assert torch.equal((x[n // 8 * 8:] != 0).cpu(), torch.from_numpy(tail.reshape(-1)))
