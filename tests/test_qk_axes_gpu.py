"""The query/key norm with a position on each of several axes, on the GPU.

It is the rotation by one position whose tables were gathered for each token
(row t of cos: cos[p[axis[j]][t]][j]), which the one-position kernels, tested
against 64 bits by themselves, give bit for bit (the gains' gradients are summed in
another order); and all against 64 bits with test_qk_gpu.py's tolerances.  Rotation alone rounds twice in binary32 (a product
and a fused sum of two terms): 2 2^-24 of the terms' magnitudes, and once to the
type.
"""
import pytest

from test_qk_gpu import U, backward64, code, dt, forward64, near, rotate, tables, z  # noqa: F401

pytestmark = pytest.mark.gpu

# tokens, q heads, k heads, D, sections, in turn, dtype, interleaved, gain per head, layout
CASES = [
    (1, 32, 8, 128, (16, 24, 24), False, "bf16", False, False, "fused"),
    (3, 1, 0, 2, (1,), False, "fp32", False, True, "own"),
    (37, 3, 1, 6, (1, 1, 1), False, "fp16", True, True, "own"),
    (300, 32, 8, 128, (16, 24, 24), False, "bf16", False, False, "fused"),
    (301, 12, 4, 64, (12, 10, 10), True, "fp16", False, False, "own"),
    (302, 12, 4, 64, (12, 10, 10), False, "bf16", True, True, "own"),
    (77, 5, 5, 80, (20, 20), False, "fp16", False, False, "odd"),
    (1000, 16, 16, 80, (20, 20), False, "bf16", False, False, "fused"),
    (90, 2, 1, 510, (60, 60, 4, 3), True, "bf16", False, False, "odd"),
    (91, 2, 1, 512, (64, 64, 64, 64), False, "fp32", True, True, "own"),
    (92, 2, 2, 96, (0, 18, 30), False, "fp32", False, False, "own"),
    (70, 3, 1, 128, (), False, "bf16", False, False, "own"),      # nothing turns
    (2500, 32, 8, 128, (5, 30, 29), True, "bf16", False, False, "own"),
]


class Case:
    def __init__(self, z, case, normalise=True, seed=0):  # noqa: F811
        import torch
        from zero_sharded_mixed_05_gb300.qk import axis_of_pairs
        (self.T, self.hq, self.hk, self.D, sections, turn, self.name, self.inter, self.per_head, layout) = case
        T, D = self.T, self.D
        g = torch.Generator(device="cuda").manual_seed(seed)

        def tensor(h):
            x = torch.randn(T, h, D, device="cuda", generator=g).to(dt(self.name))
            if layout == "odd":
                st = h * (D + 1) + 3
                flat = torch.zeros(T * st + 1, device="cuda", dtype=x.dtype)
                return flat[1:].as_strided((T, h, D), (st, D + 1, 1)).copy_(x)
            return x
        if layout == "fused":
            qkv = tensor(self.hq + 2 * self.hk)
            self.q, self.k = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hk]
        else:
            self.q, self.k = tensor(self.hq), tensor(self.hk)
        self.gq, self.gk = tensor(self.hq), tensor(self.hk)
        self.axis = axis_of_pairs(sections, turn)
        self.rot = 2 * len(self.axis)
        n_pos = 512
        self.cos, self.sin = tables(n_pos, self.rot)
        A = max(1, len(sections))
        self.pos = torch.randint(0, n_pos, (A, T), device="cuda", generator=g)
        if T > 2:                      # padding: a negative position on any one axis
            for a in range(A):
                self.pos[a, torch.rand(T, device="cuda", generator=g) < 0.07] = -1 - a
        lead = lambda h: (h, D) if self.per_head else (D,)  # noqa: E731
        self.qg = self.kg = None
        if normalise:
            self.qg = 1 + 0.3 * torch.randn(*lead(self.hq), device="cuda", generator=g)
            self.kg = 1 + 0.3 * torch.randn(*lead(self.hk), device="cuda", generator=g)
        # the same by one position: gathered tables
        ax = torch.tensor(self.axis, device="cuda", dtype=torch.int64)
        at = self.pos.clamp(min=0)[ax].T
        pair = torch.arange(len(self.axis), device="cuda")
        self.cos1, self.sin1 = self.cos[at, pair].contiguous(), self.sin[at, pair].contiguous()
        self.pos1 = torch.where((self.pos < 0).any(0), -1, torch.arange(T, device="cuda"))
        self.z = z
        cfg = z.make_qk_config(self.hq, self.hk, D, self.rot, code(z, self.name), self.inter, 1e-6, self.per_head)
        self.one = z.zero_qk_create(cfg)
        self.many = z.zero_qk_create(cfg, z.make_qk_axes(self.axis, axes=A, normalise=normalise))

    def outs(self):
        import torch
        return [torch.full((self.T, h, self.D), float("nan"), device="cuda", dtype=dt(self.name))
                for h in (self.hq, self.hk)]

    def forward(self, h, *where):
        o = self.outs()
        self.z.zero_qk_norm_rope(h, self.q, self.k, *o, self.qg, self.kg, *where)
        return o

    def backward(self, h, *where):
        import torch
        o, dg = self.outs(), [None if g is None else torch.full_like(g, float("nan")) for g in (self.qg, self.kg)]
        self.z.zero_qk_norm_rope_backward(h, self.gq, self.gk, self.q, self.k, *o, *dg, self.qg, self.kg, *where)
        return o + [g for g in dg if g is not None]

    def many_at(self, pos=None):
        return self.cos, self.sin, self.pos if pos is None else pos

    def close(self):
        self.z.zero_qk_destroy(self.one)
        self.z.zero_qk_destroy(self.many)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_gathered_tables_and_64_bits(z, case):  # noqa: F811
    import torch
    c = Case(z, case)
    for run in (c.forward, c.backward):
        want = run(c.one, c.cos1, c.sin1, c.pos1)
        for pos in (c.pos, c.pos.int()):
            got = run(c.many, *c.many_at(pos))
            assert all(torch.equal(a, b) for a, b in zip(got[:2], want))
            if c.hk:
                assert all(torch.equal(a, b) for a, b in zip(got, run(c.many, *c.many_at(pos))))
    fw, bw = c.forward(c.many, *c.many_at()), c.backward(c.many, *c.many_at())
    for i, (x, go, gain) in enumerate(((c.q, c.gq, c.qg), (c.k, c.gk, c.kg))):
        if x.shape[1]:
            ref = forward64(x, gain, c.pos1, c.cos1, c.sin1, c.rot, c.inter)
            near(fw[i], ref, ref.abs().amax(-1, keepdim=True), c.name, c.D)
            ref, mag, terms = backward64(go, x, gain, c.pos1, c.cos1, c.sin1, c.rot, c.inter)
            near(bw[i], ref, mag, c.name, c.D)
            dims = 0 if c.per_head else (0, 1)
            n = c.T if c.per_head else c.T * x.shape[1]
            scale = terms.abs().amax(-1, keepdim=True) if c.rot else terms.abs()
            tol = (n + c.D + 16) * 2.0 ** -24 * scale.expand_as(terms).sum(dims)
            assert ((bw[2 + i].double() - terms.sum(dims)).abs() <= tol).all()
    c.close()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotation_alone(z, case):  # noqa: F811
    """Forward, and backward from the gradients alone: NaN in q and k is not seen."""
    import torch
    c = Case(z, case, normalise=False, seed=1)

    def check(got, x, sign):
        ref = rotate(x.double(), c.pos1, c.cos1, c.sin1, c.rot, c.inter, sign)
        mag = rotate(x.double().abs(), c.pos1, c.cos1.abs(), c.sin1.abs(), c.rot, c.inter, 1.0).abs() \
            + rotate(x.double().abs(), c.pos1, c.cos1.abs(), c.sin1.abs(), c.rot, c.inter, -1.0).abs()
        tol = U[c.name] * ref.abs() + 3 * 2.0 ** -24 * mag + (2.0 ** -25 if c.name == "fp16" else 0)
        assert ((got.double() - ref).abs() <= tol).all()
    fw = c.forward(c.many, *c.many_at())
    c.q.fill_(float("nan"))
    bw = c.backward(c.many, *c.many_at())
    c2 = Case(z, case, normalise=False, seed=1)
    for got, back, x, go in ((fw[0], bw[0], c2.q, c2.gq), (fw[1], bw[1], c2.k, c2.gk)):
        if x.shape[1]:
            check(got, x, 1.0)
            check(back, go, -1.0)
    # in place, and rows of extreme size, which no norm bounds
    q, k = c2.q.clone(), c2.k.clone()
    z.zero_qk_norm_rope(c2.many, c2.q, c2.k, q, k, None, None, *c2.many_at())
    z.zero_qk_norm_rope(c2.many, c2.q, c2.k, c2.q, c2.k, None, None, *c2.many_at())
    assert torch.equal(q, c2.q) and torch.equal(k, c2.k)
    if c.name == "fp32":
        c2.gq.fill_(1e30)
        assert c2.backward(c2.many, *c2.many_at())[0].isfinite().all()
    c.close()
    c2.close()


def test_a_position_without_an_angle(z):  # noqa: F811
    """One axis at n_pos or far behind it: that token's rows, and the gains'
    gradients, are NaN; padding on another axis comes first."""
    import torch
    for big in (512, 2 ** 31 - 1, 2 ** 31 + 5, 2 ** 40):
        c = Case(z, (50, 4, 2, 64, (10, 10, 12), False, "bf16", False, False, "own"), seed=2)
        c.pos.clamp_(min=0)
        clean = c.forward(c.many, *c.many_at())
        c.pos[2, 7] = big
        c.pos[1, 8], c.pos[0, 8] = big, -1
        got = c.forward(c.many, *c.many_at())
        for a, b in zip(got, clean):
            assert a[7].isnan().all() and not a[8].any()
            keep = [i for i in range(50) if i not in (7, 8)]
            assert torch.equal(a[keep], b[keep])
        dq, dk, dqg, dkg = c.backward(c.many, *c.many_at())
        assert dq[7].isnan().all() and dqg.isnan().all() and dkg.isnan().all() and not dk[8].any()
        c.close()


def test_no_tokens_and_no_norm(z):  # noqa: F811
    import torch
    c = Case(z, (0, 4, 2, 64, (16, 16), False, "bf16", False, False, "own"), normalise=False)
    c.forward(c.many, *c.many_at())
    c.backward(c.many, *c.many_at())
    assert z.zero_qk_launch_count(c.many) == 0
    c.close()


def test_graph(z):  # noqa: F811
    """Captured calls read the positions that are there when they are replayed."""
    import torch
    c = Case(z, (300, 8, 4, 128, (16, 24, 24), False, "bf16", False, False, "own"), seed=3)
    c.forward(c.many, *c.many_at()), c.backward(c.many, *c.many_at())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fw, bw = c.forward(c.many, *c.many_at()), c.backward(c.many, *c.many_at())
    c.pos.copy_(c.pos.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    for got, want in zip(fw + bw, c.forward(c.many, *c.many_at()) + c.backward(c.many, *c.many_at())):
        assert torch.equal(got, want)
    c.close()


def test_autograd(z):  # noqa: F811
    """Through the wrapper, normalised and only rotated, against torch's autograd
    in 64 bits: (D + 40) 2^-24 of the largest terms, below 8, of 30 tokens x 4
    heads for the gains."""
    import torch
    from zero_sharded_mixed_05_gb300.qk import QkNormRope, axis_of_pairs, make_qk_axes, rotation_tables
    g = torch.Generator(device="cuda").manual_seed(4)
    T, hq, hk, D = 30, 4, 2, 64
    axis = axis_of_pairs((8, 12, 12), alternate=True)
    cos, sin = rotation_tables(40, D, axis=axis)
    pos = torch.randint(0, 40, (3, T), device="cuda", generator=g)
    pos[:, 5] = -1
    live = (pos >= 0).all(0)
    ax, pair = torch.tensor(axis, device="cuda"), torch.arange(32, device="cuda")
    c, s = (t.double()[pos.clamp(min=0)[ax].T, pair][:, None] for t in (cos, sin))
    w = [torch.randn(T, h, D, device="cuda", generator=g) for h in (hq, hk)]
    for normalise in (True, False):
        norm = QkNormRope(z.make_qk_config(hq, hk, D, dtype=z.FP32), make_qk_axes(axis, normalise=normalise))
        leaves = [torch.randn(T, h, D, device="cuda", generator=g) for h in (hq, hk)]
        if normalise:
            leaves += [1 + 0.1 * torch.randn(D, device="cuda", generator=g) for _ in range(2)]
        got, ref = [t.clone().requires_grad_() for t in leaves], [t.double().requires_grad_() for t in leaves]
        qo, ko = norm(*got[:2], *(got[2:] or (None, None)), cos, sin, pos)
        ((qo * w[0]).sum() + (ko * w[1]).sum()).backward()
        loss = 0.0
        for i in range(2):
            y = ref[i]
            if normalise:
                y = y * (y.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * ref[2 + i]
            u, v = y[..., :32], y[..., 32:]
            loss = loss + (torch.cat((u * c - v * s, v * c + u * s), -1) * w[i] * live[:, None, None]).sum()
        loss.backward()
        for a, b in zip(got, ref):
            terms = 1 if a.dim() == 3 else T * hq
            assert ((a.grad.double() - b.grad).abs() <= (D + 40) * 2.0 ** -24 * 8 * terms).all()
        norm.close()
