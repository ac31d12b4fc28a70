"""The query/key norm with rotation on the GPU against the formulas in 64 bits.

Tolerances.  A result is computed in binary32 and rounded once to the data's
type: half a unit in the last place of the type (u = 2^-11 fp16, 2^-8 bf16,
2^-24 fp32, and fp16's subnormal spacing 2^-25), plus the binary32 arithmetic.
That is below (D + 16) 2^-24 of the largest terms of the row for a sum of D
squares in any order; the gains' gradients add at most T * heads terms, each
with an error below 16 * 2^-24, in some order: (T * heads + 16) 2^-24 of the
sum of their magnitudes.
"""
import pytest

pytestmark = pytest.mark.gpu

U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
EPS = 1e-6


@pytest.fixture(scope="module")
def z():
    import zero_sharded_mixed_05_gb300 as z
    z.lib()
    return z


def dt(name):
    import torch
    return dict(fp16=torch.float16, bf16=torch.bfloat16, fp32=torch.float32)[name]


def code(z, name):
    return dict(fp16=z.FP16, bf16=z.BF16, fp32=z.FP32)[name]


def tables(n_pos, rot, dev="cuda"):
    import torch
    f = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(n_pos, device=dev, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def rotate(x, pos, cos, sin, rot, inter, sign):
    import torch
    live = pos >= 0
    at = pos.clamp(min=0).long()
    c, s = cos.double()[at][:, None], sign * sin.double()[at][:, None]
    y = x.clone()
    if rot:
        u, v = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2],
                                                                 x[..., rot // 2:rot])
        a, b = u * c - v * s, v * c + u * s
        if inter:
            y[..., 0:rot:2], y[..., 1:rot:2] = a, b
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = a, b
    return torch.where(live[:, None, None], y, torch.zeros_like(y))


def forward64(x, gain, pos, cos, sin, rot, inter):
    x = x.double()
    r = (x.square().mean(-1, keepdim=True) + EPS) ** -0.5
    return rotate(x * r * gain.double(), pos, cos, sin, rot, inter, 1.0)


def backward64(go, x, gain, pos, cos, sin, rot, inter):
    """(dx, magnitude of dx's terms, dgain terms [T, H, D])"""
    import torch
    x, dy = x.double(), rotate(go.double(), pos, cos, sin, rot, inter, -1.0)
    r = (x.square().mean(-1, keepdim=True) + EPS) ** -0.5
    dn = dy * gain.double()
    m = (dn * x).mean(-1, keepdim=True)
    dx = r * dn - x * r ** 3 * m
    mag = r * dn.abs().amax(-1, keepdim=True) + \
        x.abs().amax(-1, keepdim=True) * r ** 3 * (dn * x).abs().mean(-1, keepdim=True)
    live = (pos >= 0)[:, None, None]
    terms = torch.where(live, dy * x * r, torch.zeros_like(dy))
    return torch.where(live, dx, torch.zeros_like(dx)), mag, terms


def near(got, ref, mag, name, dim):
    tol = U[name] * ref.abs() + (dim + 16) * 2.0 ** -24 * mag
    if name == "fp16":
        tol = tol + 2.0 ** -25
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), ((got.double() - ref).abs() / tol).max()


# tokens, q heads, k heads, D, rotary_dim, dtype, interleaved, gain per head, layout
CASES = [
    (1, 32, 8, 128, 128, "bf16", False, False, "fused"),
    (1, 1, 0, 2, 2, "fp32", False, True, "own"),
    (2, 3, 1, 6, 2, "fp16", True, True, "own"),
    (3, 4, 2, 64, 64, "fp16", True, False, "fused"),
    (17, 12, 12, 80, 40, "fp16", True, True, "fused"),
    (17, 12, 12, 80, 40, "bf16", False, False, "odd"),
    (33, 5, 3, 96, 96, "bf16", False, True, "own"),
    (40, 2, 2, 512, 512, "fp16", False, True, "own"),
    (29, 2, 1, 510, 254, "bf16", False, False, "odd"),
    (64, 6, 2, 256, 128, "fp32", True, False, "own"),
    (65, 300, 2, 8, 8, "bf16", False, True, "own"),
    (70, 3, 1, 128, 0, "bf16", False, False, "own"),
    (257, 8, 4, 128, 128, "bf16", False, True, "heads_first"),
    (600, 32, 8, 64, 64, "fp16", False, False, "fused"),
    (300, 32, 8, 128, 128, "bf16", False, True, "fused"),     # heads spread over two CTAs
    (90, 33, 0, 128, 64, "fp16", True, True, "own"),
]


def make(case, seed=0, big=1.0):
    import torch
    T, hq, hk, D, rot, name, inter, per_head, layout = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, device="cuda", generator=g) * big

    def tensor(h):
        if layout == "heads_first":
            return rand(h, T, D).to(dt(name)).transpose(0, 1)
        if layout == "odd":      # an odd base address and odd strides
            flat = rand(T * (h * (D + 1) + 3) + 1).to(dt(name))
            return flat[1:].as_strided((T, h, D), (h * (D + 1) + 3, D + 1, 1))
        return rand(T, h, D).to(dt(name))

    if layout == "fused":
        qkv = rand(T, hq + 2 * hk, D).to(dt(name))
        q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    else:
        q, k = tensor(hq), tensor(hk)
    n_pos = 1024
    cos, sin = tables(n_pos, rot)
    pos = torch.randint(0, n_pos, (T,), device="cuda", generator=g)
    if T > 2:
        pos[torch.rand(T, device="cuda", generator=g) < 0.2] = -1
        pos[0], pos[1] = 0, n_pos - 1
    lead = lambda h: (h, D) if per_head else (D,)  # noqa: E731
    qg = 1 + 0.3 * torch.randn(*lead(hq), device="cuda", generator=g)
    kg = 1 + 0.3 * torch.randn(*lead(hk), device="cuda", generator=g)
    return q, k, qg, kg, cos, sin, pos


def handle(z, case):
    T, hq, hk, D, rot, name, inter, per_head, _ = case
    return z.zero_qk_create(z.make_qk_config(hq, hk, D, rot, code(z, name), inter, EPS, per_head))


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("pos32", [False, True])
def test_forward(z, case, pos32):
    import torch
    T, hq, hk, D, rot, name, inter, per_head, _ = case
    q, k, qg, kg, cos, sin, pos = make(case, 1)
    h = handle(z, case)
    try:
        qo = torch.full((T, hq, D), float("nan"), device="cuda", dtype=dt(name))
        ko = torch.full((T, hk, D), float("nan"), device="cuda", dtype=dt(name))
        before = (q.clone(), k.clone())
        z.zero_qk_norm_rope(h, q, k, qo, ko, qg, kg, cos, sin, pos.int() if pos32 else pos)
        assert torch.equal(q, before[0]) and torch.equal(k, before[1])
        for got, x, gain in ((qo, q, qg), (ko, k, kg)):
            if x.shape[1] == 0:
                continue
            ref = forward64(x, gain, pos, cos, sin, rot, inter)
            near(got, ref, ref.abs().amax(-1, keepdim=True), name, D)
        # in place gives the bits of another output of the same layout (the
        # width of the loads, and with it the order of a sum, goes by layout)
        qi, ki = make(case, 1)[:2]
        ql, kl = make(case, 4)[:2]
        z.zero_qk_norm_rope(h, q, k, ql, kl, qg, kg, cos, sin, pos)
        z.zero_qk_norm_rope(h, qi, ki, qi, ki, qg, kg, cos, sin, pos)
        assert torch.equal(qi, ql) and torch.equal(ki, kl)
    finally:
        z.zero_qk_destroy(h)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(z, case):
    import torch
    T, hq, hk, D, rot, name, inter, per_head, _ = case
    q, k, qg, kg, cos, sin, pos = make(case, 2)
    gq, gk = make(case, 3)[:2]
    h = handle(z, case)
    try:
        dq = torch.full((T, hq, D), float("nan"), device="cuda", dtype=dt(name))
        dk = torch.full((T, hk, D), float("nan"), device="cuda", dtype=dt(name))
        dqg, dkg = torch.full_like(qg, float("nan")), torch.full_like(kg, float("nan"))
        args = (qg, kg, cos, sin, pos)
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, dq, dk, dqg, dkg, *args)
        for got, dg, go, x, gain in ((dq, dqg, gq, q, qg), (dk, dkg, gk, k, kg)):
            if x.shape[1] == 0:
                continue
            ref, mag, terms = backward64(go, x, gain, pos, cos, sin, rot, inter)
            near(got, ref, mag, name, D)
            dims = 0 if per_head else (0, 1)
            n = T if per_head else T * x.shape[1]
            # a term's own error is relative to the pair that was turned back
            scale = terms.abs().amax(-1, keepdim=True) if rot else terms.abs()
            tol = (n + D + 16) * 2.0 ** -24 * scale.expand_as(terms).sum(dims)
            bad = (dg.double() - terms.sum(dims)).abs() > tol
            assert not bad.any()
        # the same bits again, and without the gains' gradients, and in place
        again = [torch.empty_like(t) for t in (dq, dk, dqg, dkg)]
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, *again, *args)
        for a, b in zip(again, (dq, dk, dqg, dkg)):
            assert torch.equal(a, b)
        iq, ik = make(case, 3)[:2]
        lq, lk = make(case, 4)[:2]
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, lq, lk, None, None, *args)
        z.zero_qk_norm_rope_backward(h, iq, ik, q, k, iq, ik, None, None, *args)
        assert torch.equal(iq, lq) and torch.equal(ik, lk)
    finally:
        z.zero_qk_destroy(h)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
def test_gradient_against_differences(z, inter, per_head):
    """Directional derivatives of L = sum w * out by central differences of
    the binary32 forward call.  With step e and inputs of size one, the
    difference quotient's error is below e^2 |L'''| / 6 (of the order of e^2
    times the sum of |w|) plus the results' rounding 2^-22 sum |w| / e; both
    sums are over N numbers of random sign, so their square root counts, times
    six for certainty."""
    import torch
    case = (12, 3, 2, 16, 8, "fp32", inter, per_head, "own")
    T, hq, hk, D = case[:4]
    q, k, qg, kg, cos, sin, pos = make(case, 5)
    wq, wk = make(case, 6)[:2]
    h = handle(z, case)
    try:
        def loss(q, k, qg, kg):
            qo, ko = torch.empty_like(q), torch.empty_like(k)
            z.zero_qk_norm_rope(h, q, k, qo, ko, qg, kg, cos, sin, pos)
            return float((qo.double() * wq).sum() + (ko.double() * wk).sum())
        grads = [torch.empty_like(t) for t in (q, k, qg, kg)]
        z.zero_qk_norm_rope_backward(h, wq, wk, q, k, *grads, qg, kg, cos, sin, pos)
        e = 2.0 ** -8
        n = (q.numel() + k.numel()) ** 0.5
        tol = 6 * n * (e * e + 2.0 ** -22 / e)
        at = [q, k, qg, kg]
        g = torch.Generator(device="cuda").manual_seed(9)
        for i, d in enumerate(grads):
            v = torch.randn(d.shape, device="cuda", generator=g)
            hi, lo = list(at), list(at)
            hi[i], lo[i] = at[i] + e * v, at[i] - e * v
            num = (loss(*hi) - loss(*lo)) / (2 * e)
            assert abs(num - float((d.double() * v).sum())) <= tol, i
    finally:
        z.zero_qk_destroy(h)


def test_padding_reads_nothing_and_unknown_positions_are_nan(z):
    import torch
    case = (5, 2, 1, 64, 64, "bf16", False, False, "own")
    q, k, qg, kg, cos, sin, pos = make(case, 7)
    pos[:] = torch.tensor([3, -1, 1024, -7, 5], device="cuda")
    q[1], k[1] = float("nan"), float("inf")     # what a padding slot may hold
    q[3], k[3] = float("inf"), float("nan")
    gq, gk = q.clone(), k.clone()
    h = handle(z, case)
    try:
        outs = [torch.ones_like(t) for t in (q, k, q, k)]
        dqg, dkg = torch.empty_like(qg), torch.empty_like(kg)
        z.zero_qk_norm_rope(h, q, k, outs[0], outs[1], qg, kg, cos, sin, pos)
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, outs[2], outs[3], dqg, dkg, qg, kg, cos, sin,
                                     pos)
        for t in outs:
            assert (t[1] == 0).all() and (t[3] == 0).all()
            assert t[2].isnan().all()
            assert t[0].isfinite().all() and t[4].isfinite().all()
        pos[2] = -1
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, outs[2], outs[3], dqg, dkg, qg, kg, cos, sin,
                                     pos)
        assert dqg.isfinite().all() and dkg.isfinite().all()
        pos[:] = -1
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, outs[2], outs[3], dqg, dkg, qg, kg, cos, sin,
                                     pos)
        assert (dqg == 0).all() and (dkg == 0).all() and (outs[2] == 0).all()
    finally:
        z.zero_qk_destroy(h)


def test_zero_rows_zero_tokens_and_no_gain(z):
    import torch
    case = (4, 2, 2, 32, 32, "fp16", False, False, "own")
    q, k, qg, kg, cos, sin, pos = make(case, 8)
    q[0] = 0
    h = handle(z, case)
    try:
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        z.zero_qk_norm_rope(h, q, k, qo, ko, None, None, cos, sin, pos)
        ones = torch.ones_like(qg)
        q1, k1 = torch.empty_like(q), torch.empty_like(k)
        z.zero_qk_norm_rope(h, q, k, q1, k1, ones, ones, cos, sin, pos)
        assert torch.equal(qo, q1) and torch.equal(ko, k1) and (qo[0] == 0).all()
        n = z.zero_qk_launch_count(h)
        e = q[:0]
        dqg, dkg = torch.ones_like(qg), torch.ones_like(kg)
        z.zero_qk_norm_rope(h, e, e, e, e, qg, kg, cos, sin, pos[:0])
        z.zero_qk_norm_rope_backward(h, e, e, e, e, e, e, dqg, dkg, qg, kg, cos, sin, pos[:0])
        assert (dqg == 0).all() and (dkg == 0).all() and z.zero_qk_launch_count(h) == n
    finally:
        z.zero_qk_destroy(h)


def test_another_stream_and_a_graph(z):
    import torch
    case = (50, 4, 2, 64, 64, "bf16", False, False, "fused")
    q, k, qg, kg, cos, sin, pos = make(case, 10)
    gq, gk = make(case, 11)[:2]
    h = handle(z, case)
    try:
        def outs():
            return [torch.empty(50, 4, 64, device="cuda", dtype=q.dtype),
                    torch.empty(50, 2, 64, device="cuda", dtype=q.dtype),
                    torch.empty_like(qg), torch.empty_like(kg)]

        def both(a, b):
            z.zero_qk_norm_rope(h, q, k, a[0], a[1], qg, kg, cos, sin, pos)
            z.zero_qk_norm_rope_backward(h, gq, gk, q, k, *b, qg, kg, cos, sin, pos)
        a, b = outs(), outs()
        both(a, b)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        c, d = outs(), outs()
        with torch.cuda.stream(s):
            both(c, d)
        s.synchronize()
        e, f = outs(), outs()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both(e, f)
        graph.replay()
        torch.cuda.synchronize()
        for x, y, w in zip(a[:2] + b, c[:2] + d, e[:2] + f):
            assert torch.equal(x, y) and torch.equal(x, w)
    finally:
        z.zero_qk_destroy(h)


def test_binding_refuses(z):
    import torch
    case = (4, 2, 1, 32, 32, "fp16", False, False, "own")
    q, k, qg, kg, cos, sin, pos = make(case, 12)
    h = handle(z, case)
    try:
        good = dict(q=q, k=k, q_out=q.clone(), k_out=k.clone(), q_gain=qg, k_gain=kg, cos=cos,
                    sin=sin, positions=pos)
        z.zero_qk_norm_rope(h, **good)
        for name, bad in [("q", q.float()), ("q", q.cpu()), ("k", k[:3]), ("q_out", q[:, :1]),
                          ("q_out", q.transpose(1, 2).contiguous().transpose(1, 2)),
                          ("q_gain", qg.half()), ("k_gain", kg[:16]), ("cos", cos[:, :8]),
                          ("sin", sin[:5]), ("cos", cos.double()), ("positions", pos.float()),
                          ("positions", pos[:2])]:
            with pytest.raises(ValueError):
                z.zero_qk_norm_rope(h, **{**good, name: bad})
        with pytest.raises(ValueError):
            z.zero_qk_norm_rope(h + 8, **good)
    finally:
        z.zero_qk_destroy(h)
