"""The orthogonalised update on the GPU against its definition in 64 bits.

Tolerance of O.  The products' operands are rounded to binary16 (relative
2^-12 at most, 2^-12/sqrt(3) in the mean) in A, in b A + c A A and in X, five
times over; a rounding of a step reaches the result multiplied by the later
steps' slope, which is below one near the singular values where most end.
Three roundings a step, five steps, added as squares: sqrt(15) 2^-12/sqrt(3) =
5.5e-4, times the largest factor that a matrix enters a product with,
|b| + 2 |c| = 8.8 in X <- a X + (b A + c A A) X against results of size one,
gives 4.8e-3 as the bound of the Frobenius norm; the result's type adds its
own rounding, u.
"""
import pytest

pytestmark = pytest.mark.gpu

ABC = (3.4445, -4.7750, 2.0315)
TOL = 4.8e-3
U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


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


def ortho64(g, eps=1e-7, coefs=(ABC,) * 5):
    import torch
    x = g.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    for a, b, c in coefs:
        A = x @ x.mT
        x = a * x + (b * A + c * A @ A) @ x
    x = x.mT if tall else x
    return x.contiguous() if isinstance(x, torch.Tensor) else x


def spectrum(kind, b, m, n, gen, dev="cuda"):
    import torch

    def rand(*s):
        return torch.randn(*s, device=dev, generator=gen)
    if kind == "gauss":
        return rand(b, m, n)
    k = min(m, n)
    if kind == "signal":          # a few directions that fall off, over noise
        r = max(1, k // 4)
        s = 1.0 / torch.arange(1, r + 1, device=dev)
        return (rand(b, m, r) * s) @ rand(b, r, n) + 0.1 * rand(b, m, n)
    if kind == "rank1":
        return rand(b, m, 1) @ rand(b, 1, n)
    if kind == "decay":           # singular values over six powers of ten
        u = torch.linalg.qr(rand(b, m, k))[0]
        v = torch.linalg.qr(rand(b, n, k))[0]
        s = 10.0 ** (-6.0 * torch.arange(k, device=dev) / k)
        return (u * s) @ v.mT
    raise ValueError(kind)


def close(got, ref, name, what=""):
    """Per matrix, in the Frobenius norm."""
    d = (got.double() - ref).flatten(-2).norm(dim=-1)
    lim = (TOL + U[name]) * ref.flatten(-2).norm(dim=-1)
    assert (d <= lim).all(), (what, (d / lim).max())


SHAPES = [(1, 1, 1), (1, 7, 3), (7, 1, 2), (2, 3, 5), (15, 17, 2), (17, 15, 1), (64, 64, 1),
          (63, 65, 4), (100, 300, 2), (300, 100, 1), (128, 128, 3), (129, 257, 1), (256, 256, 2),
          (257, 129, 2), (255, 511, 1), (511, 255, 1), (640, 130, 1), (384, 520, 1), (16, 2000, 2),
          (2000, 16, 1), (1000, 777, 1), (520, 1300, 1), (80, 4200, 2), (5000, 300, 1),
          (257, 6000, 1), (3000, 1, 2), (1025, 1025, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind,src,dst", [("gauss", "bf16", "bf16"), ("signal", "fp32", "fp16"),
                                          ("rank1", "fp16", "fp32"), ("decay", "fp32", "fp32")])
def test_orthogonalize(z, shape, kind, src, dst):
    import torch
    m, n, b = shape
    g = spectrum(kind, b, m, n, torch.Generator(device="cuda").manual_seed(m * n)).to(dt(src))
    h = z.zero_muon_create(z.make_muon_config(), [(m, n, b)])
    try:
        out = torch.full((b, m, n), float("nan"), device="cuda", dtype=dt(dst))
        before = g.clone()
        z.zero_muon_orthogonalize(h, [g], [out])
        assert torch.equal(g, before)
        close(out, ortho64(g), dst)
        again = torch.empty_like(out)
        z.zero_muon_orthogonalize(h, [g], [again])
        assert torch.equal(out, again)
        info = z.zero_muon_last_step(h)
        assert (info.skipped, info.fault) == (0, 0)
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("shape", [(60, 500, 2), (128, 1000, 3), (513, 90, 2), (128, 2048, 2), (1801, 77, 20),
                                   (100, 100, 200), (5, 128, 400)], ids=str)
@pytest.mark.parametrize("kind,src,dst", [("signal", "bf16", "fp32"), ("decay", "fp32", "bf16")])
def test_on_the_chip(z, shape, kind, src, dst):
    """Clusters of two, four and eight CTAs, and more matrices than SMs; with
    one CTA a matrix the same bits for it on its own and among others."""
    import torch
    m, n, b = shape
    g = spectrum(kind, b, m, n, torch.Generator(device="cuda").manual_seed(m + n)).to(dt(src))
    one, many = z.zero_muon_create(z.make_muon_config(), [(m, n)]), z.zero_muon_create(z.make_muon_config(), [shape])
    try:
        out = torch.full((b, m, n), float("nan"), device="cuda", dtype=dt(dst))
        z.zero_muon_orthogonalize(many, [g], [out])
        close(out, ortho64(g), dst)
        alone = torch.empty_like(out[0])
        z.zero_muon_orthogonalize(one, [g[b - 1]], [alone])
        close(alone[None], ortho64(g[b - 1:]), dst)
        if max(m, n) <= 128:
            assert torch.equal(alone, out[b - 1])
    finally:
        z.zero_muon_destroy(one)
        z.zero_muon_destroy(many)


@pytest.mark.parametrize("shape", [(300, 1030, 2), (1030, 300, 1), (257, 257, 3), (90, 4300, 1)], ids=str)
@pytest.mark.parametrize("param,master", [("bf16", True), ("fp16", False)])
def test_step_through_the_workspace(z, shape, param, master):
    """Result blocks that end inside a tile, with and without binary32 masters."""
    import torch
    mats = matrices([shape], "bf16", 21)
    for x in mats:
        x["param16"] = x["param16"].to(dt(param))
        if not master:
            x["master"] = None
    h = z.zero_muon_create(z.make_muon_config(grad_dtype=z.BF16, param_dtype=code(z, param), lr=1e-2, momentum=0.9,
                                              weight_decay=0.1, scale_rule=1), [shape])
    try:
        mom, tol_m, w, tol_w = expected(z, mats[0], 1.0, 1e-2, 0.9, 0.1, True, 1)
        z.zero_muon_step(h, z.make_muon_list(mats))
        got = mats[0]["param16"].double()
        assert ((mats[0]["momentum"].double() - mom).abs() <= tol_m).all()
        tol_w = tol_w + U[param] * w.flatten(-2).norm(dim=-1)      # one rounding to 16 bits
        assert ((got - w).flatten(-2).norm(dim=-1) <= tol_w).all()
        if master:
            assert torch.equal(mats[0]["param16"], mats[0]["master"].to(dt(param)))
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("scale", [1e-6, 1e-3, 1e4])
def test_scale_of_the_input(z, scale):
    """|G| far from one, and against the eps that is added to it."""
    import torch
    g = spectrum("gauss", 1, 96, 160, torch.Generator(device="cuda").manual_seed(1))[0] * scale
    for eps in (1e-7, 0.0):
        h = z.zero_muon_create(z.make_muon_config(eps=eps), [(96, 160)])
        out = torch.empty_like(g)
        z.zero_muon_orthogonalize(h, [g], [out])
        close(out, ortho64(g, eps), "fp32")
        z.zero_muon_destroy(h)


def test_many_shapes_one_call_strides_and_in_place(z):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    shapes = [(40, 100, 3), (300, 257, 1), (100, 40, 2), (1, 1, 1), (513, 300, 2), (64, 1000, 1)]
    ins, outs, refs = [], [], []
    for i, (m, n, b) in enumerate(shapes):
        wide = torch.randn(b, m + 1, n + 5 + i, device="cuda", generator=gen).to(torch.bfloat16)
        ins.append(wide[:, 1:, i:i + n])                 # rows with gaps, at odd addresses
        store = torch.full((b, m, n + 3), 7.0, device="cuda", dtype=torch.bfloat16)
        outs.append(store[:, :, 1:n + 1])
        refs.append(ortho64(ins[-1]))
    h = z.zero_muon_create(z.make_muon_config(), shapes)
    try:
        z.zero_muon_orthogonalize(h, ins, outs)
        for x, o, r in zip(ins, outs, refs):
            close(o, r, "bf16", o.shape)
            edge = o._base
            assert (edge[:, :, 0] == 7).all() and (edge[:, :, -2:] == 7).all()
        z.zero_muon_orthogonalize(h, ins, ins)
        for x, o in zip(ins, outs):
            assert torch.equal(x, o)
        # each matrix's result does not depend on its company
        for i, s in enumerate(shapes):
            h1 = z.zero_muon_create(z.make_muon_config(), [s])
            one = [torch.empty(s[2], s[0], s[1], device="cuda", dtype=torch.bfloat16)]
            z.zero_muon_orthogonalize(h1, [refs[i].to(torch.bfloat16)], one)
            close(one[0], ortho64(refs[i].to(torch.bfloat16)), "bf16")
            z.zero_muon_destroy(h1)
    finally:
        z.zero_muon_destroy(h)


def test_zero_and_bad_matrices_of_a_batch(z):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(6)
    g = torch.randn(4, 70, 50, device="cuda", generator=gen)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    h = z.zero_muon_create(z.make_muon_config(), [(70, 50, 4)])
    try:
        out = torch.empty_like(g)
        z.zero_muon_orthogonalize(h, [g], [out])
        assert (out[1] == 0).all() and out[2].isnan().all()
        close(out[[0, 3]], ortho64(g[[0, 3]]), "fp32")
        g[2] = 1.0                                     # the workspace holds no NaN over
        z.zero_muon_orthogonalize(h, [g], [out])
        close(out[[0, 2, 3]], ortho64(g[[0, 2, 3]]), "fp32")
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("steps", [1, 2, 3, 6])
def test_steps_and_coefficients(z, steps):
    """Other numbers of steps, with a triple of their own each."""
    import torch
    coefs = [(1.5 + 0.3 * i, -0.5 - 0.1 * i, 0.05 * i) for i in range(steps)]
    g = spectrum("gauss", 2, 130, 200, torch.Generator(device="cuda").manual_seed(steps))
    h = z.zero_muon_create(z.make_muon_config(steps=steps, coefs=coefs), [(130, 200, 2)])
    out = torch.empty_like(g)
    z.zero_muon_orthogonalize(h, [g], [out])
    close(out, ortho64(g, coefs=coefs), "fp32")
    z.zero_muon_destroy(h)


def matrices(shapes, grad, seed, scale=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for m, n, b in shapes:
        g = spectrum("signal", b, m, n, gen) * 1e-3
        mom = spectrum("signal", b, m, n, gen) * 5e-3
        w = torch.randn(b, m, n, device="cuda", generator=gen) * 0.02
        out.append(dict(grad=(g * scale).to(dt(grad)), momentum=mom, master=w,
                        param16=w.to(dt(grad))))
    return out


def rule(z, scale_rule, m, n):
    return {z.MUON_SCALE_ONE: 1.0, z.MUON_SCALE_RMS: 0.2 * max(m, n) ** 0.5,
            z.MUON_SCALE_ASPECT: max(1.0, m / n) ** 0.5}[scale_rule]


def expected(z, m, f, lr, mu, wd, nesterov, scale_rule):
    """(momentum, its tolerance, master, its Frobenius tolerance) after a step."""
    g = m["grad"].double() * f
    mom = mu * m["momentum"].double() + g
    tol_m = 3 * 2.0 ** -24 * ((mu * m["momentum"].double()).abs() + g.abs())
    o = ortho64(g + mu * mom if nesterov else mom)
    s = rule(z, scale_rule, *o.shape[-2:])
    w0 = (m["master"] if m["master"] is not None else m["param16"]).double()
    w = w0 * (1 - lr * wd) - lr * s * o
    tol_w = TOL * lr * s * o.flatten(-2).norm(dim=-1) + 3 * 2.0 ** -24 * w0.flatten(-2).norm(dim=-1)
    return mom, tol_m, w, tol_w


@pytest.mark.parametrize("grad,param,nesterov,scale_rule", [
    ("bf16", "bf16", True, 1), ("fp16", "bf16", False, 2), ("fp16", "fp16", True, 0)])
def test_step(z, grad, param, nesterov, scale_rule):
    import torch
    shapes = [(64, 64, 2), (100, 300, 1), (257, 90, 2), (33, 1, 1), (320, 256, 1)]
    lr, mu, wd, scale = 1e-2, 0.9, 0.1, 512.0
    mats = matrices(shapes, grad, 11, scale)
    for m in mats:
        m["param16"] = m["param16"].to(dt(param))
    cfg = z.make_muon_config(grad_dtype=code(z, grad), param_dtype=code(z, param), lr=lr,
                             momentum=mu, nesterov=nesterov, weight_decay=wd,
                             scale_rule=scale_rule)
    h = z.zero_muon_create(cfg, shapes)
    try:
        lst = z.make_muon_list(mats)
        for step in range(3):
            want = [expected(z, m, 1 / scale, lr, mu, wd, nesterov, scale_rule) for m in mats]
            grads = [m["grad"].clone() for m in mats]
            z.zero_muon_step(h, lst, grad_scale=1 / scale)
            for m, g, (mom, tol_m, w, tol_w) in zip(mats, grads, want):
                assert torch.equal(m["grad"], g)
                assert ((m["momentum"].double() - mom).abs() <= tol_m).all()
                assert ((m["master"].double() - w).flatten(-2).norm(dim=-1) <= tol_w).all()
                assert torch.equal(m["param16"], m["master"].to(dt(param)))
            lr /= 2
            z.zero_muon_set_lr(h, lr)
    finally:
        z.zero_muon_destroy(h)


def test_sixteen_bit_masters(z):
    """master None: the 16-bit parameter is widened, updated and rounded."""
    import torch
    shapes = [(70, 130, 2), (64, 48, 1)]
    a, b = matrices(shapes, "bf16", 12), matrices(shapes, "bf16", 12)
    cfg = dict(grad_dtype=z.BF16, lr=1e-2, scale_rule=1, weight_decay=0.1)
    h = z.zero_muon_create(z.make_muon_config(**cfg), shapes)
    try:
        for m in a:
            m["master"] = None
        for m in b:
            m["master"] = m["param16"].float()
        z.zero_muon_step(h, z.make_muon_list(a))
        z.zero_muon_step(h, z.make_muon_list(b))
        for x, y in zip(a, b):
            assert torch.equal(x["param16"], y["param16"])
            assert torch.equal(x["momentum"], y["momentum"])
    finally:
        z.zero_muon_destroy(h)


def test_odd_addresses(z):
    """Arrays at addresses that are multiples of their element only, as slices
    of a flat buffer are."""
    import torch
    m, n = 65, 40
    want, got = matrices([(m, n, 1)], "fp16", 13)[0], matrices([(m, n, 1)], "fp16", 13)[0]
    for name in got:
        flat = torch.full((m * n + 2,), 5.0, device="cuda", dtype=got[name].dtype)
        flat[1:-1] = got[name].flatten()
        got[name] = flat[1:-1].view(1, m, n)
    h = z.zero_muon_create(z.make_muon_config(lr=1e-2), [(m, n)])
    try:
        for x in (want, got):
            z.zero_muon_step(h, z.make_muon_list([x]))
        for name in got:
            assert torch.equal(got[name], want[name]), name
            assert got[name]._base[0] == 5 and got[name]._base[-1] == 5
    finally:
        z.zero_muon_destroy(h)


def test_step_goes_by_the_other_parameters_decision(z):
    """Loss scale, clip and skip come from zero_opt_step's decision on the device."""
    import torch
    shapes = [(48, 96, 1), (120, 64, 2)]
    lr, mu, wd = 1e-2, 0.95, 0.0
    n = 1000
    opt = z.zero_opt_create(z.make_config(numel=n, grad_dtype=z.FP16, max_grad_norm=0.5,
                                          init_scale=1024.0, lr=1e-3))
    h = z.zero_muon_create(z.make_muon_config(lr=lr), shapes)
    try:
        p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
        p16 = torch.zeros(n, device="cuda", dtype=torch.float16)
        grad = torch.full((n,), 64.0, device="cuda", dtype=torch.float16)
        bufs = z.make_buffers(p, m, v, p16, [grad], grads_shard_local=True)
        mats = matrices(shapes, "fp16", 14, 1024.0)
        lst = z.make_muon_list(mats)
        where = z.zero_opt_decision(opt)
        z.zero_opt_step(opt, 0, bufs)
        coef = z.zero_opt_last_step(opt).coef
        assert 0 < coef < 1 / 1024.0                      # clipped
        want = [expected(z, x, coef, lr, mu, wd, True, 0) for x in mats]
        z.zero_muon_step(h, lst, decision=where)
        for x, (mom, tol_m, w, tol_w) in zip(mats, want):
            assert ((x["momentum"].double() - mom).abs() <= tol_m).all()
            assert ((x["master"].double() - w).flatten(-2).norm(dim=-1) <= tol_w).all()
        assert z.zero_muon_last_step(h).skipped == 0
        # an overflow: nothing moves, here as there
        grad[5] = float("inf")
        mats[0]["grad"][0, 0, 0] = float("inf")
        before = [{k: t.clone() for k, t in x.items()} for x in mats]
        z.zero_opt_step(opt, 0, bufs)
        z.zero_muon_step(h, lst, decision=where)
        assert z.zero_opt_last_step(opt).skipped == 1 and z.zero_muon_last_step(h).skipped == 1
        for x, y in zip(mats, before):
            for k in x:
                assert torch.equal(x[k], y[k])
    finally:
        z.zero_muon_destroy(h)
        z.zero_opt_destroy(opt)


def test_another_stream_and_a_graph(z):
    import torch
    shapes = [(100, 60, 1), (256, 300, 2)]
    h = z.zero_muon_create(z.make_muon_config(lr=1e-2), shapes)
    try:
        runs = []
        for how in ("plain", "stream", "graph"):
            mats = matrices(shapes, "fp16", 15)
            lst = z.make_muon_list(mats)
            torch.cuda.synchronize()
            if how == "plain":
                z.zero_muon_step(h, lst)
                z.zero_muon_step(h, lst)
            elif how == "stream":
                s = torch.cuda.Stream()
                with torch.cuda.stream(s):
                    z.zero_muon_step(h, lst)
                z.zero_muon_step(h, lst, stream=s)
                s.synchronize()
            else:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    z.zero_muon_step(h, lst)
                g.replay()
                g.replay()
            torch.cuda.synchronize()
            runs.append(mats)
        for a, b, c in zip(*runs):
            for k in a:
                assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k])
    finally:
        z.zero_muon_destroy(h)


def test_an_empty_list_and_the_workspace(z):
    h = z.zero_muon_create(z.make_muon_config(), [])
    z.zero_muon_step(h, z.make_muon_list([]))
    z.zero_muon_orthogonalize(h, [], [])
    assert z.zero_muon_launch_count(h) == 0
    z.zero_muon_destroy(h)
    h = z.zero_muon_create(z.make_muon_config(), [(512, 1024)])
    # X twice and its second part, 2 bytes each; A and B
    assert z.zero_muon_workspace_bytes(h) >= 512 * 1024 * 6 + 512 * 512 * 4
    z.zero_muon_destroy(h)


def test_binding_refuses(z):
    import torch
    h = z.zero_muon_create(z.make_muon_config(), [(8, 16), (4, 4, 3)])
    try:
        a, b = torch.randn(8, 16, device="cuda"), torch.randn(3, 4, 4, device="cuda")
        z.zero_muon_orthogonalize(h, [a, b], [a.clone(), b.clone()])
        for bad in (a.cpu(), a.double(), a.half(), a[:4], a.T, a[None].repeat(2, 1, 1),
                    torch.randn(16, 8, device="cuda").T):
            with pytest.raises(ValueError):
                z.zero_muon_orthogonalize(h, [bad, b], [a.clone(), b.clone()])
        with pytest.raises(ValueError):
            z.zero_muon_orthogonalize(h, [a], [a])
        with pytest.raises(ValueError):
            z.zero_muon_orthogonalize(h + 8, [a, b], [a, b])
        with pytest.raises(ValueError):
            z.make_muon_list([dict(grad=a.T, momentum=a, master=a, param16=a)])
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("shape", [(100, 60, 1), (128, 1000, 2), (257, 300, 1), (1536, 1536, 4)], ids=str)
def test_a_wait_that_runs_out_is_a_reported_fault(z, shape):
    """On the chip, with a CTA and a cluster a matrix, and through the workspace,
    with single CTAs' tiles and with pairs': the call ends by itself, says
    so, writes no result, and the next one is whole."""
    import torch
    m, n, b = shape
    g = torch.randn(b, m, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    h = z.zero_muon_create(z.make_muon_config(), [shape])
    try:
        out = torch.full_like(g, 7.0)
        z.zero_muon_inject_wait_fault(h)
        z.zero_muon_orthogonalize(h, [g], [out])
        info = z.zero_muon_last_step(h)
        assert (info.skipped, info.fault) == (0, 1) and (out == 7).all()
        z.zero_muon_orthogonalize(h, [g], [out])
        assert z.zero_muon_last_step(h).fault == 0
        close(out, ortho64(g), "fp32")
    finally:
        z.zero_muon_destroy(h)
