"""The join's and dropout's autograd wrappers, and the operators together in a
decoder's blocks, against torch's autograd on the formulas in 64 bits."""
import gc

import pytest

import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import zero_sharded_mixed_05_gb300 as z
    z.lib()
    return z


def norm64(x):
    return x * (x.square().mean(-1, keepdim=True) + R.EPS) ** -0.5


def keep_of(T, D, p, *rng):
    import torch
    return torch.from_numpy(R.kept(T, D, p, *rng)).cuda().double() * R.factor(p)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("uses", ["both", "x_out", "h"])
def test_gradients(z, post, uses):
    """x broadcast over tokens and a gate broadcast over them, gains, both
    results or one.  Binary32: (D + 48) 2^-24 of terms below 30, twice through a
    norm, summed over up to T tokens."""
    import torch
    from zero_sharded_mixed_05_gb300.block import BlockJoin
    g = torch.Generator(device="cuda").manual_seed(1)
    T, D, p = 50, 72, 0.25
    leaves = dict(x=torch.randn(1, D, device="cuda", generator=g), y=torch.randn(T, D, device="cuda", generator=g),
                  yg=1 + 0.1 * torch.randn(D, device="cuda", generator=g),
                  gn=1 + 0.1 * torch.randn(D, device="cuda", generator=g),
                  gate=torch.randn(1, D, device="cuda", generator=g))
    w = [torch.randn(T, D, device="cuda", generator=g) for _ in range(2)]
    mask = torch.rand(T, device="cuda", generator=g) < 0.8
    use = dict(both=(1, 1), x_out=(1, 0), h=(0, 1))[uses]
    join = BlockJoin(z.make_block_config(D, dtype=z.FP32, norm_branch=post, gate=z.GATE_SIGMOID, alpha=1.5,
                                         beta=0.5, dropout=p))
    a = {k: t.clone().requires_grad_() for k, t in leaves.items()}
    xo, h = join(a["x"].expand(T, D), a["y"], a["yg"], a["gn"], gate=a["gate"].expand(T, D), mask=mask, seed=3,
                 call=1, step=2)
    sum((o * v).sum() for o, v, u in zip((xo, h), w, use) if u).backward()
    b = {k: t.double().requires_grad_() for k, t in leaves.items()}
    y = norm64(b["y"]) if post else b["y"]
    x = 1.5 * b["x"] + 0.5 * y * b["yg"] * torch.sigmoid(b["gate"]) * keep_of(T, D, p, 3, 1, 2)
    m = mask[:, None]
    ref = (x * m, norm64(x) * b["gn"] * m)
    sum((o * v).sum() for o, v, u in zip(ref, w, use) if u).backward()
    for k in leaves:
        if uses == "x_out" and k == "gn":
            assert a[k].grad is None or not a[k].grad.any()
            continue
        n = T if k != "y" else 1
        assert ((a[k].grad.double() - b[k].grad).abs() <= 2 * (D + 48) * R.E32 * 30 * n).all(), k
    join.close()


def test_norm_alone_and_who_wants_what(z):
    import torch
    from zero_sharded_mixed_05_gb300.block import BlockJoin
    g = torch.Generator(device="cuda").manual_seed(2)
    T, D = 40, 256
    x, w = (torch.randn(T, D, device="cuda", generator=g) for _ in range(2))
    join = BlockJoin(z.make_block_config(D, dtype=z.FP32))
    a, ga = x.clone().requires_grad_(), torch.ones(D, device="cuda", requires_grad=True)
    (join.norm(a, ga) * w).sum().backward()
    b, gb = x.double().requires_grad_(), torch.ones(D, device="cuda", dtype=torch.float64, requires_grad=True)
    (norm64(b) * gb * w).sum().backward()
    assert ((a.grad.double() - b.grad).abs() <= (D + 48) * R.E32 * 30).all()
    assert ((ga.grad.double() - gb.grad).abs() <= (D + 48) * R.E32 * 30 * T).all()
    # a constant stream, a y without a gradient, gains without one
    y = torch.randn(T, D, device="cuda", generator=g).requires_grad_()
    for x_, y_ in ((x, y), (x.clone().requires_grad_(), y.detach())):
        before = z.zero_block_launch_count(join._handle)
        xo, h = join(x_, y_)
        h.sum().backward()
        assert z.zero_block_launch_count(join._handle) == before + 2      # no sums of gains
    with pytest.raises(ValueError):
        join(x, None)
    with pytest.raises(ValueError):
        join(x, y, gate=x)
    with pytest.raises(RuntimeError):                      # a second derivative
        (d,) = torch.autograd.grad(join.norm(a, ga).square().sum(), a, create_graph=True)
        d.sum().backward()
    # the graph keeps the handle
    out = join.norm(a, ga).sum()
    del join
    gc.collect()
    out.backward()


def test_a_changed_step_is_noticed(z):
    """The backward pass makes the forward pass's bits again from the step on the
    device: torch refuses one that was changed in between."""
    import torch
    from zero_sharded_mixed_05_gb300.block import BlockJoin, dropout
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    join = BlockJoin(z.make_block_config(64, dtype=z.FP32, dropout=0.5))
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    for out in (dropout(x, 0.5, step=step).sum(), join(x, x, step=step)[1].sum()):
        step += 1
        with pytest.raises(RuntimeError):
            out.backward()
    join.close()


def test_dropout_gradient(z):
    import torch
    from zero_sharded_mixed_05_gb300.block import dropout
    x = torch.randn(6, 5, 44, device="cuda").transpose(0, 1)
    a = x.clone().requires_grad_()
    w = torch.randn(5, 6, 44, device="cuda").transpose(1, 2).contiguous().transpose(1, 2)
    out = dropout(a.transpose(0, 1).transpose(0, 1), 0.4, seed=8, call=2, step=5)
    k = keep_of(30, 44, 0.4, 8, 2, 5).view(5, 6, 44)
    (out * w).sum().backward()
    assert ((out.double() - x.double() * k).abs() <= 2 * R.E32 * x.double().abs() * k).all()
    assert ((a.grad.double() - w.double() * k).abs() <= 2 * R.E32 * w.double().abs() * k).all()


def test_together_in_a_decoder(z):
    """Two blocks of a small decoder over a picture between words: the stream's
    norms and joins with dropout, and queries and keys turned by three axes, in
    binary32; every gradient against the formulas in 64 bits.  The products and
    the attention are torch's, whose binary32 errors dominate: within 2e-4 of
    each gradient's largest number (sums of up to 2 x 90 x 128 rounded terms,
    2^-24 sqrt(23040) = 9e-6 in the mean, through two blocks)."""
    import torch
    from zero_sharded_mixed_05_gb300.block import BlockJoin, dropout
    from zero_sharded_mixed_05_gb300.qk import QkNormRope, axis_of_pairs, make_qk_axes, rotation_tables
    torch.backends.cuda.matmul.allow_tf32 = False
    g = torch.Generator(device="cuda").manual_seed(5)
    T, D, H, HD, p = 90, 128, 4, 32, 0.1

    def rand(*s, scale=1.0):
        return torch.randn(*s, device="cuda", generator=g) * scale
    weights = dict(embed=rand(T, D), final=1 + 0.1 * rand(D))
    for i in range(2):
        weights.update({f"qkv{i}": rand(3 * D, D, scale=D ** -0.5), f"out{i}": rand(D, D, scale=D ** -0.5),
                        f"up{i}": rand(2 * D, D, scale=D ** -0.5), f"down{i}": rand(D, 2 * D, scale=D ** -0.5),
                        f"gate{i}": rand(D, D, scale=D ** -0.5),
                        **{f"{n}{i}": 1 + 0.1 * rand(D) for n in ("n1_", "n2_", "y1_", "y2_")},
                        **{f"{n}{i}": 1 + 0.1 * rand(HD) for n in ("qg", "kg")}})
    target = rand(T, D)
    axis = axis_of_pairs((4, 6, 6))
    cos, sin = rotation_tables(64, HD)
    t = torch.arange(T, device="cuda")
    inside = (t >= 10) & (t < 74)
    pos = torch.stack([torch.where(inside, 10, t), torch.where(inside, 10 + (t - 10) // 8, t),
                       torch.where(inside, 10 + (t - 10) % 8, t)]).clamp(max=63)
    ax, pair = torch.tensor(axis, device="cuda"), torch.arange(HD // 2, device="cuda")
    c64, s64 = (v.double()[pos[ax].T, pair][:, None] for v in (cos, sin))
    causal = torch.ones(T, T, device="cuda", dtype=torch.bool).tril()
    qk = QkNormRope(z.make_qk_config(H, H, HD, dtype=z.FP32), make_qk_axes(axis))
    attn = BlockJoin(z.make_block_config(D, dtype=z.FP32, norm_branch=True, gate=z.GATE_SIGMOID, dropout=p))
    mlp = BlockJoin(z.make_block_config(D, dtype=z.FP32, norm_branch=True, dropout=p))

    def attend(q, k, v):
        a = (torch.einsum("qhd,khd->hqk", q, k) * HD ** -0.5).masked_fill(~causal, float("-inf"))
        return torch.einsum("hqk,khd->qhd", a.softmax(-1), v).reshape(T, D)

    def own(w):
        x = dropout(w["embed"], p, seed=9, call=0, step=7)
        h = attn.norm(x, w["n1_0"])
        for i in range(2):
            q, k, v = (h @ w[f"qkv{i}"].T).view(T, 3 * H, HD).split(H, 1)
            q, k = qk(q, k, w[f"qg{i}"], w[f"kg{i}"], cos, sin, pos)
            x, h = attn(x, attend(q, k, v) @ w[f"out{i}"].T, w[f"y1_{i}"], w[f"n2_{i}"],
                        gate=h @ w[f"gate{i}"].T, seed=9, call=1 + 2 * i, step=7)
            y = torch.relu(h @ w[f"up{i}"].T).square() @ w[f"down{i}"].T
            x, h = mlp(x, y, w[f"y2_{i}"], w["n1_1"] if i == 0 else w["final"], seed=9, call=2 + 2 * i, step=7)
        return (h * target.to(h.dtype)).sum() + x.square().sum() * 0.1

    def plain(w):
        x = w["embed"] * keep_of(T, D, p, 9, 0, 7)
        h = norm64(x) * w["n1_0"]
        for i in range(2):
            q, k, v = (h @ w[f"qkv{i}"].T).view(T, 3 * H, HD).split(H, 1)

            def turn(y, gain):
                y = norm64(y) * gain
                u, o = y[..., :HD // 2], y[..., HD // 2:]
                return torch.cat((u * c64 - o * s64, o * c64 + u * s64), -1)
            y = attend(turn(q, w[f"qg{i}"]), turn(k, w[f"kg{i}"]), v) @ w[f"out{i}"].T
            x = x + norm64(y) * w[f"y1_{i}"] * torch.sigmoid(h @ w[f"gate{i}"].T) * keep_of(T, D, p, 9, 1 + 2 * i, 7)
            h = norm64(x) * w[f"n2_{i}"]
            y = torch.relu(h @ w[f"up{i}"].T).square() @ w[f"down{i}"].T
            x = x + norm64(y) * w[f"y2_{i}"] * keep_of(T, D, p, 9, 2 + 2 * i, 7)
            h = norm64(x) * (w["n1_1"] if i == 0 else w["final"])
        return (h * target.double()).sum() + x.square().sum() * 0.1
    a = {k: v.clone().requires_grad_() for k, v in weights.items()}
    b = {k: v.double().requires_grad_() for k, v in weights.items()}
    la, lb = own(a), plain(b)
    la.backward()
    lb.backward()
    assert abs(la.item() - lb.item()) <= 1e-4 * T * D
    for k in weights:
        d = (a[k].grad.double() - b[k].grad).abs().max()
        assert d <= 2e-4 * b[k].grad.abs().max(), (k, d.item(), b[k].grad.abs().max().item())
    for o in (qk, attn, mlp):
        o.close()
