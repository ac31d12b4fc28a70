"""The rows of a decoder's block between its matrix products, as a training
program calls them: each operator in a plain form (elementary torch operations
in binary32, rounded once at the end) and as calls of this package.

- ``join`` / ``join_grad``: a block's output y is put on the residual stream x
  and the next block's input h taken from it in the same pass.
      z  = y / sqrt(mean y^2 + eps) * y_gain     (or y * y_gain: a scale a channel)
      b  = dropout(beta * z * act(gate))
      x' = alpha * x + b
      h  = x' / sqrt(mean x'^2 + eps) * gain
  and the gradients with respect to x, y, the gate and the gains.  A token whose
  mask is false is padding: its outputs and gradients are zero.
- ``drop``: dropout by a counter-based generator.  Number (t, d) of a tensor of
  D columns takes half d % 8 of the eight 16-bit halves (of each word the lower
  one first) that Philox 4x32 with ten rounds (Salmon et al., 2011) makes of the
  counter (t ceil(D / 8) + d / 8 in 64 bits, call, step) and the key (seed); it
  is kept where that half is at least round(65536 p), and scaled by
  65536 / (65536 - round(65536 p)).  The same bits drop inside ``join``.
- ``axes`` / ``axes_grad``: queries and keys normalised and rotated by positions
  of several axes (time, height, width), each pair of numbers by the position of
  its own axis, and the gradients.  A token with a negative position is padding.
"""
import math
import weakref

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
EPS = 1e-6
SEED, CALL, STEP = 0x5EED0001C0FFEE, 3, 1000


# ---------------------------------------------------------------- cases

def _join(name, op, tokens, dim, dtype, stream=None, post=False, gate="none", p=0.0, mask=0.0, alpha=1.0,
          beta=1.0):
    c = dict(op=op, tokens=tokens, dim=dim, dtype=dtype, stream=stream or dtype, post=post, gate=gate, p=p,
             mask=mask, alpha=alpha, beta=beta)
    return dict(c, name=name) if name else c


def _axes(name, op, tokens, hq, hk, dim, dtype, sections, mixed=False, inter=False, normalise=True, fused=True,
          pad=0.0):
    c = dict(op=op, tokens=tokens, hq=hq, hk=hk, dim=dim, dtype=dtype, sections=sections, mixed=mixed,
             inter=inter, normalise=normalise, fused=fused, pad=pad)
    return dict(c, name=name) if name else c


def listed():
    return [
        # One new token of a served sequence: latency only.
        _join("join one token", "join", 1, 4096, "bf16", post=True),
        # A ragged batch of an odd width with padding, a gate computed from the block's input, dropout.
        _join("join ragged 515x777", "join", 515, 777, "fp16", gate="sigmoid", p=0.1, mask=0.1),
        # A long prompt, or one forward pass of a training micro-batch, with norms before and after.
        _join("join 16384x4096", "join", 16384, 4096, "bf16", post=True),
        # A small model's training step: the stream in binary32, dropout on the branch.
        _join("join gradient 2048x768", "join_grad", 2048, 768, "fp16", stream="fp32", p=0.1),
        # The same of an odd width, with its gate and a norm of the branch.
        _join("join gradient 1001x777", "join_grad", 1001, 777, "fp16", post=True, gate="sigmoid", p=0.1,
              mask=0.1),
        # The backward pass of the large micro-batch.
        _join("join gradient 16384x4096", "join_grad", 16384, 4096, "bf16", post=True),
        # An odd tensor, as a classifier's features.
        dict(name="dropout 1001x777", op="drop", rows=1001, dim=777, dtype="fp16", p=0.1),
        # The embeddings of a large micro-batch.
        dict(name="dropout 16384x4096", op="drop", rows=16384, dim=4096, dtype="bf16", p=0.1),
        # One image between a prompt's words: a few hundred tokens.
        _axes("axes one image", "axes", 300, 32, 8, 128, "bf16", "16,24,24"),
        # A video's clip.
        _axes("axes 16384 tokens", "axes", 16384, 32, 8, 128, "bf16", "16,24,24"),
        # An image encoder's patches, rotated by height and width without a norm.
        _axes("axes patches 4096", "axes", 4096, 16, 16, 80, "fp16", "20,20", normalise=False),
        # The backward pass of a small ragged batch, the axes taking turns over the pairs.
        _axes("axes gradient 3001", "axes_grad", 3001, 12, 4, 64, "fp16", "12,10,10", mixed=True, fused=False,
              pad=0.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["join", "join_grad", "drop", "axes", "axes_grad"])
    if op in ("axes", "axes_grad"):
        dim = rng.choice([64, 80, 96, 128, 128])
        axes = rng.choice([2, 3, 3])
        first = dim // 8 if axes == 3 else dim // 4
        rest = dim // 2 - first
        sections = "%d,%d" % (first, rest) if axes == 2 else "%d,%d,%d" % (first, rest // 2, rest - rest // 2)
        hk = rng.choice([1, 2, 4, 8])
        return _axes(None, op, _log(rng, 1, 8192 if op == "axes_grad" else 16384), hk * rng.choice([1, 2, 4]),
                     hk, dim, rng.choice(["bf16", "bf16", "fp16"]), sections, mixed=rng.random() < 0.3,
                     inter=rng.random() < 0.3, normalise=rng.random() < 0.75, fused=rng.random() < 0.5,
                     pad=rng.choice([0.0, 0.0, 0.1]))
    while True:
        rows, dim = _log(rng, 1, 16384), _log(rng, 64, 8192)
        # widths of models are multiples of 64; an odd one now and then
        dim = dim | 1 if rng.random() < 0.25 else -(-dim // 64) * 64
        if rows * dim <= 16384 * 4096:
            break
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "drop":
        return dict(op=op, rows=rows, dim=dim, dtype=dtype, p=rng.choice([0.05, 0.1, 0.3, 0.5]))
    wide = rng.random() < 0.25 and rows * dim <= 8192 * 4096   # no more bytes than the largest listed
    return _join(None, op, rows, dim, dtype, stream="fp32" if wide else dtype, post=rng.random() < 0.5,
                 gate=rng.choice(["none", "none", "none", "plain", "sigmoid"]) if rows * dim <= 8192 * 4096
                 else "none", p=rng.choice([0.0, 0.0, 0.1]), mask=rng.choice([0.0, 0.0, 0.1]),
                 alpha=rng.choice([1.0, 1.0, 1.5]), beta=rng.choice([1.0, 1.0, 0.5]))


def work(case):
    op = case["op"]
    if op == "drop":
        n = case["rows"] * case["dim"]
        return {"bytes": 2 * n * SIZE[case["dtype"]], "flops": n}
    if op in ("join", "join_grad"):
        n = case["tokens"] * case["dim"]
        es, ss = SIZE[case["dtype"]], SIZE[case["stream"]]
        gate = case["gate"] != "none"
        small = 2 * case["dim"] * 4 + (case["tokens"] if case["mask"] else 0)
        if op == "join":       # x, y, gate; the stream and the next input
            return {"bytes": n * (2 * ss + 2 * es + gate * es) + small, "flops": n * 12}
        # the stream, its gradient, y, dh, gate; dx, dy, the gate's gradient
        return {"bytes": n * (3 * ss + 3 * es + 2 * gate * es) + 2 * small, "flops": n * 30}
    heads, T, D = case["hq"] + case["hk"], case["tokens"], case["dim"]
    row = heads * D * SIZE[case["dtype"]]
    small = min(T, _n_pos(case)) * D * 4 + T * 8 * len(_sections(case)) + case["normalise"] * 2 * D * 4
    if op == "axes":
        return {"bytes": T * 2 * row + small, "flops": T * heads * D * 8}
    moved = 3 if case["normalise"] else 2        # without a norm the gradient needs no x
    return {"bytes": T * moved * row + small + case["normalise"] * 2 * D * 4, "flops": T * heads * D * 16}


# ---------------------------------------------------------------- inputs

class State:
    """What a user's program holds; a handle in it is destroyed with it."""

    def __init__(self, case):
        self.case = case

    def keep(self, handle, destroy):
        self.handle = handle
        weakref.finalize(self, destroy, handle)


def _rand(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _sections(case):
    return [int(v) for v in case["sections"].split(",")]


def _axis_of(case):
    """The axis of each pair: one section after another, or the axes in turn
    while they have pairs left."""
    left = _sections(case)
    if not case["mixed"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _n_pos(case):
    return 1 << max(6, case["tokens"].bit_length())


def _positions(case, gen):
    """Words, whose axes agree, around pictures of up to 24 x 24 patches."""
    T, A = case["tokens"], len(_sections(case))
    at = torch.arange(T, device="cuda")
    start = torch.randint(0, 64, (T // 600 + 1,), device="cuda", generator=gen).repeat_interleave(600)[:T]
    inside, side = at % 600 - 24, 24
    picture = (inside >= 0) & (inside < side * side)
    grid = [at // 600, inside // side, inside % side][3 - A:]
    base = at // 600 * 8 + start
    rows = [torch.where(picture, base + g, base) for g in grid]
    return torch.stack(rows).remainder(_n_pos(case))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 29)
    s = State(case)
    s.seed = SEED + seed
    if case["op"] == "drop":
        s.x = _rand(gen, case["rows"], case["dim"]).to(DTYPES[case["dtype"]])
        s.out = torch.empty_like(s.x)
        return s
    if case["op"] in ("join", "join_grad"):
        T, D, dt, st = case["tokens"], case["dim"], DTYPES[case["dtype"]], DTYPES[case["stream"]]
        # a few channels of the stream are much larger than the others, as in trained models
        strong = 1.0 + 10.0 * (torch.rand(D, device="cuda", generator=gen) < 0.005)
        s.x = (_rand(gen, T, D) * strong).to(st)         # the gradient's case: the stream behind the block
        s.y = (_rand(gen, T, D) * 0.7).to(dt)
        s.gate = _rand(gen, T, D).to(dt) if case["gate"] != "none" else None
        s.y_gain = (1.0 if case["post"] else 0.5) * (1.0 + 0.2 * _rand(gen, D))
        s.gain = 1.0 + 0.2 * _rand(gen, D)
        s.mask = torch.rand(T, device="cuda", generator=gen) >= case["mask"] if case["mask"] else None
        if case["op"] == "join":
            s.x_out, s.h = torch.empty_like(s.x), torch.empty_like(s.y)
        else:
            s.dx_out, s.dh = (_rand(gen, T, D) * 0.02).to(st), (_rand(gen, T, D) * 0.02).to(dt)
            s.dx, s.dy = torch.empty_like(s.x), torch.empty_like(s.y)
            s.dgate = torch.empty_like(s.y) if s.gate is not None else None
            s.dy_gain, s.dgain = torch.empty_like(s.y_gain), torch.empty_like(s.gain)
        if own:
            import zero_sharded_mixed_05_gb300 as z
            code = {"fp16": z.FP16, "bf16": z.BF16, "fp32": z.FP32}
            cfg = z.make_block_config(D, dtype=code[case["dtype"]], stream_dtype=code[case["stream"]],
                                      norm_branch=case["post"], norm_out=True, alpha=case["alpha"],
                                      gate={"none": z.GATE_NONE, "plain": z.GATE_PLAIN,
                                            "sigmoid": z.GATE_SIGMOID}[case["gate"]],
                                      beta=case["beta"], dropout=case["p"], eps=EPS)
            s.keep(z.zero_block_create(cfg), z.zero_block_destroy)
        return s
    T, hq, hk, D = (case[k] for k in ("tokens", "hq", "hk", "dim"))
    dt = DTYPES[case["dtype"]]

    def heads(sigma):
        """Queries and keys: views of the projection's one output (with the
        values behind them) or tensors of their own."""
        if case["fused"]:
            qkv = (_rand(gen, T, hq + 2 * hk, D) * sigma).to(dt)
            return qkv[:, :hq], qkv[:, hq:hq + hk]
        return (_rand(gen, T, hq, D) * sigma).to(dt), (_rand(gen, T, hk, D) * sigma).to(dt)

    s.q, s.k = heads(1.3)
    s.qg = s.kg = s.dqg = s.dkg = None
    if case["normalise"]:
        s.qg, s.kg = 1 + 0.2 * _rand(gen, D), 1 + 0.2 * _rand(gen, D)
    freq = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    angle = torch.arange(_n_pos(case), device="cuda", dtype=torch.float64)[:, None] * freq
    s.cos, s.sin = angle.cos().float(), angle.sin().float()
    s.pos = _positions(case, gen)
    if case["pad"]:
        s.pos[:, torch.rand(T, device="cuda", generator=gen) < case["pad"]] = -1
    if case["op"] == "axes_grad":
        s.dqo, s.dko = (_rand(gen, T, hq, D) * 0.02).to(dt), (_rand(gen, T, hk, D) * 0.02).to(dt)
        if case["normalise"]:
            s.dqg, s.dkg = torch.empty_like(s.qg), torch.empty_like(s.kg)
    s.qo, s.ko = torch.empty(T, hq, D, device="cuda", dtype=dt), torch.empty(T, hk, D, device="cuda", dtype=dt)
    if own:
        import zero_sharded_mixed_05_gb300 as z
        cfg = z.make_qk_config(q_heads=hq, k_heads=hk, head_dim=D, interleaved=case["inter"], eps=EPS,
                               dtype=z.dtype_code(dt))
        axes = z.make_qk_axes(_axis_of(case), normalise=case["normalise"])
        s.keep(z.zero_qk_create(cfg, axes), z.zero_qk_destroy)
    return s


# ---------------------------------------------------------------- plain forms

def _threshold(p):
    return int(math.floor(65536 * p + 0.5))


def _halves(rows, dim, seed):
    """The generator's 16-bit halves of a [rows, dim] tensor.  Words are held in
    64-bit integers; a product's bits wrap as they should."""
    low = 0xFFFFFFFF
    blocks = -(-dim // 8)
    n = torch.arange(rows * blocks, device="cuda")
    c0, c1 = n & low, n >> 32
    c2, c3 = torch.full_like(n, CALL), torch.full_like(n, STEP)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    words = torch.stack((c0, c1, c2, c3), -1)
    return torch.stack((words & 0xFFFF, words >> 16), -1).view(rows, blocks * 8)[:, :dim]


def _kept(s, rows, dim):
    """Which numbers stay, and what they are scaled by."""
    t = _threshold(s.case["p"])
    return _halves(rows, dim, s.seed) >= t, 65536.0 / (65536 - t)


def _dropped(x, s):
    if s.case["p"] == 0.0:
        return x
    keep, scale = _kept(s, *x.shape)
    return torch.where(keep, x * scale, 0.0)


def _live(x, s):
    return x if s.mask is None else torch.where(s.mask[:, None], x, 0.0)


def _act(s):
    """The gate's factor and its derivative."""
    if s.gate is None:
        return 1.0, 0.0
    g = s.gate.float()
    if s.case["gate"] == "plain":
        return g, 1.0
    a = 1.0 / (1.0 + torch.exp(-g))
    return a, a * (1.0 - a)


def _inverse(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _join_plain(s):
    c = s.case
    y = s.y.float()
    if c["post"]:
        y = y * _inverse(y)
    b = _dropped(c["beta"] * (y * s.y_gain) * _act(s)[0], s)
    x = c["alpha"] * s.x.float() + b
    h = x * _inverse(x) * s.gain
    return _live(x, s).to(s.x.dtype), _live(h, s).to(s.y.dtype)


def _join_grad_plain(s):
    c = s.case
    x, y, dh = _live(s.x.float(), s), _live(s.y.float(), s), _live(s.dh.float(), s)
    r = _inverse(x)
    xhat, dn = x * r, dh * s.gain
    G = _live(s.dx_out.float(), s) + r * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
    db = _dropped(c["beta"] * G, s)
    ry = _inverse(y) if c["post"] else 1.0
    yhat = y * ry
    act, slope = _act(s)
    dz = db * act
    dn = dz * s.y_gain
    dy = ry * (dn - yhat * (dn * yhat).mean(-1, keepdim=True)) if c["post"] else dn
    out = [(c["alpha"] * G).to(s.x.dtype), dy.to(s.y.dtype), (dz * yhat).sum(0), (dh * xhat).sum(0)]
    if s.gate is not None:
        out.append(_live(db * yhat * s.y_gain * slope, s).to(s.y.dtype))
    return out


def _pairs(x, inter):
    half = x.shape[-1] // 2
    return (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :half], x[..., half:])


def _joined(a, b, inter):
    return torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)


def _tables(s):
    """Whether a token is there, and its pairs' cosines and sines."""
    axis = torch.tensor(_axis_of(s.case), device="cuda")
    at, pair = s.pos.clamp(min=0)[axis].T, torch.arange(len(axis), device="cuda")
    live = (s.pos >= 0).all(0)[:, None, None]
    return live, s.cos[at, pair][:, None], s.sin[at, pair][:, None]


def _axes_plain(x, gain, s, live, cos, sin):
    y = x.float()
    if gain is not None:
        y = y * _inverse(y) * gain
    u, v = _pairs(y, s.case["inter"])
    return torch.where(live, _joined(u * cos - v * sin, v * cos + u * sin, s.case["inter"]), 0.0).to(x.dtype)


def _axes_grad_plain(dout, x, gain, s, live, cos, sin):
    dout = torch.where(live, dout.float(), 0.0)
    u, v = _pairs(dout, s.case["inter"])
    dy = _joined(u * cos + v * sin, v * cos - u * sin, s.case["inter"])
    if gain is None:
        return dy.to(x.dtype), None
    x = x.float()
    r = _inverse(x)
    xhat, dn = x * r, dy * gain
    dx = r * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
    return dx.to(s.q.dtype), (dy * xhat).sum((0, 1))


# ---------------------------------------------------------------- one pass

def run(s):
    case = s.case
    if own:
        import zero_sharded_mixed_05_gb300 as z
    if case["op"] == "drop":
        if own:
            z.zero_dropout(s.x, s.out, case["p"], seed=s.seed, call=CALL, step=STEP)
            return s.out
        return _dropped(s.x.float(), s).to(s.x.dtype)
    if case["op"] == "join":
        if own:
            z.zero_block_join(s.handle, s.x, s.y, s.x_out, s.h, s.y_gain, s.gain, gate=s.gate, mask=s.mask,
                              seed=s.seed, call=CALL, step=STEP)
            return s.x_out, s.h
        return _join_plain(s)
    if case["op"] == "join_grad":
        if own:
            z.zero_block_join_backward(s.handle, s.dx_out, s.dh, s.x, s.y, s.dx, s.dy, s.dy_gain, s.dgain,
                                       s.y_gain, s.gain, gate=s.gate, dgate=s.dgate, mask=s.mask, seed=s.seed,
                                       call=CALL, step=STEP)
            out = [s.dx, s.dy, s.dy_gain, s.dgain]
            return out if s.gate is None else out + [s.dgate]
        return _join_grad_plain(s)
    if case["op"] == "axes":
        if own:
            z.zero_qk_norm_rope(s.handle, s.q, s.k, s.qo, s.ko, s.qg, s.kg, s.cos, s.sin, s.pos)
            return s.qo, s.ko
        t = _tables(s)
        return _axes_plain(s.q, s.qg, s, *t), _axes_plain(s.k, s.kg, s, *t)
    if own:
        z.zero_qk_norm_rope_backward(s.handle, s.dqo, s.dko, s.q, s.k, s.qo, s.ko, s.dqg, s.dkg,
                                     s.qg, s.kg, s.cos, s.sin, s.pos)
        return (s.qo, s.ko, s.dqg, s.dkg) if case["normalise"] else (s.qo, s.ko)
    t = _tables(s)
    dq, dqg = _axes_grad_plain(s.dqo, s.q, s.qg, s, *t)
    dk, dkg = _axes_grad_plain(s.dko, s.k, s.kg, s, *t)
    return (dq, dk, dqg, dkg) if case["normalise"] else (dq, dk)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_keep(rows, dim, seed, p):
    """The generator once more, word by word: products by their 16-bit digits."""
    def product(x, m):
        lo, hi = (x & 0xFFFF) * m, (x >> 16) * m          # below 2^48
        mid = hi + (lo >> 16)
        return mid >> 16, (mid & 0xFFFF) << 16 | lo & 0xFFFF

    per = (dim + 7) // 8
    row = torch.arange(rows, device="cuda")[:, None] * per
    number = (row + torch.arange(per, device="cuda")).reshape(-1)
    x = [number % 2 ** 32, number // 2 ** 32, torch.full_like(number, CALL), torch.full_like(number, STEP)]
    for i in range(10):
        key = [(seed % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32]
        high0, low0 = product(x[0], 0xD2511F53)
        high1, low1 = product(x[2], 0xCD9E8D57)
        x = [high1 ^ x[1] ^ key[0], low1, high0 ^ x[3] ^ key[1], low0]
    halves = torch.empty(rows, per, 8, dtype=torch.int32, device="cuda")
    for w in range(4):
        halves[:, :, 2 * w] = (x[w] % 65536).view(rows, per)
        halves[:, :, 2 * w + 1] = (x[w] // 65536).view(rows, per)
    return (halves.view(rows, per * 8)[:, :dim] >= round(65536 * p)).double()


def _normed(x):
    return x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) ** 0.5


def _exact_turn(x, s):
    """The rotation as a product of complex numbers."""
    axis = _axis_of(s.case)
    at = s.pos.clamp(min=0)
    w = torch.stack([torch.complex(s.cos[at[a], j].double(), s.sin[at[a], j].double())
                     for j, a in enumerate(axis)], -1)[:, None]
    z = torch.complex(*(t.contiguous() for t in _pairs(x, s.case["inter"]))) * w
    return _joined(z.real, z.imag, s.case["inter"]) * (s.pos.amin(0) >= 0).double()[:, None, None]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    factor = 65536.0 / (65536.0 - round(65536 * case["p"])) if case.get("p") else 1.0
    if case["op"] == "drop":
        return s.x.double() * _exact_keep(case["rows"], case["dim"], s.seed, case["p"]) * factor
    if case["op"] in ("join", "join_grad"):
        there = torch.ones_like(s.y[:, :1], dtype=torch.float64) if s.mask is None else s.mask.double()[:, None]
        keep = there * factor
        if case["p"]:
            keep = keep * _exact_keep(case["tokens"], case["dim"], s.seed, case["p"])

        def branch(y, y_gain, gate):
            z = (_normed(y) if case["post"] else y) * y_gain
            if gate is not None:
                z = z * (gate if case["gate"] == "plain" else torch.sigmoid(gate))
            return case["beta"] * z * keep

        gate = None if s.gate is None else s.gate.double()
        if case["op"] == "join":
            x = there * (case["alpha"] * s.x.double() + branch(s.y.double(), s.y_gain.double(), gate))
            return x, _normed(x) * s.gain.double()
        # the stream behind the block is given, so its gradient comes first and the branch's from it
        with torch.enable_grad():
            x, gain = s.x.double().requires_grad_(), s.gain.double().requires_grad_()
            G, dgain = torch.autograd.grad(_normed(x) * gain * there, (x, gain), s.dh.double())
            G = G + s.dx_out.double() * there
            leaves = [s.y.double().requires_grad_(), s.y_gain.double().requires_grad_()]
            if gate is not None:
                leaves.append(gate.requires_grad_())
            grads = torch.autograd.grad(branch(leaves[0], leaves[1], gate), leaves, G)
        return [case["alpha"] * G, grads[0], grads[1], dgain, *grads[2:]]

    def forward(x, gain):
        return _exact_turn(x if gain is None else _normed(x) * gain, s)

    if case["op"] == "axes":
        return tuple(forward(x.double(), None if g is None else g.double())
                     for x, g in ((s.q, s.qg), (s.k, s.kg)))
    out = []
    with torch.enable_grad():
        for x, g, d in ((s.q, s.qg, s.dqo), (s.k, s.kg, s.dko)):
            leaves = [x.double().requires_grad_()]
            if g is not None:
                leaves.append(g.double().requires_grad_())
            out.append(torch.autograd.grad(forward(leaves[0], leaves[1] if g is not None else None), leaves,
                                           d.double()))
    return tuple(o[0] for o in out) + tuple(o[1] for o in out if len(o) > 1)
