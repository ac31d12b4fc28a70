"""The matrix-update and query/key operators, as a training program calls them.

Three operators, each in a plain form (elementary torch operations in binary32,
rounded once at the end) and as calls of this package:

- ``ortho``: the orthogonalised form of a matrix (or a stack of them) by five
  Newton-Schulz steps.  With X = G / (|G|_F + eps), k = the smaller side:
  A = X X^T, B = b A + c A A, X <- a X + B X (tall matrices: the same on the
  transpose).
- ``muon``: the optimizer step of a list of matrices with that product: the
  gradient unscaled, M <- mu M + g, U = g + mu M, O = ortho(U),
  W <- W (1 - lr wd) - lr 0.2 sqrt(max(rows, cols)) O, and the 16-bit copy of W.
- ``qk`` / ``qk_grad``: each head's query and key normalised
  (y = x / sqrt(mean x^2 + eps) * gain) and rotated by its token's position in
  the same pass, and the gradients with respect to x and the gains.  A token
  with position -1 is padding: its outputs and gradients are zero.
"""
import math
import weakref

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
ABC = (3.4445, -4.7750, 2.0315)
STEPS = 5
ORTHO_EPS = 1e-7
MUON = dict(lr=2e-4, mu=0.95, wd=0.1)
QK_EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One small matrix on its own (a low-rank adapter's product, a router's weight): latency only.
        dict(name="ortho one 64x64", op="ortho", batch=1, rows=64, cols=64, src="fp32", dst="fp16"),
        # Odd sizes, taller than wide, a few at once.
        dict(name="ortho 3 of 1000x777", op="ortho", batch=3, rows=1000, cols=777, src="fp16", dst="bf16"),
        # The blocks of 32 attention heads, each orthogonalised by itself.
        dict(name="ortho 32 of 128x1024", op="ortho", batch=32, rows=128, cols=1024, src="bf16", dst="bf16"),
        # One feed-forward matrix of the per-tensor list.
        dict(name="ortho 14336x4096", op="ortho", batch=1, rows=14336, cols=4096, src="bf16", dst="bf16"),
        # A small model's step: two blocks of width 256, where launches count.
        dict(name="muon width 256", op="muon", shapes="256x256x8,1024x256x2,256x1024x2",
             grad="fp16", scale=1024.0),
        # Twelve attention blocks of width 768, query/key/value in one matrix.
        dict(name="muon width 768", op="muon", shapes="2304x768x12,768x768x12",
             grad="bf16", scale=1.0),
        # One decoder layer of the per-tensor list (query, output; key, value; gate, up; down).
        dict(name="muon width 4096", op="muon",
             shapes="4096x4096x2,1024x4096x2,14336x4096x2,4096x14336x1", grad="bf16", scale=1.0),
        # One new token of a served sequence.
        dict(name="qk one token", op="qk", tokens=1, hq=32, hk=8, dim=128, rot=128, dtype="bf16",
             gains="head_dim", inter=False, fused=True, pad=0.0),
        # A ragged batch with padding tokens, a head of 80 of which 40 rotate, in adjacent pairs.
        dict(name="qk ragged 515", op="qk", tokens=515, hq=12, hk=12, dim=80, rot=40, dtype="fp16",
             gains="per_head", inter=True, fused=True, pad=0.2),
        # A long prompt, or one forward pass of a training micro-batch.
        dict(name="qk 16384 tokens", op="qk", tokens=16384, hq=32, hk=8, dim=128, rot=128,
             dtype="bf16", gains="head_dim", inter=False, fused=True, pad=0.0),
        # The backward pass of a small ragged micro-batch with gains for each head.
        dict(name="qk gradient 777", op="qk_grad", tokens=777, hq=12, hk=4, dim=64, rot=64,
             dtype="fp16", gains="per_head", inter=False, fused=False, pad=0.1),
        # The backward pass of the large micro-batch.
        dict(name="qk gradient 16384", op="qk_grad", tokens=16384, hq=32, hk=8, dim=128, rot=128,
             dtype="bf16", gains="head_dim", inter=False, fused=True, pad=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ortho", "muon", "qk", "qk_grad"])
    if op == "ortho":
        most = work(listed()[3])["flops"]
        while True:
            c = dict(op=op, batch=_log(rng, 1, 64), rows=_log(rng, 8, 14336), cols=_log(rng, 8, 14336),
                     src=rng.choice(["bf16", "fp16", "fp32"]), dst=rng.choice(["bf16", "fp16"]))
            if rng.random() < 0.5:   # half of them multiples of 16, as most weights are; half odd
                c["rows"], c["cols"] = -(-c["rows"] // 80) * 80, -(-c["cols"] // 80) * 80
            else:
                c["rows"], c["cols"] = c["rows"] | 1, c["cols"] | 1
            if work(c)["flops"] <= most and c["batch"] * c["rows"] * c["cols"] <= 14336 * 4096:
                return c
    if op == "muon":
        most = work(listed()[6])
        while True:
            width = -(-_log(rng, 64, 2048) // 8) * 8
            layers, kv = _log(rng, 1, 24), width // rng.choice([1, 2, 4])
            ffn = -(-rng.choice([2, 3, 4]) * width // 80) * 80
            c = dict(op=op, shapes="%dx%dx%d,%dx%dx%d,%dx%dx%d,%dx%dx%d" % (
                width, width, 2 * layers, kv, width, 2 * layers, ffn, width, layers, width, ffn, layers),
                grad=rng.choice(["bf16", "fp16"]), scale=rng.choice([1.0, 256.0, 1024.0]))
            if 2 * work(c)["flops"] <= most["flops"] and 2 * work(c)["bytes"] <= most["bytes"]:
                return c
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    hk = rng.choice([1, 2, 4, 8])
    return dict(op=op, tokens=_log(rng, 1, 16384), hq=hk * rng.choice([1, 2, 4]), hk=hk, dim=dim,
                rot=rng.choice([dim, dim, dim // 2]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                gains=rng.choice(["head_dim", "per_head"]), inter=rng.random() < 0.3,
                fused=rng.random() < 0.5, pad=rng.choice([0.0, 0.0, 0.1]))


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _ortho_flops(rows, cols):
    # X X^T and A A are symmetric: one triangle each.  B X is not.
    k, l = min(rows, cols), max(rows, cols)
    return STEPS * (k * (k + 1) * l + k * (k + 1) * k + 2 * k * k * l)


def work(case):
    if case["op"] == "ortho":
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": n * (SIZE[case["src"]] + SIZE[case["dst"]]),
                "flops": case["batch"] * _ortho_flops(case["rows"], case["cols"])}
    if case["op"] == "muon":
        # gradient read; momentum and master read and written; 16-bit copy written
        return {"bytes": sum(b * r * c * (2 + 8 + 8 + 2) for r, c, b in _shapes(case)),
                "flops": sum(b * _ortho_flops(r, c) for r, c, b in _shapes(case))}
    heads = case["hq"] + case["hk"]
    row = heads * case["dim"] * SIZE[case["dtype"]]
    table = case["tokens"] * (case["rot"] * 4 + 8)
    gains = 2 * case["dim"] * 4 if case["gains"] == "head_dim" else heads * case["dim"] * 4
    if case["op"] == "qk":
        return {"bytes": case["tokens"] * 2 * row + table + gains,
                "flops": case["tokens"] * heads * case["dim"] * 8}
    return {"bytes": case["tokens"] * 3 * row + table + 2 * gains,
            "flops": case["tokens"] * heads * case["dim"] * 16}


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


def _matrices(gen, batch, rows, cols, sigma):
    """Gradients as a weight matrix gets them: a few strong directions that fall
    off, over noise that fills every direction."""
    r = max(1, min(32, min(rows, cols) // 4))
    s = 1.0 / torch.arange(1, r + 1, device="cuda", dtype=torch.float32)
    g = torch.matmul(_rand(gen, batch, rows, r) * s, _rand(gen, batch, r, cols))
    return g.add_(_rand(gen, batch, rows, cols), alpha=0.5).mul_(sigma)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 17)
    s = State(case)
    if case["op"] == "ortho":
        s.src = _matrices(gen, case["batch"], case["rows"], case["cols"], 1e-3).to(DTYPES[case["src"]])
        s.dst = torch.empty(s.src.shape, device="cuda", dtype=DTYPES[case["dst"]])
        if own:
            import zero_sharded_mixed_05_gb300 as z
            cfg = z.make_muon_config(steps=STEPS, coefs=ABC, eps=ORTHO_EPS)
            s.keep(z.zero_muon_create(cfg, [(case["rows"], case["cols"], case["batch"])]),
                   z.zero_muon_destroy)
        return s
    if case["op"] == "muon":
        s.mats = []
        for rows, cols, batch in _shapes(case):
            grad = _matrices(gen, batch, rows, cols, 1e-3)
            mom = _matrices(gen, batch, rows, cols, 5e-3).add_(grad, alpha=4.0)
            grad = grad.mul_(case["scale"]).to(DTYPES[case["grad"]])
            master = _rand(gen, batch, rows, cols).mul_(0.02)
            s.mats.append(dict(rows=rows, cols=cols, batch=batch, grad=grad, momentum=mom,
                               master=master, param16=master.to(DTYPES[case["grad"]])))
        if own:
            import zero_sharded_mixed_05_gb300 as z
            code = z.dtype_code(DTYPES[case["grad"]])
            cfg = z.make_muon_config(grad_dtype=code, lr=MUON["lr"], momentum=MUON["mu"],
                                     weight_decay=MUON["wd"], nesterov=True, steps=STEPS, coefs=ABC,
                                     eps=ORTHO_EPS, scale_rule=z.MUON_SCALE_RMS)
            s.keep(z.zero_muon_create(cfg, [(m["rows"], m["cols"], m["batch"]) for m in s.mats]),
                   z.zero_muon_destroy)
            s.list = z.make_muon_list(s.mats)
        return s
    T, hq, hk, D, rot = (case[k] for k in ("tokens", "hq", "hk", "dim", "rot"))
    dt = DTYPES[case["dtype"]]

    def heads(sigma):
        """Queries and keys: views of the projection's one output (with the
        values behind them) or tensors of their own."""
        if case["fused"]:
            qkv = (_rand(gen, T, hq + 2 * hk, D) * sigma).to(dt)
            return qkv[:, :hq], qkv[:, hq:hq + hk]
        return (_rand(gen, T, hq, D) * sigma).to(dt), (_rand(gen, T, hk, D) * sigma).to(dt)

    s.q, s.k = heads(1.3)
    lead = (lambda n: (n, D)) if case["gains"] == "per_head" else (lambda n: (D,))
    s.qg, s.kg = 1 + 0.2 * _rand(gen, *lead(hq)), 1 + 0.2 * _rand(gen, *lead(hk))
    n_pos = 1 << max(6, T.bit_length())
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * freq
    s.cos, s.sin = angle.cos().float(), angle.sin().float()
    # several sequences after one another, each from its own first position
    start = torch.randint(0, n_pos, (T // 256 + 1,), device="cuda", generator=gen)
    s.pos = (start.repeat_interleave(256)[:T] + torch.arange(T, device="cuda") % 256) % n_pos
    if case["pad"]:
        s.pos[torch.rand(T, device="cuda", generator=gen) < case["pad"]] = -1
    if case["op"] == "qk_grad":
        s.dqo, s.dko = (_rand(gen, T, hq, D) * 0.02).to(dt), (_rand(gen, T, hk, D) * 0.02).to(dt)
        s.dqg, s.dkg = torch.empty_like(s.qg), torch.empty_like(s.kg)
    s.qo, s.ko = torch.empty(T, hq, D, device="cuda", dtype=dt), torch.empty(T, hk, D, device="cuda", dtype=dt)
    if own:
        import zero_sharded_mixed_05_gb300 as z
        cfg = z.make_qk_config(q_heads=hq, k_heads=hk, head_dim=D, rotary_dim=rot,
                               dtype=z.dtype_code(dt), interleaved=case["inter"], eps=QK_EPS,
                               gain_per_head=case["gains"] == "per_head")
        s.keep(z.zero_qk_create(cfg), z.zero_qk_destroy)
    return s


# ---------------------------------------------------------------- plain forms

def _ortho_plain(g):
    x = g.float()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + ORTHO_EPS)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    a, b, c = ABC
    for _ in range(STEPS):
        A = x @ x.mT
        B = b * A + c * (A @ A)
        x = a * x + B @ x
    return x.mT if tall else x


def _muon_plain(m, scale):
    g = m["grad"].float() * (1.0 / scale)
    m["momentum"].mul_(MUON["mu"]).add_(g)
    o = _ortho_plain(g + MUON["mu"] * m["momentum"])
    step = MUON["lr"] * 0.2 * math.sqrt(max(m["rows"], m["cols"]))
    m["master"].mul_(1.0 - MUON["lr"] * MUON["wd"]).sub_(step * o)
    m["param16"].copy_(m["master"])
    return m["momentum"], m["master"], m["param16"]


def _pairs(x, rot, inter):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])


def _joined(a, b, rest, inter):
    both = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((both, rest), -1)


def _tables(s, kind=torch.float32):
    live = (s.pos >= 0)[:, None, None]
    at = s.pos.clamp(min=0)
    return live, s.cos[at].to(kind)[:, None], s.sin[at].to(kind)[:, None]


def _qk_plain(x, gain, s, live, cos, sin):
    rot, inter = s.case["rot"], s.case["inter"]
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + QK_EPS) * gain
    u, v = _pairs(y, rot, inter)
    out = _joined(u * cos - v * sin, v * cos + u * sin, y[..., rot:], inter)
    return torch.where(live, out, 0.0).to(s.q.dtype)


def _qk_grad_plain(dout, x, gain, s, live, cos, sin):
    rot, inter = s.case["rot"], s.case["inter"]
    x, dout = x.float(), torch.where(live, dout.float(), 0.0)
    u, v = _pairs(dout, rot, inter)
    dy = _joined(u * cos + v * sin, v * cos - u * sin, dout[..., rot:], inter)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + QK_EPS)
    xhat, dn = x * r, dy * gain
    dx = r * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
    return dx.to(s.q.dtype), (dy * xhat).sum(0 if gain.dim() == 2 else (0, 1))


# ---------------------------------------------------------------- one pass

def run(s):
    case = s.case
    if case["op"] == "ortho":
        if own:
            import zero_sharded_mixed_05_gb300 as z
            z.zero_muon_orthogonalize(s.handle, [s.src], [s.dst])
            return s.dst
        return _ortho_plain(s.src).to(s.dst.dtype)
    if case["op"] == "muon":
        if own:
            import zero_sharded_mixed_05_gb300 as z
            z.zero_muon_step(s.handle, s.list, grad_scale=1.0 / case["scale"])
            return [(m["momentum"], m["master"], m["param16"]) for m in s.mats]
        return [_muon_plain(m, case["scale"]) for m in s.mats]
    if case["op"] == "qk":
        if own:
            import zero_sharded_mixed_05_gb300 as z
            z.zero_qk_norm_rope(s.handle, s.q, s.k, s.qo, s.ko, s.qg, s.kg, s.cos, s.sin, s.pos)
            return s.qo, s.ko
        t = _tables(s)
        return _qk_plain(s.q, s.qg, s, *t), _qk_plain(s.k, s.kg, s, *t)
    if own:
        import zero_sharded_mixed_05_gb300 as z
        z.zero_qk_norm_rope_backward(s.handle, s.dqo, s.dko, s.q, s.k, s.qo, s.ko, s.dqg, s.dkg,
                                     s.qg, s.kg, s.cos, s.sin, s.pos)
        return s.qo, s.ko, s.dqg, s.dkg
    t = _tables(s)
    dq, dqg = _qk_grad_plain(s.dqo, s.q, s.qg, s, *t)
    dk, dkg = _qk_grad_plain(s.dko, s.k, s.kg, s, *t)
    return dq, dk, dqg, dkg


# ---------------------------------------------------------------- the definition in 64 bits

def _ortho_exact(g):
    """X <- (a I + b A + c A^2) X with A the Gram matrix of the shorter side,
    from the left for wide matrices and from the right for tall ones."""
    x = g.double()
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + ORTHO_EPS)
    tall = x.shape[-2] > x.shape[-1]
    a, b, c = ABC
    eye = torch.eye(min(x.shape[-2:]), device=x.device, dtype=torch.float64)
    for _ in range(STEPS):
        gram = x.mT @ x if tall else x @ x.mT
        p = a * eye + gram @ (b * eye + c * gram)
        x = x @ p if tall else p @ x
    return x


def _turn(x, s, sign):
    """The rotation as a product of complex numbers; `sign` -1 turns back."""
    rot, inter = s.case["rot"], s.case["inter"]
    at = s.pos.clamp(min=0)
    w = torch.complex(s.cos[at].double(), sign * s.sin[at].double())[:, None]
    z = torch.complex(*(t.contiguous() for t in _pairs(x, rot, inter))) * w
    out = x.clone()
    if inter:
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
    return out * (s.pos >= 0).double()[:, None, None]


def exact(case, seed):
    if case["op"] in ("ortho", "muon") and work(case)["flops"] > 8e12:
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "ortho":
        return _ortho_exact(s.src)
    if case["op"] == "muon":
        out = []
        for m in s.mats:
            g = m["grad"].double() / case["scale"]
            mom = MUON["mu"] * m["momentum"].double() + g
            o = _ortho_exact(g + MUON["mu"] * mom)
            step = MUON["lr"] * 0.2 * math.sqrt(max(m["rows"], m["cols"]))
            w = m["master"].double() * (1.0 - MUON["lr"] * MUON["wd"]) - step * o
            out.append((mom, w, w))
        return out

    def inverse_norm(x):
        return 1.0 / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["dim"] + QK_EPS) ** 0.5

    def forward(x, gain):
        x = x.double()
        return _turn(x * inverse_norm(x) * gain.double(), s, 1.0)

    def backward(dout, x, gain):
        x, dy = x.double(), _turn(dout.double(), s, -1.0)
        r = inverse_norm(x)
        dn = dy * gain.double()
        # d/dx of x r(x), with dr/dx = -r^3 x / dim
        dx = r * dn - r ** 3 * x * (dn * x).sum(-1, keepdim=True) / case["dim"]
        dg = (dy * x * r).sum(0)
        return dx, dg if gain.dim() == 2 else dg.sum(0)

    if case["op"] == "qk":
        return forward(s.q, s.qg), forward(s.k, s.kg)
    (dq, dqg), (dk, dkg) = backward(s.dqo, s.q, s.qg), backward(s.dko, s.k, s.kg)
    return dq, dk, dqg, dkg
