"""The join of a block with the residual stream, and dropout, from their
formulas in 64 bits, with the magnitudes that binary32 arithmetic's errors are
relative to.  Plain torch and numpy; the generator is numpy's 64-bit products."""
import numpy as np

U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
E32 = 2.0 ** -24
EPS = 1e-6


def dt(name):
    import torch
    return dict(fp16=torch.float16, bf16=torch.bfloat16, fp32=torch.float32)[name]


def philox(c, k, rounds=10):
    """Four words [n] each of counters c (4 arrays) and key k (2 numbers)."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, np.uint64) for v in c]
    k0, k1 = (np.uint64(v) for v in k)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        s = np.uint64(32)
        c = [(p1 >> s) ^ c[1] ^ k0, p1 & m, (p0 >> s) ^ c[3] ^ k1, p0 & m]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & m, (k1 + np.uint64(0xBB67AE85)) & m
    return c


def cut_of(p):
    return int(np.floor(65536 * p + 0.5))


def kept(rows, dim, p, seed=0, call=0, step=0, first_row=0):
    """bool [rows, dim]: which numbers stay."""
    per = -(-dim // 8)
    block = (np.arange(rows * per, dtype=np.uint64) + np.uint64(first_row * per))
    w = philox([block & np.uint64(0xFFFFFFFF), block >> np.uint64(32), np.full_like(block, call),
                np.full_like(block, step & 0xFFFFFFFF)], (seed & 0xFFFFFFFF, seed >> 32))
    halves = np.stack([h for v in w for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], -1)
    return halves.reshape(rows, per * 8)[:, :dim] >= cut_of(p)


def factor(p):
    c = cut_of(p)
    return 65536.0 / (65536.0 - c) if c < 65536 else 0.0


class Ref:
    """One join of given inputs (torch tensors; y, gate, mask may be None)."""

    def __init__(self, x, y, y_gain, gain, gate=None, kind="none", post=False, pre=True, alpha=1.0,
                 beta=1.0, p=0.0, mask=None, rng=(0, 0, 0)):
        import torch
        self.post, self.pre, self.alpha, self.beta, self.kind = post, pre, alpha, beta, kind
        D = x.shape[1]
        self.D = D
        live = torch.ones(x.shape[0], dtype=torch.bool, device=x.device) if mask is None else mask.bool()
        self.live = live[:, None]
        ones = torch.ones(D, dtype=torch.float64, device=x.device)
        self.x = self.only(x.double())
        self.gain = ones if gain is None else gain.double()
        self.y_gain = ones if y_gain is None else y_gain.double()
        self.y = None if y is None else self.only(y.double())
        self.act, self.slope = 1.0, 0.0
        if gate is not None and kind != "none":
            g = self.only(gate.double())
            self.act = g if kind == "plain" else torch.sigmoid(g)
            self.slope = torch.ones_like(g) if kind == "plain" else self.act * (1 - self.act)
        self.keep = torch.ones(x.shape, dtype=torch.bool, device=x.device)
        if p > 0 and y is not None:
            k = kept(*x.shape, p, *rng)
            self.keep = torch.from_numpy(k).to(x.device)
        self.scale = beta * factor(p) if p < 1 else 0.0

    def only(self, t):
        import torch
        return torch.where(self.live, t, torch.zeros_like(t))

    def dropped(self, t):
        import torch
        return torch.where(self.keep, t, torch.zeros_like(t)) * self.scale

    def inv(self, t):
        return (t.square().mean(-1, keepdim=True) + EPS) ** -0.5

    def forward(self):
        """(x', h, tolerances of their binary32 arithmetic)."""
        n = self.D + 32
        if self.y is None:
            x, mag = self.x, self.x.abs()
        else:
            yhat = self.y * self.inv(self.y) if self.post else self.y
            b = self.dropped(yhat * self.y_gain * self.act)
            x = self.only(self.alpha * self.x + b)
            mag = self.only((self.alpha * self.x).abs() + b.abs())
        r = self.inv(x)
        h = self.only(x * r * self.gain)
        # r's own error: of the sum of squares and of what went into it
        rel = n * E32 * (1 + (mag * x.abs()).sum(-1, keepdim=True) /
                         (x.square().sum(-1, keepdim=True) + self.D * EPS))
        tol_x = (n * E32 * mag if self.y is not None else mag * 0)
        return x, h, tol_x, (n * E32 * mag * r + rel * (x * r).abs()) * self.gain.abs()

    def backward(self, x_out, dx_out, dh):
        """dict of results and of tolerances of their binary32 arithmetic."""
        import torch
        n, T = self.D + 48, x_out.shape[0]
        x = self.only(x_out.double())
        zero = torch.zeros_like(x)
        dxo = zero if dx_out is None else self.only(dx_out.double())
        dh = zero if dh is None else self.only(dh.double())
        r = self.inv(x)
        xhat, dn = x * r, dh * self.gain
        G = dxo + r * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
        magG = dxo.abs() + r * (dn.abs() + xhat.abs() * (dn * xhat).abs().mean(-1, keepdim=True))
        alpha = self.alpha if self.y is not None else 1.0
        out = dict(dx=alpha * G, dgain=(dh * xhat).sum(0))
        tol = dict(dx=abs(alpha) * n * E32 * magG, dgain=(T + n) * E32 * (dh * xhat).abs().sum(0))
        if self.y is None:
            return out, tol
        ry = self.inv(self.y) if self.post else torch.ones_like(r)
        yhat = self.y * ry
        db, mdb = self.dropped(G), self.dropped(magG).abs()
        act = self.act if isinstance(self.act, float) else self.act
        dz, mdz = db * act, mdb * abs(act)
        t, mt = dz * self.y_gain, mdz * self.y_gain.abs()
        dy, mdy = t, mt
        if self.post:
            dy = ry * (t - yhat * (t * yhat).mean(-1, keepdim=True))
            mdy = ry * (mt + yhat.abs() * (mt * yhat.abs()).mean(-1, keepdim=True))
        out.update(dy=dy, dy_gain=(dz * yhat).sum(0), dgate=db * yhat * self.y_gain * self.slope)
        tol.update(dy=2 * n * E32 * mdy, dy_gain=(T + 2 * n) * E32 * (mdz * yhat.abs()).sum(0),
                   dgate=2 * n * E32 * mdb * (yhat * self.y_gain).abs())
        return out, tol


def near(got, ref, tol, name, what=""):
    """Within half a step of the type, and the arithmetic's tolerance."""
    tol = U[name] * ref.abs() + tol * 1.001
    if name == "fp16":
        tol = tol + 2.0 ** -25
    d = (got.double() - ref).abs()
    assert (d <= tol).all(), (what, (d / tol.clamp_min(1e-300)).max().item())
