"""The autograd wrapper of the query/key norm, with the formula in binary64 in
the kernels' place and the checks of the binding in front of it."""
import gc

import pytest
import torch

EPS = 1e-6


def turn(x, cos, sin, pos, sign):
    half = x.shape[-1] // 2
    c, s = cos.double()[pos][:, None], sign * sin.double()[pos][:, None]
    u, v = x[..., :half], x[..., half:]
    return torch.cat((u * c - v * s, v * c + u * s), -1)


def plain(x, gain, cos, sin, pos):
    y = x * (x.square().mean(-1, keepdim=True) + EPS) ** -0.5
    return turn(y if gain is None else y * gain, cos, sin, pos, 1.0)


def plain_grad(go, x, gain, cos, sin, pos):
    x, dy = x.double(), turn(go.double(), cos, sin, pos, -1.0)
    r = (x.square().mean(-1, keepdim=True) + EPS) ** -0.5
    dn = dy if gain is None else dy * gain.double()
    return r * (dn - x * r * (dn * x * r).mean(-1, keepdim=True)), (dy * x * r).sum((0, 1))


class Calls:
    """What the binding is asked for, checked as it checks it, and the formula."""

    def __init__(self):
        self.live, self.handles, self.summed = {}, 0, []

    def create(self, cfg):
        self.handles += 1
        self.live[self.handles] = (cfg.q_heads, cfg.k_heads, cfg.head_dim)
        return self.handles

    def destroy(self, h):
        del self.live[h]

    def check(self, h, q, k, *others):
        if h not in self.live:
            raise ValueError("not a handle of zero_qk_create")
        for name, t, heads in [("q", q, 0), ("k", k, 1)] + [(n, t, i % 2) for i, (n, t) in enumerate(others)]:
            shape = (q.shape[0], self.live[h][heads], self.live[h][2])
            if t.dtype is not torch.float32 or t.shape != shape or t.stride(-1) != 1:
                raise ValueError(f"{name} must be a float32 tensor of {shape} with contiguous heads")

    def forward(self, h, q, k, qo, ko, qg, kg, cos, sin, pos, stream=None):
        self.check(h, q, k, ("q_out", qo), ("k_out", ko))
        qo.copy_(plain(q.double(), qg, cos, sin, pos))
        ko.copy_(plain(k.double(), kg, cos, sin, pos))

    def backward(self, h, dqo, dko, q, k, dq, dk, dqg, dkg, qg, kg, cos, sin, pos, stream=None):
        self.check(h, q, k, ("dq_out", dqo), ("dk_out", dko), ("dq", dq), ("dk", dk))
        self.summed.append((dqg is not None, dkg is not None))
        for go, x, d, dg, gain in ((dqo, q, dq, dqg, qg), (dko, k, dk, dkg, kg)):
            dx, sums = plain_grad(go, x, gain, cos, sin, pos)
            d.copy_(dx)
            if dg is not None:
                dg.copy_(sums)


@pytest.fixture()
def calls(monkeypatch):
    import zero_sharded_mixed_05_gb300.qk as qk
    c = Calls()
    for name, fn in (("zero_qk_create", c.create), ("zero_qk_destroy", c.destroy), ("zero_qk_norm_rope", c.forward),
                     ("zero_qk_norm_rope_backward", c.backward)):
        monkeypatch.setattr(qk, name, fn)
    yield c
    for o in gc.get_objects():             # a failed test's: no handle of the library's
        if type(o) is qk.QkNormRope:
            o._handle = None


T, HQ, HK, D = 9, 4, 4, 8


def norm_of():
    import zero_sharded_mixed_05_gb300.qk as qk
    return qk.QkNormRope(qk.make_qk_config(HQ, HK, D, dtype=2))


def inputs(seed=1):
    import zero_sharded_mixed_05_gb300.qk as qk
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(T, h, D, generator=g).requires_grad_() for h in (HQ, HK))
    qg, kg = ((1 + 0.1 * torch.randn(D, generator=g)).requires_grad_() for _ in range(2))
    cos, sin = qk.rotation_tables(16, D, device="cpu")
    return q, k, qg, kg, cos, sin, torch.arange(T) + 3


def test_second_derivatives_are_refused(calls):
    """The backward kernel has no derivative of its own: an error, not a
    gradient without its share."""
    q, k, qg, kg, *rest = inputs()
    norm = norm_of()
    qo, ko = norm(q, k, qg, kg, *rest)
    dq, = torch.autograd.grad((qo * ko).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        (dq.square().sum() + q.sum()).backward()


@pytest.mark.parametrize("how", ["einsum", "matmul", "expanded", "sliced"])
def test_gradients_in_any_order(calls, how):
    """What attention and reductions send back: permuted, broadcast and cut
    gradients, against autograd on the formula."""
    ins = inputs(2)
    ref = [t.detach().double().requires_grad_() for t in ins[:4]]

    def loss(q, k):
        if how == "einsum":
            return torch.einsum("qhd,khd->hqk", q, k).softmax(-1).square().sum()
        if how == "matmul":
            return (q.transpose(0, 1) @ k.permute(1, 2, 0)).tanh().sum()
        if how == "expanded":
            return q.sum() * k.mean()
        return (q[1:, :2] * k[:-1, 2:]).sum()
    norm = norm_of()
    loss(*norm(*ins)).backward()
    loss(*(plain(x, gain, *ins[4:]) for x, gain in ((ref[0], ref[2]), (ref[1], ref[3])))).backward()
    for a, b in zip(ins[:4], ref):
        # binary32 results of sums of T * heads * D terms of size one
        assert ((a.grad.double() - b.grad).abs() <= T * HQ * D * 2.0 ** -22).all()


def test_gains_of_ones_and_gains_that_do_not_learn(calls):
    """A gain may be None, as in the call itself; sums are made for those that
    take a gradient alone."""
    q, k, qg, kg, *rest = inputs(3)
    norm = norm_of()
    for gains, summed in (((None, None), (False, False)), ((qg.detach(), kg), (False, True)),
                          ((qg, None), (True, False)), ((qg, kg), (True, True))):
        ins = [t.detach().clone().requires_grad_() for t in (q, k)]
        ref = [t.detach().double().requires_grad_() for t in (q, k)]
        for t in (qg, kg):
            t.grad = None
        qo, ko = norm(*ins, *gains, *rest)
        (qo * ko).sum().backward()
        assert calls.summed[-1] == summed
        wide = [None if t is None else t.detach().double().requires_grad_() for t in gains]
        (plain(ref[0], wide[0], *rest) * plain(ref[1], wide[1], *rest)).sum().backward()
        for a, b in zip(ins, ref):
            assert ((a.grad.double() - b.grad).abs() <= D * 2.0 ** -20).all()
        for t, w, s in zip(gains, wide, summed):
            if s:
                assert ((t.grad.double() - w.grad).abs() <= T * HQ * D * 2.0 ** -22).all()
            elif t is not None:
                assert t.grad is None


def test_the_handle_lives_as_long_as_a_graph_needs_it(calls):
    """The callable may be gone before the backward pass; its handle is
    destroyed once, after it."""
    *ins, cos, sin, pos = inputs(4)
    norm = norm_of()
    qo, ko = norm(*ins, cos, sin, pos)
    del norm
    gc.collect()
    assert len(calls.live) == 1
    (qo * ko).sum().backward()
    assert ins[0].grad is not None and ins[2].grad is not None
    del qo, ko
    gc.collect()
    assert not calls.live
    # closed by hand is closed
    norm = norm_of()
    qo, ko = norm(*ins, cos, sin, pos)
    norm.close()
    assert not calls.live
    with pytest.raises(ValueError):
        (qo * ko).sum().backward()
