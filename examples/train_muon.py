"""A small decoder trained in fp16 with a dynamic loss scale: its matrices by
orthogonalised updates, everything else by AdamW, its queries and keys
normalised and rotated in one pass.

    python examples/train_muon.py [--steps 60] [--width 256] [--layers 2]

The optimizer's state is as the library's: flat 16-bit parameters and
gradients (the module's tensors are views of them), fp32 masters.  One step:

    statistics of the matrices' gradients -> device record 0
    statistics of the others'             -> device record 1
    zero_opt_step_folded   folds both, decides (skip, clip, loss scale) on the
                           device and updates the others
    zero_muon_step         updates the matrices by that decision

Only the loss scale and the printed loss are read back.  The data are sequences whose next token is
a fixed function of the two before, so the loss falls from log(vocabulary).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_mixed_05_gb300 as z  # noqa: E402
from zero_sharded_mixed_05_gb300.qk import QkNormRope, rotation_tables  # noqa: E402

VOCAB, HEAD = 64, 64


class Flat:
    """16-bit parameters and gradients of some tensors in two flat buffers."""

    def __init__(self, params):
        self.params = params
        n = sum(p.numel() for p in params)
        dev = params[0].device
        self.param16 = torch.empty(n, dtype=torch.float16, device=dev)
        self.grad = torch.zeros(n, dtype=torch.float16, device=dev)
        at = 0
        for p in params:
            view = slice(at, at + p.numel())
            self.param16[view] = p.data.flatten().half()
            p.data = self.param16[view].view(p.shape)
            p.grad = self.grad[view].view(p.shape)
            at += p.numel()
        self.master = self.param16.float()

    def of(self, p, flat):
        at = (p.data_ptr() - self.param16.data_ptr()) // 2
        return flat[at:at + p.numel()].view(p.shape)


class Decoder:
    """Pre-norm decoder blocks; matrices [outputs, inputs]."""

    def __init__(self, width, layers, dev):
        g = torch.Generator(device=dev).manual_seed(1)
        self.q_heads, self.k_heads = width // HEAD, max(1, width // HEAD // 2)
        kv = self.k_heads * HEAD

        def mat(rows, cols):
            w = torch.randn(rows, cols, generator=g, device=dev) * cols ** -0.5
            return w.requires_grad_()

        def vec(n, value=1.0):
            return torch.full((n,), value, device=dev).requires_grad_()
        self.blocks = [dict(qkv=mat(width + 2 * kv, width), out=mat(width, width),
                            up=mat(4 * width, width), down=mat(width, 4 * width),
                            norm1=vec(width), norm2=vec(width), q_gain=vec(HEAD), k_gain=vec(HEAD))
                       for _ in range(layers)]
        self.embed = (torch.randn(VOCAB, width, generator=g, device=dev) * 0.5).requires_grad_()
        self.head = (torch.randn(VOCAB, width, generator=g, device=dev) * width ** -0.5).requires_grad_()
        self.final = vec(width)
        self.norm = QkNormRope(z.make_qk_config(self.q_heads, self.k_heads, HEAD, dtype=z.FP16))

    def matrices(self):
        return [b[n] for b in self.blocks for n in ("qkv", "out", "up", "down")]

    def others(self):
        return [self.embed, self.head, self.final] + \
            [b[n] for b in self.blocks for n in ("norm1", "norm2", "q_gain", "k_gain")]

    def loss(self, tokens, cos, sin):
        batch, length = tokens.shape[0], tokens.shape[1] - 1
        pos = torch.arange(length, device=tokens.device).repeat(batch)
        x = F.embedding(tokens[:, :-1].reshape(-1), self.embed)
        for b in self.blocks:
            h = F.rms_norm(x, (x.shape[-1],), b["norm1"])
            qkv = (h @ b["qkv"].T).view(batch * length, -1, HEAD)
            q, k, v = qkv.split([self.q_heads, self.k_heads, self.k_heads], 1)
            q, k = self.norm(q, k, b["q_gain"].float(), b["k_gain"].float(), cos, sin, pos)

            def heads(t):
                t = t.view(batch, length, -1, HEAD).transpose(1, 2)
                return t.repeat_interleave(self.q_heads // t.shape[1], 1)
            a = F.scaled_dot_product_attention(heads(q), heads(k), heads(v), is_causal=True)
            x = x + a.transpose(1, 2).reshape(batch * length, -1) @ b["out"].T
            h = F.rms_norm(x, (x.shape[-1],), b["norm2"])
            x = x + F.gelu(h @ b["up"].T) @ b["down"].T
        logits = F.rms_norm(x, (x.shape[-1],), self.final) @ self.head.T
        return F.cross_entropy(logits.float(), tokens[:, 1:].reshape(-1))


def batch_of(gen, batch, length, dev):
    t = torch.randint(0, VOCAB, (batch, length + 1), device=dev, generator=gen)
    for i in range(2, length + 1):
        t[:, i] = (3 * t[:, i - 1] + 5 * t[:, i - 2] + 1) % VOCAB
    return t


def train(steps=60, width=256, layers=2, lr=4e-3, quiet=False):
    """Losses of every step."""
    dev = torch.device("cuda", torch.cuda.current_device())
    model = Decoder(width, layers, dev)
    mats, rest = Flat(model.matrices()), Flat(model.others())
    n = rest.master.numel()
    opt = z.zero_opt_create(z.make_config(numel=n, grad_dtype=z.FP16, lr=lr, weight_decay=0.0,
                                          max_grad_norm=1.0, dynamic_scale=True, init_scale=2.0 ** 12,
                                          scale_window=100))
    m, v = torch.zeros_like(rest.master), torch.zeros_like(rest.master)
    bufs = z.make_buffers(rest.master, m, v, rest.param16, [rest.grad], grads_shard_local=True)
    muon = z.zero_muon_create(z.make_muon_config(grad_dtype=z.FP16, lr=lr, scale_rule=z.MUON_SCALE_RMS),
                              [tuple(p.shape) for p in mats.params])
    momentum = torch.zeros_like(mats.master)
    items = z.make_muon_list([dict(grad=p.grad, momentum=mats.of(p, momentum),
                                   master=mats.of(p, mats.master), param16=p.data)
                              for p in mats.params])
    records = torch.zeros(4, dtype=torch.float64, device=dev)     # two zero_opt_stats
    decision = z.zero_opt_decision(opt)
    cos, sin = rotation_tables(128, HEAD, device=dev)
    gen = torch.Generator(device=dev).manual_seed(2)
    losses = []
    try:
        for step in range(steps):
            scale = z.zero_opt_loss_scale(opt, 0).scale
            mats.grad.zero_()
            rest.grad.zero_()
            loss = model.loss(batch_of(gen, 16, 96, dev), cos, sin)
            (loss * scale).backward()
            z.zero_opt_grad_stats_noalloc([mats.grad], z.FP16, mats.grad.numel(), records[:2])
            z.zero_opt_grad_stats_async(opt, 0, bufs, records[2:])
            z.zero_opt_step_folded(opt, 0, bufs, records, 2)
            z.zero_muon_step(muon, items, decision=decision)
            losses.append(float(loss.detach()))
            if step % 10 and step != steps - 1:
                continue
            if z.zero_muon_fault_count(muon):
                raise RuntimeError("a step of the matrices ended in a fault")
            if not quiet:
                info = z.zero_opt_last_step(opt)
                print(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norm {info.norm:.3f}  "
                      f"loss scale {info.scale_used:g}{'  skipped' if info.skipped else ''}")
    finally:
        z.zero_muon_destroy(muon)
        z.zero_opt_destroy(opt)
        model.norm.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--lr", type=float, default=4e-3)
    a = ap.parse_args()
    train(a.steps, a.width, a.layers, a.lr)
