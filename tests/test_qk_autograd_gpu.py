"""The autograd wrapper of the query/key norm on the GPU, in attention written
with plain products."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gains", ["both", "none", "keys"])
@pytest.mark.parametrize("how", ["einsum", "matmul"])
def test_attention_of_plain_products(how, gains):
    """Against torch's autograd on the formula in 64 bits, the callable gone
    before the backward pass.  Everything is binary32 with sums of at most
    T * heads * D = 2560 terms of size below 8 on either side, which the
    softmax passes on divided by about T."""
    import torch
    import zero_sharded_mixed_05_gb300 as z
    from zero_sharded_mixed_05_gb300.qk import QkNormRope, rotation_tables
    T, H, D = 20, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(T, H, D, device="cuda", generator=gen) for _ in range(3))
    qg, kg = (1 + 0.1 * torch.randn(D, device="cuda", generator=gen) for _ in range(2))
    cos, sin = rotation_tables(64, D)
    pos = torch.arange(T, device="cuda") + 5

    def attention(q, k, v):
        if how == "einsum":
            return torch.einsum("qhd,khd->hqk", q, k).div(8).softmax(-1) @ v.transpose(0, 1)
        return (q.transpose(0, 1) @ k.permute(1, 2, 0) / 8).softmax(-1) @ v.transpose(0, 1)

    def plain(x, gain):
        y = x * (x.square().mean(-1, keepdim=True) + 1e-6) ** -0.5
        y = y if gain is None else y * gain
        c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)
    given = {"both": (qg, kg), "none": (None, None), "keys": (None, kg)}[gains]
    leaves = [t if t is None else t.clone().requires_grad_() for t in (q, k, *given)]
    norm = QkNormRope(z.make_qk_config(H, H, D, dtype=z.FP32))
    out = attention(*norm(*leaves, cos, sin, pos), v)
    del norm
    out.square().sum().backward()
    wide = [t if t is None else t.double().requires_grad_() for t in (q, k, *given)]
    attention(plain(wide[0], wide[2]), plain(wide[1], wide[3]), v.double()).square().sum().backward()
    # the attention's own products are torch's, in binary32
    assert not torch.backends.cuda.matmul.allow_tf32
    for a, b in zip(leaves, wide):
        if a is not None:
            assert ((a.grad.double() - b.grad).abs() <= T * H * D * 2.0 ** -24 * 8).all()
