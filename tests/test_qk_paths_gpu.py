"""The query/key norm's kernels path by path: what decides between them is in
csrc/qk.cu (run), and the sizes here are chosen by it.  Definitions and
tolerances are those of test_qk_gpu.py."""
import pytest

from test_qk_gpu import backward64, forward64, handle, make, near, z  # noqa: F401

pytestmark = pytest.mark.gpu


def at_offset(t, numbers):
    """The same numbers at an address `numbers` past a multiple of 512 bytes."""
    import torch
    flat = torch.empty(t.numel() + numbers, device=t.device, dtype=t.dtype)
    flat[numbers:] = t.flatten()
    return flat[numbers:].view(t.shape)


@pytest.mark.parametrize("numbers", [1, 2, 4, 8, 12])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("name", ["bf16", "fp32"])
def test_gains_and_tables_at_any_address(z, numbers, per_head, name):  # noqa: F811
    """Views of a flat parameter buffer, aligned to 4 to 32 bytes only, give
    what the formula gives (the width of the loads goes by the address)."""
    import torch
    case = (9, 4, 2, 128, 128, name, False, per_head, "own")
    q, k, qg, kg, cos, sin, pos = make(case, 21)
    gq, gk = make(case, 22)[:2]
    h = handle(z, case)
    try:
        args = [at_offset(t, numbers) for t in (qg, kg, cos, sin)] + [pos]
        assert args[0].data_ptr() % 64 == 4 * numbers
        qo, ko, dq, dk = (torch.full_like(t, float("nan")) for t in (q, k, q, k))
        dqg, dkg = at_offset(torch.full_like(qg, float("nan")), numbers), torch.empty_like(kg)
        z.zero_qk_norm_rope(h, q, k, qo, ko, *args)
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, dq, dk, dqg, dkg, *args)
        for got, d, dg, x, go, gain in ((qo, dq, dqg, q, gq, qg), (ko, dk, dkg, k, gk, kg)):
            ref = forward64(x, gain, pos, cos, sin, 128, False)
            near(got, ref, ref.abs().amax(-1, keepdim=True), name, 128)
            ref, mag, terms = backward64(go, x, gain, pos, cos, sin, 128, False)
            near(d, ref, mag, name, 128)
            dims = 0 if per_head else (0, 1)
            n = x.shape[0] if per_head else x.shape[0] * x.shape[1]
            scale = terms.abs().amax(-1, keepdim=True).expand_as(terms)
            tol = (n + 128 + 16) * 2.0 ** -24 * scale.sum(dims)
            assert ((dg.double() - terms.sum(dims)).abs() <= tol).all()
    finally:
        z.zero_qk_destroy(h)


@pytest.mark.parametrize("name", ["bf16", "fp32"])
@pytest.mark.parametrize("per_head", [False, True])
def test_gradients_of_rows_of_any_size(z, name, per_head, monkeypatch):  # noqa: F811
    """With eps 0 the rows' root mean square may be anything whose square
    binary32 holds: dx is of the size of its inverse, whose cube is not held."""
    import test_qk_gpu
    import torch
    monkeypatch.setattr(test_qk_gpu, "EPS", 0.0)
    case = (11, 4, 2, 64, 64, name, False, per_head, "own")
    q, k, qg, kg, cos, sin, pos = make(case, 31)
    gq, gk = make(case, 32)[:2]
    pos = pos.clamp(min=0)
    size = 10.0 ** torch.arange(-15, 18, 3, device="cuda").double()
    q, k = ((t.double() * size[:, None, None]).to(t.dtype) for t in (q, k))
    h = handle(z, case)
    try:
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        dqg, dkg = torch.empty_like(qg), torch.empty_like(kg)
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, dq, dk, dqg, dkg, qg, kg, cos, sin, pos)
        for d, dg, x, go, gain in ((dq, dqg, q, gq, qg), (dk, dkg, k, gk, kg)):
            ref, mag, terms = backward64(go, x, gain, pos, cos, sin, 64, False)
            near(d, ref, mag, name, 64)
            dims = 0 if per_head else (0, 1)
            scale = terms.abs().amax(-1, keepdim=True).expand_as(terms)
            tol = (11 * x.shape[1] + 64 + 16) * 2.0 ** -24 * scale.sum(dims)
            assert ((dg.double() - terms.sum(dims)).abs() <= tol).all()
    finally:
        z.zero_qk_destroy(h)


def test_gradient_of_a_zero_row_with_a_small_eps(z, monkeypatch):  # noqa: F811
    import test_qk_gpu
    import torch
    monkeypatch.setattr(test_qk_gpu, "EPS", 1e-30)
    case = (3, 2, 1, 64, 64, "fp32", False, False, "own")
    q, k, qg, kg, cos, sin, pos = make(case, 33)
    gq, gk = make(case, 34)[:2]
    q[1] = 0
    pos[:] = torch.tensor([4, 5, 6], device="cuda")
    h = handle(z, case)
    try:
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, dq, dk, None, None, qg, kg, cos, sin, pos)
        ref, mag, _ = backward64(gq, q, qg, pos, cos, sin, 64, False)
        near(dq, ref, mag, "fp32", 64)
    finally:
        z.zero_qk_destroy(h)


# More tokens than a wave of groups: each walks several, through both places of
# its ring and the next token's angles; two and four heads a group where head
# counts divide and rows are enough (19,456 and 38,912 of 128 numbers in 16 bits).
MANY = [
    (4500, 32, 8, 128, 128, "bf16", False, False, "fused"),     # four heads a group; backward two, summed together
    (4501, 32, 8, 128, 128, "fp16", True, True, "fused"),       # a gain a head
    (3500, 6, 2, 128, 64, "bf16", False, False, "own"),         # two heads, half of each turned
    (4200, 32, 8, 64, 64, "bf16", False, False, "heads_first"),
    (2300, 16, 16, 128, 128, "fp32", False, False, "own"),      # two heads of binary32
    (2100, 16, 4, 256, 256, "fp32", True, True, "fused"),
    (4300, 12, 12, 80, 40, "fp16", True, False, "fused"),       # 8-byte vectors
    (4300, 12, 4, 96, 48, "bf16", False, True, "fused"),
    (2500, 20, 4, 128, 128, "bf16", False, False, "odd"),       # single numbers
    (2500, 5, 3, 66, 34, "fp32", False, True, "odd"),
    (15000, 4, 0, 128, 128, "bf16", False, False, "own"),       # queries alone
    (12001, 1, 1, 128, 128, "bf16", False, False, "fused"),     # heads that do not divide
]


@pytest.mark.parametrize("case", MANY, ids=str)
def test_many_tokens(z, case):  # noqa: F811
    import test_qk_gpu
    import torch
    test_qk_gpu.test_forward(z, case, False)
    if case[2] > 0:
        return test_qk_gpu.test_backward(z, case)
    # queries alone: what belongs to keys is not looked at
    T, hq, _, D, rot, name, inter, per_head, _ = case
    q, _, qg, _, cos, sin, pos = make(case, 2)
    go = make(case, 3)[0]
    h = handle(z, case)
    try:
        runs = []
        for _ in range(2):
            dq, dqg = torch.full_like(q, float("nan")), torch.full_like(qg, float("nan"))
            z.zero_qk_norm_rope_backward(h, go, None, q, None, dq, None, dqg, None, qg, None, cos, sin, pos)
            runs.append((dq, dqg))
        ref, mag, terms = backward64(go, q, qg, pos, cos, sin, rot, inter)
        near(dq, ref, mag, name, D)
        scale = terms.abs().amax(-1, keepdim=True).expand_as(terms)
        tol = (T * hq + D + 16) * 2.0 ** -24 * scale.sum((0, 1))
        assert ((dqg.double() - terms.sum((0, 1))).abs() <= tol).all()
        assert all(torch.equal(a, b) for a, b in zip(*runs))
    finally:
        z.zero_qk_destroy(h)


@pytest.mark.parametrize("head,token", [(64, 110_000_000), (1_100_000_000, 64)])
def test_strides_past_32_bits(z, head, token):  # noqa: F811
    """Tokens or heads more than 2^31 numbers from the first."""
    import torch
    case = (40, 4, 1, 64, 64, "bf16", False, False, "own")
    q, k, qg, kg, cos, sin, pos = make(case, 41)
    gq, gk = make(case, 42)[:2]
    store = torch.empty(4_500_000_000, device="cuda", dtype=torch.bfloat16)
    h = handle(z, case)
    try:
        def spread(t):
            far = store.as_strided(t.shape, (token, head, 1), 8)
            far.copy_(t)
            return far
        qo, ko, q1, k1 = (torch.empty_like(t) for t in (q, k, q, k))
        z.zero_qk_norm_rope(h, q, k, qo, ko, qg, kg, cos, sin, pos)
        far = spread(q)
        z.zero_qk_norm_rope(h, far, k, far, k1, qg, kg, cos, sin, pos)
        assert torch.equal(far, qo) and torch.equal(k1, ko)
        z.zero_qk_norm_rope_backward(h, gq, gk, q, k, q1, k1, None, None, qg, kg, cos, sin, pos)
        far = spread(gq)
        z.zero_qk_norm_rope_backward(h, far, gk, q, k, far, ko, None, None, qg, kg, cos, sin, pos)
        assert torch.equal(far, q1) and torch.equal(ko, k1)
    finally:
        z.zero_qk_destroy(h)
        del store, far
        torch.cuda.empty_cache()
