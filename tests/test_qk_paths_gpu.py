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
