"""The query/key norm at the edges of what its documentation allows, on the GPU."""
import pytest

from test_qk_gpu import tables, z  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-12, 1e-30, 1e-44, 1e-50, 1e-300])
@pytest.mark.parametrize("axes", [False, True])
def test_rows_of_zeros_by_any_eps(z, axes, eps):  # noqa: F811
    """Zero over the root of any eps that is not zero is zero; so are the gradients
    of zeros, by eps as large as they are finite."""
    import torch
    T, D = 9, 64
    cfg = z.make_qk_config(2, 1, D, D, z.FP32, False, eps)
    h = z.zero_qk_create(cfg, z.make_qk_axes([0] * (D // 2))) if axes else z.zero_qk_create(cfg)
    cos, sin = tables(16, D)
    pos = torch.arange(T, device="cuda")
    if axes:
        pos = pos[None]
    q, k = (torch.zeros(T, n, D, device="cuda") for n in (2, 1))
    qo, ko = torch.ones_like(q), torch.ones_like(k)
    z.zero_qk_norm_rope(h, q, k, qo, ko, None, None, cos, sin, pos)
    assert not qo.any() and not ko.any()
    z.zero_qk_norm_rope_backward(h, q, k, q, k, qo, ko, None, None, None, None, cos, sin, pos)
    assert not qo.any() and not ko.any()
    z.zero_qk_destroy(h)
