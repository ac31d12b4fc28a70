"""The orthogonalised update's kernels path by path: what decides between them
is in csrc/muon.cu (choose_resident, products_cost, splits_of), and the sizes
here are chosen by it.  Definitions and tolerances are those of test_muon_gpu.py."""
import pytest

from test_muon_gpu import close, ortho64, spectrum, z  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,b", [(128, 400, 60), (900, 100, 36), (128, 2048, 18)])
def test_a_clusters_ctas_agree_call_after_call(z, m, n, b):  # noqa: F811
    """Clusters of two, four and eight CTAs, which send one another their parts
    of A while they go on to B: the same matrix in every place of the batch
    gives the same bits, in every call."""
    import torch
    g = spectrum("signal", 1, m, n, torch.Generator(device="cuda").manual_seed(n)).repeat(b, 1, 1)
    h = z.zero_muon_create(z.make_muon_config(), [(m, n, b)])
    try:
        first = torch.empty_like(g)
        z.zero_muon_orthogonalize(h, [g], [first])
        close(first, ortho64(g), "fp32")
        differ = torch.zeros((), device="cuda", dtype=torch.int64)
        out = torch.empty_like(g)
        for _ in range(60):
            z.zero_muon_orthogonalize(h, [g], [out])
            differ += (out != first[:1]).sum()
        assert int(differ) == 0
        assert z.zero_muon_last_step(h).fault == 0
    finally:
        z.zero_muon_destroy(h)
