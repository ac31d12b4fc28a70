"""Calls of the join at the edges of what its documentation allows, on the GPU
against the formulas in 64 bits.  Tolerances are test_block_gpu.py's where none
is given."""
import pytest

import block_ref as R
from test_block_gpu import Case, blank, rows, z  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [512, 517])
@pytest.mark.parametrize("fill", ["nan", "inf"])
def test_the_norm_alone_does_not_see_the_branch_s_gain(z, D, fill):  # noqa: F811
    import torch
    c = Case(z, (300, D, "bf16", "fp32", False, True, "none", 0.0, 0.2, "own", 1.0, 1.0, False), 20)
    c.y_gain = None
    want = (c.forward()[1], *c.backward(c.x).values())
    c.y_gain = torch.full((D,), float(fill), device="cuda")
    got = (c.forward()[1], *c.backward(c.x).values())
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    c.close()
