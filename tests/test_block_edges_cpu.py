"""What the join does not look at, and what its binding takes for a number.  No
launch: without a device a call that is in order is refused for that alone."""
import ctypes

import pytest

from test_block_cpu import GOOD, _buffers, _calls, z  # noqa: F401


@pytest.fixture(autouse=True)
def without_a_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")


@pytest.mark.parametrize("backward,name,over,drop_y", [
    (False, "step", dict(dropout=0.0), False), (True, "step", dict(dropout=0.0), False),
    (False, "step", {}, True), (False, "dy_gain", {}, False), (False, "dgain", {}, False),
    (False, "y_gain", {}, True), (True, "y_gain", {}, True), (False, "gain", dict(norm_out=False), False),
    (True, "gain", dict(norm_out=False), False)])
def test_what_a_call_does_not_use_is_not_checked(z, backward, name, over, drop_y):  # noqa: F811
    h = z.zero_block_create(z.make_block_config(**dict(GOOD, **over)))
    b = _buffers(z)
    if drop_y:
        b.y.data = None
    if name == "step":
        b.rng.step_dev = 0x1004
    else:
        setattr(b, name, 0x100002)
    assert _calls(z, backward)(h, ctypes.byref(b), None) == z.ZERO_ECUDA
    z.zero_block_destroy(h)
