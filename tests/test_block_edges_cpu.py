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


def test_integers_of_any_kind_choose_the_numbers(z):  # noqa: F811
    """numpy's and others that index: what is refused is what is no integer, and by
    the binding's own error."""
    import numpy as np
    import torch
    h = z.zero_block_create(z.make_block_config(64, dtype=z.FP32, dropout=0.1))
    t = torch.zeros(3, 64)
    try:
        for seed, call, step in ((np.int64(5), np.uint32(7), np.int64(9)), (True, False, True),
                                 (torch.tensor(3), torch.tensor(4), 5), (2 ** 64 - 1, 2 ** 32 - 1, -2 ** 63)):
            with pytest.raises(z.ZeroOptError):       # nothing wrong but the missing device
                z.zero_block_join(h, t, t, t, t, None, None, seed=seed, call=call, step=step)
        for bad in (dict(seed=1.0), dict(call=1.5), dict(step=2.0), dict(step="1"), dict(seed=None), dict(step=None),
                    dict(call=np.float32(1)), dict(step=np.int64(3) + 0.5)):
            with pytest.raises(ValueError):
                z.zero_block_join(h, t, t, t, t, None, None, **bad)
    finally:
        z.zero_block_destroy(h)


@pytest.mark.parametrize("field,value", [("alpha", 1e39), ("beta", -1e39), ("alpha", 1e308), ("beta", 3.5e38)])
def test_factors_that_binary32_does_not_hold_are_refused(z, field, value):  # noqa: F811
    """They would be infinities in the kernels."""
    cfg = z.make_block_config(**GOOD)
    setattr(cfg, field, value)
    h = ctypes.c_void_p(123)
    assert z.lib().zero_block_create(ctypes.byref(cfg), ctypes.byref(h)) == z.ZERO_EINVAL and h.value is None
    setattr(cfg, field, 3.4e38)
    assert z.lib().zero_block_create(ctypes.byref(cfg), ctypes.byref(h)) == z.ZERO_OK
    z.lib().zero_block_destroy(h)
