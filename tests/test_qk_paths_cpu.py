"""What the query/key norm refuses, beyond test_qk_cpu.py.  No launch."""
import ctypes

import pytest

from test_qk_cpu import GOOD, _buffers, z  # noqa: F401


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("strides,tokens,ok", [
    ((0, 64), 3, False), ((63, 64), 3, False), ((256, 0), 3, False), ((256, 63), 3, False),
    ((256, 0), 1, False), ((0, 64), 1, True), ((64, 256), 3, True), ((-256, 64), 3, True), ((256, -64), 3, True)])
def test_results_that_lie_on_one_another_are_refused(z, backward, strides, tokens, ok):  # noqa: F811
    """As a broadcast tensor's do: they would be written by several tokens or
    heads at once.  Inputs may be broadcast."""
    import torch
    h = z.zero_qk_create(z.make_qk_config(**GOOD))
    call = z.lib().zero_qk_norm_rope_backward if backward else z.lib().zero_qk_norm_rope
    try:
        for name in ("dq", "dk") if backward else ("q_out", "k_out"):
            b = _buffers(z, backward)
            b.tokens = tokens
            b.q = z.zero_qk_tensor(0x1000, 0, 0)
            setattr(b, name, z.zero_qk_tensor(0x7000, *strides))
            if not ok:
                assert call(h, ctypes.byref(b), None) == z.ZERO_EINVAL
            elif not torch.cuda.is_available():
                assert call(h, ctypes.byref(b), None) == z.ZERO_ECUDA
        assert z.zero_qk_launch_count(h) == 0
    finally:
        z.zero_qk_destroy(h)
