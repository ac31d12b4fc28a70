"""Argument checks of the query/key norm calls.  No test here launches a kernel."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def z():
    from zero_sharded_mixed_05_gb300 import _build
    _build.build()
    import zero_sharded_mixed_05_gb300 as z
    z.lib()
    return z


GOOD = dict(q_heads=4, k_heads=2, head_dim=64, rotary_dim=32)


@pytest.mark.parametrize("field,value", [
    ("q_heads", 0), ("k_heads", -1), ("k_heads", 4093), ("head_dim", 63), ("head_dim", 0),
    ("head_dim", 514), ("rotary_dim", 66), ("rotary_dim", 31), ("rotary_dim", -2), ("dtype", 3),
    ("interleaved", 2), ("gain_per_head", -1), ("eps", -1e-6), ("eps", float("nan")),
])
def test_create_refuses(z, field, value):
    cfg = z.make_qk_config(**GOOD)
    setattr(cfg, field, value)
    h = ctypes.c_void_p(123)
    assert z.lib().zero_qk_create(ctypes.byref(cfg), ctypes.byref(h)) == z.ZERO_EINVAL
    assert h.value is None and z.lib().zero_opt_last_error()


def test_null_arguments(z):
    L = z.lib()
    assert L.zero_qk_create(None, None) == z.ZERO_EINVAL
    assert L.zero_qk_norm_rope(None, None, None) == z.ZERO_EINVAL
    assert L.zero_qk_norm_rope_backward(None, None, None) == z.ZERO_EINVAL
    assert L.zero_qk_launch_count(None, None) == z.ZERO_EINVAL
    assert L.zero_qk_destroy(None) == z.ZERO_OK


def _buffers(z, backward):
    b = z.zero_qk_buffers()
    b.tokens, b.n_pos = 3, 8
    for i, name in enumerate(["q", "k", "q_out", "k_out"] + (["dq", "dk"] if backward else [])):
        setattr(b, name, z.zero_qk_tensor(0x1000 * (i + 1), 256, 64))
    b.cos, b.sin, b.positions = 0x10000, 0x20000, 0x30000
    return b


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("broken", ["tokens", "n_pos", "q", "k", "q_out", "k_out", "out", "cos",
                                    "sin", "positions", "none"])
def test_calls_refuse(z, backward, broken):
    h = z.zero_qk_create(z.make_qk_config(**GOOD))
    call = z.lib().zero_qk_norm_rope_backward if backward else z.lib().zero_qk_norm_rope
    try:
        b = _buffers(z, backward)
        if broken in ("tokens", "n_pos"):
            setattr(b, broken, -1)
        elif broken in ("cos", "sin", "positions"):
            setattr(b, broken, None)
        elif broken == "out":
            setattr(b, "dk" if backward else "k_out", z.zero_qk_tensor(None, 256, 64))
        elif broken != "none":
            setattr(b, broken, z.zero_qk_tensor(None, 256, 64))
        import torch
        if broken == "none":
            if torch.cuda.is_available():
                pytest.skip("a CUDA device is present")
            assert call(h, ctypes.byref(b), None) == z.ZERO_ECUDA
        else:
            assert call(h, ctypes.byref(b), None) == z.ZERO_EINVAL
        assert z.zero_qk_launch_count(h) == 0
    finally:
        z.zero_qk_destroy(h)
