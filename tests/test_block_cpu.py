"""Argument checks of the join and of dropout, and the tests' generator.  No
test here launches a kernel."""
import ctypes

import numpy as np
import pytest

import block_ref as R


@pytest.fixture(scope="module")
def z():
    from zero_sharded_mixed_05_gb300 import _build
    _build.build()
    import zero_sharded_mixed_05_gb300 as z
    z.lib()
    return z


def test_the_generator_gives_the_published_numbers():
    """Known answers of Philox 4x32-10, as published with the method."""
    ones = 0xFFFFFFFF
    for c, k, want in [
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((ones,) * 4, (ones,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        got = R.philox([np.array([v]) for v in c], k)
        assert tuple(int(v[0]) for v in got) == want


GOOD = dict(dim=64, dtype=1, norm_branch=True, gate=2, dropout=0.1)


@pytest.mark.parametrize("field,value", [
    ("dim", 0), ("dim", 16385), ("dtype", 3), ("dtype", -1), ("stream_dtype", 0), ("stream_dtype", 3),
    ("norm_branch", 2), ("norm_out", -1), ("gate", 3), ("gate", -1), ("eps", -1e-6), ("eps", float("nan")),
    ("eps", float("inf")), ("alpha", float("nan")), ("alpha", float("inf")), ("beta", float("nan")),
    ("dropout", -0.1), ("dropout", 1.1), ("dropout", float("nan")),
])
def test_create_refuses(z, field, value):
    cfg = z.make_block_config(**GOOD)
    setattr(cfg, field, value)
    h = ctypes.c_void_p(123)
    assert z.lib().zero_block_create(ctypes.byref(cfg), ctypes.byref(h)) == z.ZERO_EINVAL
    assert h.value is None and z.lib().zero_opt_last_error()


def test_the_widest_rows(z):
    for dim, dtype, kw, ok in [(16384, z.BF16, {}, True), (8192, z.FP32, {}, True), (8193, z.FP32, {}, False),
                               (16384, z.BF16, dict(gate=1), True), (16384, z.BF16, dict(stream_dtype=z.FP32), True),
                               (12288, z.BF16, dict(stream_dtype=z.FP32, gate=1), True),
                               (12289, z.FP16, dict(stream_dtype=z.FP32, gate=2), False)]:
        cfg, h = z.make_block_config(dim, dtype=dtype, **kw), ctypes.c_void_p()
        status = z.lib().zero_block_create(ctypes.byref(cfg), ctypes.byref(h))
        assert status == (z.ZERO_OK if ok else z.ZERO_EINVAL)
        z.lib().zero_block_destroy(h)


def test_null_arguments(z):
    L = z.lib()
    assert L.zero_block_create(None, None) == z.ZERO_EINVAL
    assert L.zero_block_join(None, None, None) == z.ZERO_EINVAL
    assert L.zero_block_join_backward(None, None, None) == z.ZERO_EINVAL
    assert L.zero_block_launch_count(None, None) == z.ZERO_EINVAL
    assert L.zero_block_destroy(None) == z.ZERO_OK
    assert L.zero_dropout(None, None) == z.ZERO_EINVAL
    h = z.zero_block_create(z.make_block_config(**GOOD))
    assert L.zero_block_join(h, None, None) == z.ZERO_EINVAL
    z.zero_block_destroy(h)


def _buffers(z):
    b = z.zero_block_buffers()
    b.tokens = 3
    for i, (name, _) in enumerate(z.zero_block_buffers._fields_[1:11]):
        setattr(b, name, z.zero_block_rows(0x1000 * (i + 1), 64))
    for i, name in enumerate(["y_gain", "gain", "dy_gain", "dgain", "mask"]):
        setattr(b, name, 0x100000 * (i + 1))
    return b


def _calls(z, backward):
    return z.lib().zero_block_join_backward if backward else z.lib().zero_block_join


@pytest.mark.parametrize("backward,broken", [
    (False, "x"), (True, "x_out"), (False, "gate"), (True, "gate"), (False, "h"), (True, "both"),
    (False, "tokens"), (True, "tokens"), (False, "none"), (True, "none")])
def test_calls_refuse(z, backward, broken):
    import torch
    h = z.zero_block_create(z.make_block_config(**GOOD))
    try:
        b = _buffers(z)
        if broken == "tokens":
            b.tokens = -1
        elif broken == "both":
            b.dx_out.data = b.dh.data = None
        elif broken != "none":
            getattr(b, broken).data = None
        if broken == "none":
            if torch.cuda.is_available():
                pytest.skip("a CUDA device is present")
            assert _calls(z, backward)(h, ctypes.byref(b), None) == z.ZERO_ECUDA
        else:
            assert _calls(z, backward)(h, ctypes.byref(b), None) == z.ZERO_EINVAL
        assert z.zero_block_launch_count(h) == 0
    finally:
        z.zero_block_destroy(h)


def test_no_result_wanted_is_refused(z):
    h = z.zero_block_create(z.make_block_config(64, norm_out=False))
    b = _buffers(z)
    b.x_out.data = None
    assert z.lib().zero_block_join(h, ctypes.byref(b), None) == z.ZERO_EINVAL
    b = _buffers(z)
    b.dx_out.data = None              # without norm_out dh is no gradient
    assert z.lib().zero_block_join_backward(h, ctypes.byref(b), None) == z.ZERO_EINVAL
    z.zero_block_destroy(h)


@pytest.mark.parametrize("backward,name", [(False, "x_out"), (False, "h"), (True, "dx"), (True, "dy"),
                                           (True, "dgate")])
@pytest.mark.parametrize("stride,tokens,ok", [(0, 3, False), (63, 3, False), (-63, 3, False), (0, 1, True),
                                              (64, 3, True), (-64, 3, True)])
def test_results_that_lie_on_one_another_are_refused(z, backward, name, stride, tokens, ok):
    """As a broadcast tensor's do: they would be written by several CTAs at
    once.  Inputs may be broadcast."""
    import torch
    h = z.zero_block_create(z.make_block_config(**GOOD))
    b = _buffers(z)
    b.tokens = tokens
    b.gate.stride = b.y.stride = 0
    getattr(b, name).stride = stride
    if not ok:
        assert _calls(z, backward)(h, ctypes.byref(b), None) == z.ZERO_EINVAL
    elif not torch.cuda.is_available():
        assert _calls(z, backward)(h, ctypes.byref(b), None) == z.ZERO_ECUDA
    assert z.zero_block_launch_count(h) == 0
    z.zero_block_destroy(h)


@pytest.mark.parametrize("backward,name", [(False, "x"), (False, "y"), (False, "h"), (True, "dx_out"),
                                           (True, "dy"), (False, "gain"), (True, "dgain"), (False, "step")])
def test_misaligned_pointers_are_refused(z, backward, name):
    h = z.zero_block_create(z.make_block_config(**GOOD))
    b = _buffers(z)
    if name == "step":
        b.rng.step_dev = 0x1004
    elif name in ("gain", "dgain"):
        setattr(b, name, 0x1002)
    else:
        getattr(b, name).data = 0x1001
    assert _calls(z, backward)(h, ctypes.byref(b), None) == z.ZERO_EINVAL
    z.zero_block_destroy(h)


def _drop(z):
    b = z.zero_drop_buffers()
    b.in_, b.out, b.rows, b.cols, b.in_stride, b.out_stride, b.dtype, b.p = 0x1000, 0x2000, 3, 10, 0, 10, z.BF16, 0.5
    return b


@pytest.mark.parametrize("field,value", [
    ("rows", -1), ("cols", -1), ("dtype", 3), ("p", -0.1), ("p", 1.5), ("p", float("nan")), ("in_", None),
    ("out", None), ("in_", 0x1001), ("out", 0x2001), ("out_stride", 9), ("out_stride", 0), ("none", 0)])
def test_dropout_refuses(z, field, value):
    import torch
    b = _drop(z)
    if field != "none":
        setattr(b, field, value)
        assert z.lib().zero_dropout(ctypes.byref(b), None) == z.ZERO_EINVAL
    elif not torch.cuda.is_available():
        assert z.lib().zero_dropout(ctypes.byref(b), None) == z.ZERO_ECUDA


def test_the_binding_refuses(z):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    h = z.zero_block_create(z.make_block_config(64, dtype=z.FP32, dropout=0.1))
    try:
        good = torch.zeros(3, 64)
        for bad in (torch.zeros(3, 65), torch.zeros(3, 64).half(), torch.zeros(3, 64, 1),
                    torch.zeros(64, 3).T, torch.zeros(4, 64)):
            with pytest.raises(ValueError):
                z.zero_block_join(h, good, bad, good, good, None, None)
        for seed, call, step in ((-1, 0, 0), (2 ** 64, 0, 0), (0, 2 ** 32, 0), (0, -1, 0), (0, 0, 2 ** 63),
                                 (0, 0, torch.zeros(2, dtype=torch.int64)), (0, 0, torch.zeros(1))):
            with pytest.raises(ValueError):
                z.zero_block_join(h, good, good, good, good, None, None, seed=seed, call=call, step=step)
        for gain in (torch.zeros(63), torch.zeros(64).half(), torch.zeros(128)[::2]):
            with pytest.raises(ValueError):
                z.zero_block_join(h, good, good, good, good, gain, None)
        for mask in (torch.ones(4, dtype=torch.bool), torch.ones(3)):
            with pytest.raises(ValueError):
                z.zero_block_join(h, good, good, good, good, None, None, mask=mask)
        with pytest.raises(z.ZeroOptError):       # nothing wrong but the missing device
            z.zero_block_join(h, good, good, good, good, None, None)
        with pytest.raises(ValueError):
            z.zero_block_join(12345, good, good, good, good, None, None)
    finally:
        z.zero_block_destroy(h)
    with pytest.raises(ValueError):
        z.zero_dropout(torch.zeros(3, 4), torch.zeros(3, 4), 0.5)
