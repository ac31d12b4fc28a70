"""Argument checks of the orthogonalised update.  No test here launches a kernel."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def z():
    from zero_sharded_mixed_05_gb300 import _build
    _build.build()
    import zero_sharded_mixed_05_gb300 as z
    z.lib()
    return z


@pytest.mark.parametrize("field,value", [
    ("grad_dtype", 2), ("param_dtype", -1), ("nesterov", 2), ("steps", 0), ("steps", 17),
    ("scale_rule", 3), ("scale_rule", -1), ("lr", -1e-3), ("lr", float("nan")), ("momentum", 1.0),
    ("momentum", -0.1), ("weight_decay", -1.0), ("eps", -1e-9), ("coef", float("inf")),
])
def test_create_refuses_config(z, field, value):
    cfg = z.make_muon_config()
    if field == "coef":
        cfg.coef[4][2] = value
    else:
        setattr(cfg, field, value)
    h = ctypes.c_void_p(123)
    shapes = (z.zero_muon_shape * 1)((8, 8, 1))
    assert z.lib().zero_muon_create(ctypes.byref(cfg), shapes, 1, ctypes.byref(h)) == z.ZERO_EINVAL
    assert h.value is None and z.lib().zero_opt_last_error()


@pytest.mark.parametrize("shape,status", [
    ((0, 8, 1), 1), ((8, 0, 1), 1), ((8, 8, 0), 1), ((-1, 8, 1), 1), (((1 << 20) + 1, 1, 1), 2),
    ((1, (1 << 20) + 1, 1), 2), ((1 << 18, 1 << 17, 1), 2), ((8, 8, (1 << 20) + 1), 2),
])
def test_create_refuses_shape(z, shape, status):
    with pytest.raises(z.ZeroOptError) as e:
        z.zero_muon_create(z.make_muon_config(), [(8, 8), shape])
    assert e.value.status == status


def test_create_limits(z):
    with pytest.raises(z.ZeroOptError) as e:
        z.zero_muon_create(z.make_muon_config(), [(8, 8)] * 257)
    assert e.value.status == z.ZERO_ERANGE
    for n in (0, 256):
        z.zero_muon_destroy(z.zero_muon_create(z.make_muon_config(), [(8, 8)] * n))


def test_null_arguments(z):
    L = z.lib()
    assert L.zero_muon_config_default(None) == z.ZERO_EINVAL
    assert L.zero_muon_create(None, None, 0, None) == z.ZERO_EINVAL
    assert L.zero_muon_workspace_bytes(None, None) == z.ZERO_EINVAL
    assert L.zero_muon_set_lr(None, 1.0) == z.ZERO_EINVAL
    assert L.zero_muon_orthogonalize(None, None, 0, 0, None) == z.ZERO_EINVAL
    assert L.zero_muon_step(None, None, 1.0, None, None) == z.ZERO_EINVAL
    assert L.zero_muon_last_step(None, None, None) == z.ZERO_EINVAL
    assert L.zero_muon_launch_count(None, None) == z.ZERO_EINVAL
    assert L.zero_muon_inject_wait_fault(None) == z.ZERO_EINVAL
    assert L.zero_muon_destroy(None) == z.ZERO_OK
    assert L.zero_opt_decision(None, None) == z.ZERO_EINVAL


def test_defaults(z):
    c = z.zero_muon_config()
    assert z.lib().zero_muon_config_default(ctypes.byref(c)) == z.ZERO_OK
    assert (c.lr, c.momentum, c.weight_decay, c.eps) == (2e-2, 0.95, 0.0, 1e-7)
    assert c.nesterov == 1 and c.steps == 5 and list(c.coef[4]) == [3.4445, -4.7750, 2.0315]


@pytest.fixture()
def handle(z):
    h = z.zero_muon_create(z.make_muon_config(), [(8, 16), (5, 3, 2)])
    yield h
    z.zero_muon_destroy(h)


def test_calls_refuse(z, handle):
    L = z.lib()
    ok = [(0x1000, 0x2000, 16, 128, 16, 128), (0x3000, 0x4000, 3, 15, 3, 15)]

    def ortho(items, i=0, o=0):
        return L.zero_muon_orthogonalize(handle, (z.zero_muon_operand * 2)(*items), i, o, None)
    assert ortho(ok, 3) == ortho(ok, 0, -1) == z.ZERO_EINVAL
    for j, v in [(0, None), (1, None), (2, 15), (4, 15), (3, -1), (5, -1), (2, -16)]:
        bad = list(ok[0])
        bad[j] = v
        assert ortho([tuple(bad), ok[1]]) == z.ZERO_EINVAL, (j, v)
    assert L.zero_muon_orthogonalize(handle, None, 0, 0, None) == z.ZERO_EINVAL
    mats = [(0x1000, 0x2000, 0x3000, 0x4000), (0x5000, 0x6000, None, 0x7000)]
    for j in (0, 1, 3):
        bad = list(mats[0])
        bad[j] = None
        arr = (z.zero_muon_matrix * 2)(tuple(bad), mats[1])
        assert L.zero_muon_step(handle, arr, 1.0, None, None) == z.ZERO_EINVAL
    arr = (z.zero_muon_matrix * 2)(*mats)
    for v in (float("nan"), float("inf")):
        assert L.zero_muon_step(handle, arr, v, None, None) == z.ZERO_EINVAL
    with pytest.raises(z.ZeroOptError):
        z.zero_muon_set_lr(handle, -1.0)
    with pytest.raises(ValueError):
        z.zero_muon_step(handle, z.make_muon_list([]))
    with pytest.raises(ValueError):
        z.make_muon_config(steps=3, coefs=[(1, 0, 0)] * 2)
    assert z.zero_muon_launch_count(handle) == 0


def test_valid_calls_without_a_device_are_cuda_errors(z, handle):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    L = z.lib()
    mats = (z.zero_muon_matrix * 2)((1, 2, 3, 4), (5, 6, 7, 8))
    assert L.zero_muon_step(handle, mats, 1.0, None, None) == z.ZERO_ECUDA
    info = z.zero_muon_info()
    assert L.zero_muon_last_step(handle, None, ctypes.byref(info)) == z.ZERO_ECUDA
    h = z.zero_opt_create(z.make_config(numel=8))
    with pytest.raises(z.ZeroOptError) as e:
        z.zero_opt_decision(h)
    assert e.value.status == z.ZERO_ECUDA
    z.zero_opt_destroy(h)
