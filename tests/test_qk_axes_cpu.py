"""What the rotation over several axes refuses, and its helpers.  No launch."""
import ctypes

import pytest

from test_qk_cpu import GOOD, _buffers, z  # noqa: F401


def create(z, axes, **over):  # noqa: F811
    h = ctypes.c_void_p(123)
    s = z.lib().zero_qk_create_axes(ctypes.byref(z.make_qk_config(**dict(GOOD, **over))), ctypes.byref(axes),
                                    ctypes.byref(h))
    return s, h


@pytest.mark.parametrize("field,value", [("axes", 0), ("axes", 5), ("axes", -1), ("axes", 2), ("normalise", 2),
                                         ("normalise", -1), ("axis", 3)])
def test_create_refuses(z, field, value):  # noqa: F811
    axes = z.make_qk_axes([0, 1, 2] * 5 + [0])
    if field == "axis":
        axes.axis[15] = value          # the last of 16 pairs
    else:
        setattr(axes, field, value)
    s, h = create(z, axes)
    assert s == z.ZERO_EINVAL and h.value is None and z.lib().zero_opt_last_error()


def test_create_checks_the_rest_as_ever(z):  # noqa: F811
    for over in (dict(head_dim=63), dict(rotary_dim=600), dict(rotary_dim=-2), dict(q_heads=0)):
        s, h = create(z, z.make_qk_axes([0] * 16), **over)
        assert s == z.ZERO_EINVAL and h.value is None
    axes = z.make_qk_axes([0] * 16)
    axes.axis[16] = 9                  # behind the last pair: not looked at
    s, h = create(z, axes)
    assert s == z.ZERO_OK
    z.lib().zero_qk_destroy(h)
    assert z.lib().zero_qk_create_axes(None, None, None) == z.ZERO_EINVAL
    for bad in ([0] * 257, [-1], [256]):
        with pytest.raises(ValueError):
            z.make_qk_axes(bad)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("broken", ["n_pos", "positions", "q_gain", "k_gain", "dq_gain", "q", "q_out", "dq", "none"])
def test_calls_refuse(z, backward, broken):  # noqa: F811
    """Without the norm there are no gains, and the backward call needs no rows."""
    import torch
    h = z.zero_qk_create(z.make_qk_config(**GOOD), z.make_qk_axes([0, 1] * 8, normalise=False))
    try:
        b = _buffers(z, backward)
        ok = broken == "none"
        if broken == "n_pos":
            b.n_pos = 2 ** 31
        elif broken == "positions":
            b.positions, b.positions64 = 0x30004, 1
        elif broken in ("q_gain", "k_gain", "dq_gain"):
            setattr(b, broken, 0x9000)
            ok = broken == "dq_gain" and not backward
        elif broken in ("q", "q_out", "dq"):
            setattr(b, broken, z.zero_qk_tensor(None, 256, 64))
            ok = broken == ("q" if backward else "dq")
        call = z.lib().zero_qk_norm_rope_backward if backward else z.lib().zero_qk_norm_rope
        if not ok:
            assert call(h, ctypes.byref(b), None) == z.ZERO_EINVAL
        elif not torch.cuda.is_available():
            assert call(h, ctypes.byref(b), None) == z.ZERO_ECUDA
        assert z.zero_qk_launch_count(h) == 0
    finally:
        z.zero_qk_destroy(h)


def test_the_binding_takes_a_position_an_axis(z):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    h = z.zero_qk_create(z.make_qk_config(2, 0, 8, dtype=z.FP32), z.make_qk_axes([0, 1, 2, 0]))
    q, table = torch.zeros(5, 2, 8), torch.zeros(9, 4)
    for shape in ((5,), (2, 5), (5, 3)):
        with pytest.raises(ValueError):
            z.zero_qk_norm_rope(h, q, None, q, None, None, None, table, table, torch.zeros(shape, dtype=torch.int64))
    with pytest.raises(z.ZeroOptError):
        z.zero_qk_norm_rope(h, q, None, q, None, None, None, table, table, torch.zeros(3, 5, dtype=torch.int32))
    z.zero_qk_destroy(h)


def test_helpers():
    import torch
    from zero_sharded_mixed_05_gb300.qk import axis_of_pairs, rotation_tables
    assert axis_of_pairs((2, 0, 3)) == [0, 0, 2, 2, 2]
    assert axis_of_pairs((3, 1, 2), alternate=True) == [0, 1, 2, 0, 2, 0]
    cos, sin = rotation_tables(7, 8, 100.0, "cpu", axis=[0, 1, 1, 0])
    for j, power in enumerate([0, 0, 0.5, 0.5]):
        a = torch.arange(7, dtype=torch.float64) * 100.0 ** -power
        assert torch.equal(cos[:, j], a.cos().float()) and torch.equal(sin[:, j], a.sin().float())
    a, b = rotation_tables(7, 8, device="cpu"), rotation_tables(7, 8, device="cpu", axis=[0] * 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):
        rotation_tables(7, 8, device="cpu", axis=[0, 1])
