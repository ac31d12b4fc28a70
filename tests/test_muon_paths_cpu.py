"""What the orthogonalised update refuses and says without a launch."""
import ctypes

import pytest

from test_muon_cpu import handle, z  # noqa: F401


def test_fault_count_refuses(z, handle):  # noqa: F811
    import torch
    out = ctypes.c_int64()
    assert z.lib().zero_muon_fault_count(None, None, ctypes.byref(out)) == z.ZERO_EINVAL
    assert z.lib().zero_muon_fault_count(handle, None, None) == z.ZERO_EINVAL
    if not torch.cuda.is_available():
        with pytest.raises(z.ZeroOptError) as e:
            z.zero_muon_fault_count(handle)
        assert e.value.status == z.ZERO_ECUDA
