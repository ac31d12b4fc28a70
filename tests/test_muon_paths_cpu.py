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


WAITS = r"""
#include <cstdio>
#include "sm103.cuh"
using sm103::Patience;
constexpr uint64_t kMs = 1000 * 1000;
// looks `each` ns apart from `from` on, `pause` ns once after `at` of them: the
// time until the wait is given up
uint64_t given_up(uint64_t from, uint64_t each, int at, uint64_t pause) {
  Patience p;
  uint64_t now = from;
  for (int n = 0; n < 100000000; ++n) {
    if (p.out(now)) return now - from;
    now += each + (n == at ? pause : 0);
  }
  return 0;
}
int main() {
  std::printf("%.3f %.3f %.3f %.3f\n", given_up(5, kMs / 100, -1, 0) / 1e6,
              given_up(5, kMs / 100, 0, 3600000 * kMs) / 1e6, given_up(5, kMs / 100, 1000, 3600000 * kMs) / 1e6,
              given_up(5, 500 * kMs, -1, 0) / 1e6);
}
"""


def test_a_wait_does_not_count_what_the_gpu_did_meanwhile(tmp_path):
    """Two seconds of looking on; an hour between two looks counts as a
    twentieth of them; and every wait ends, however seldom it looks."""
    import subprocess

    from zero_sharded_mixed_05_gb300 import _build
    src, exe = tmp_path / "waits.cu", tmp_path / "waits"
    src.write_text(WAITS)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-I", _build.CSRC, "-o", str(exe), str(src)],
                   check=True)
    steady, early, late, seldom = map(float, subprocess.run([str(exe)], check=True, capture_output=True,
                                                            text=True).stdout.split())
    hour = 3600e3
    assert 2000 <= steady < 2001
    for paused in (early, late):
        assert hour + 1900 <= paused < hour + 1902
    assert 10000 <= seldom <= 11000


def test_step_refuses_tensors_that_are_not_the_handles(z, handle):  # noqa: F811
    """Before any launch: the call itself would say that there is no device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")

    def items(**change):
        shapes, half = [(8, 16), (2, 5, 3)], torch.float16
        return [dict(grad=torch.zeros(s, dtype=half), momentum=torch.zeros(s), master=torch.zeros(s),
                     param16=torch.zeros(s, dtype=half)) | change for s in shapes]
    with pytest.raises(ValueError, match="item 0: grad"):
        z.zero_muon_step(handle, z.make_muon_list(items()))              # tensors of the host
    with pytest.raises(ValueError, match="2"):
        z.zero_muon_step(handle, z.make_muon_list(items()[:1]))
    with pytest.raises(ValueError):
        z.zero_muon_step(handle + 8, z.make_muon_list(items()))
    addresses = z.make_muon_list([dict(grad=16, momentum=32, master=None, param16=64)] * 2)
    with pytest.raises(z.ZeroOptError) as e:
        z.zero_muon_step(handle, addresses)
    assert e.value.status == z.ZERO_ECUDA and addresses.fits is z._muon_handles[handle]


def test_results_that_lie_on_one_another_are_refused(z):  # noqa: F811
    """As a broadcast tensor's do: they would be written by several matrices at
    once.  Rows' strides are looked at as before."""
    h = z.zero_muon_create(z.make_muon_config(), [(8, 16, 3)])
    one = z.zero_muon_create(z.make_muon_config(), [(8, 16, 1)])
    try:
        for stride in (0, 1, 15):
            item = (z.zero_muon_operand * 1)((0x1000, 0x2000, 16, 128, 16, stride))
            assert z.lib().zero_muon_orthogonalize(h, item, 0, 0, None) == z.ZERO_EINVAL
        import torch
        if not torch.cuda.is_available():
            for handle_, item in [(h, (0x1000, 0x2000, 16, 0, 16, 128)),      # a broadcast input
                                  (h, (0x1000, 0x2000, 16, 128, 48, 16)),     # matrices side by side
                                  (one, (0x1000, 0x2000, 16, 0, 16, 0))]:
                arr = (z.zero_muon_operand * 1)(item)
                assert z.lib().zero_muon_orthogonalize(handle_, arr, 0, 0, None) == z.ZERO_ECUDA
    finally:
        z.zero_muon_destroy(h)
        z.zero_muon_destroy(one)
