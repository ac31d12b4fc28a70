// qk_axes.cu -- the query/key norm's kernels with a position for each of several axes.
#include "qk_kernels.cuh"

const void* zo::qk_kernel_axes(int32_t dtype, bool inter, bool backward, bool sum, int v, int r) {
  return kernel_of<true>(dtype, inter, backward, sum, v, r);
}
