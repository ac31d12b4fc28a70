// qk_one.cu -- the query/key norm's kernels with one position a token.
#include "qk_kernels.cuh"

const void* zo::qk_kernel_one(int32_t dtype, bool inter, bool backward, bool sum, int v, int r) {
  return kernel_of<false>(dtype, inter, backward, sum, v, r);
}
