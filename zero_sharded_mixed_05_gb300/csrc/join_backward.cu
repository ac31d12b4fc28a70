// join_backward.cu -- the join's backward kernels, by types, chunks a thread and
// whether rows lie on 16-byte boundaries.
#include "block_host.h"
#include "block_kernels.cuh"

namespace zo {
namespace {

template <typename T, typename S>
const void* of(int c, bool wide) {
  if (!wide)
    return c == 1 ? (const void*)join_backward_kernel<T, S, 1, false>
                  : (const void*)join_backward_kernel<T, S, 4, false>;
  return c == 1   ? (const void*)join_backward_kernel<T, S, 1, true>
         : c == 2 ? (const void*)join_backward_kernel<T, S, 2, true>
                  : (const void*)join_backward_kernel<T, S, 4, true>;
}

}  // namespace

const void* join_backward(int32_t dtype, int32_t stream, int c, bool wide) {
  if (dtype == ZERO_FP32) return of<float, float>(c, wide);
  if (dtype == ZERO_FP16) return stream == ZERO_FP32 ? of<__half, float>(c, wide) : of<__half, __half>(c, wide);
  return stream == ZERO_FP32 ? of<__nv_bfloat16, float>(c, wide) : of<__nv_bfloat16, __nv_bfloat16>(c, wide);
}

}  // namespace zo
