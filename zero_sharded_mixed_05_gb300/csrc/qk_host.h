// qk_host.h -- the query/key norm's kernels as the host picks them.
#pragma once

#include <stdint.h>

namespace zo {

// Kernels that take a QkArgs (one position a token) or a QkAxesArgs; v numbers a
// vector, r heads a group, sum: one sum of gain gradients a group.
const void* qk_kernel_one(int32_t dtype, bool inter, bool backward, bool sum, int v, int r);
const void* qk_kernel_axes(int32_t dtype, bool inter, bool backward, bool sum, int v, int r);

}  // namespace zo
