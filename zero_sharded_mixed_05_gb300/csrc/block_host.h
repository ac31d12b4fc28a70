// block_host.h -- the join's kernels as the host picks them.
#pragma once

#include <stdint.h>

namespace zo {

// Kernels that take a JoinArgs; c: 1, 2 (wide only) or 4 chunks a thread.
const void* join_forward(int32_t dtype, int32_t stream, int c, bool wide);
const void* join_backward(int32_t dtype, int32_t stream, int c, bool wide);

}  // namespace zo
