// join_pick.cuh -- the join's kernels of one pair of types.
#pragma once

#include "block_host.h"
#include "block_kernels.cuh"

namespace zo {

template <typename T, typename S, int kC, bool kWide, bool kExtra>
const void* join_of(bool backward, bool post) {
  if (backward)
    return post ? (const void*)join_backward_kernel<T, S, kC, kWide, true, kExtra>
                : (const void*)join_backward_kernel<T, S, kC, kWide, false, kExtra>;
  return post ? (const void*)join_kernel<T, S, kC, kWide, true, kExtra>
              : (const void*)join_kernel<T, S, kC, kWide, false, kExtra>;
}

template <typename T, typename S>
const void* join_of(const JoinPick& p) {
  if (!p.wide) return p.chunks == 1 ? join_of<T, S, 1, false, true>(p.backward, p.post) : join_of<T, S, 4, false, true>(p.backward, p.post);
  if (p.chunks == 4) return join_of<T, S, 4, true, true>(p.backward, p.post);
  if (p.chunks == 2)
    return p.extra ? join_of<T, S, 2, true, true>(p.backward, p.post) : join_of<T, S, 2, true, false>(p.backward, p.post);
  return p.extra ? join_of<T, S, 1, true, true>(p.backward, p.post) : join_of<T, S, 1, true, false>(p.backward, p.post);
}

}  // namespace zo
