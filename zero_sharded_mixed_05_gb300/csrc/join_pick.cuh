// join_pick.cuh -- the join's kernels of one pair of types.
#pragma once

#include "block_host.h"
#include "block_kernels.cuh"

namespace zo {

template <typename T, typename S, int kC, bool kWide, int kHas, int kMost = kJoinThreads>
const void* join_of(bool backward, bool post) {
  if (backward)
    return post ? (const void*)join_backward_kernel<T, S, kC, kWide, true, kHas>
                : (const void*)join_backward_kernel<T, S, kC, kWide, false, kHas>;
  return post ? (const void*)join_kernel<T, S, kC, kWide, true, kHas, kMost>
              : (const void*)join_kernel<T, S, kC, kWide, false, kHas, kMost>;
}

template <typename T, typename S, int kC>
const void* join_of(const JoinPick& p) {
  if constexpr (kC == 2)
    if (!p.backward && !p.large)
      return p.has == kBare   ? join_of<T, S, kC, true, kBare, 256>(false, p.post)
             : p.has == kDrop ? join_of<T, S, kC, true, kDrop, 256>(false, p.post)
                              : join_of<T, S, kC, true, kGated, 256>(false, p.post);
  return p.has == kBare   ? join_of<T, S, kC, true, kBare>(p.backward, p.post)
         : p.has == kDrop ? join_of<T, S, kC, true, kDrop>(p.backward, p.post)
                          : join_of<T, S, kC, true, kGated>(p.backward, p.post);
}

template <typename T, typename S, int kC, int kMost>
const void* shifted_join_of(const JoinPick& p) {
  return p.has == kBare ? join_of<T, S, kC, false, kBare, kMost>(p.backward, p.post)
                        : join_of<T, S, kC, false, kGated, kMost>(p.backward, p.post);
}

// Long rows, which binary32 blocks have not, have one kernel for all that a branch may
// have.
template <typename T, typename S>
const void* join_of(const JoinPick& p) {
  if constexpr (sizeof(T) == 2)
    if (p.chunks == 4)
      return p.wide ? join_of<T, S, 4, true, kGated>(p.backward, p.post)
                    : join_of<T, S, 4, false, kGated>(p.backward, p.post);
  if (!p.wide)
    return p.chunks == 1           ? shifted_join_of<T, S, 1, kJoinThreads>(p)
           : p.large || p.backward ? shifted_join_of<T, S, 2, kJoinThreads>(p)
                                   : shifted_join_of<T, S, 2, 320>(p);
  return p.chunks == 2 ? join_of<T, S, 2>(p) : join_of<T, S, 1>(p);
}

}  // namespace zo
