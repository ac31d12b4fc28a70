// block_host.h -- the join's kernels as the host picks them.
#pragma once

#include <stdint.h>

namespace zo {

struct JoinPick {
  bool backward, wide;
  bool post;       // the branch is normalised
  int has;         // 0; 1: a dropout; 2: a gate and maybe a dropout
  int chunks;      // a thread: 1, 2 or 4
  bool large;      // more than 256 threads a CTA, or 320 where not wide
};

// Kernels that take a JoinArgs, by the types of the block and of the stream.
const void* join_half(const JoinPick& p);
const void* join_half_float(const JoinPick& p);
const void* join_bf16(const JoinPick& p);
const void* join_bf16_float(const JoinPick& p);
const void* join_float(const JoinPick& p);

}  // namespace zo
