// join_bf16_float.cu -- the join's kernels for bf16 blocks on a binary32 stream.
#include "join_pick.cuh"

const void* zo::join_bf16_float(const JoinPick& p) { return join_of<__nv_bfloat16, float>(p); }
