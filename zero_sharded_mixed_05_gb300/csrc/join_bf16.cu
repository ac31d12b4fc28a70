// join_bf16.cu -- the join's kernels for bf16 blocks on a bf16 stream.
#include "join_pick.cuh"

const void* zo::join_bf16(const JoinPick& p) { return join_of<__nv_bfloat16, __nv_bfloat16>(p); }
