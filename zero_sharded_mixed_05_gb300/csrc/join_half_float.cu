// join_half_float.cu -- the join's kernels for fp16 blocks on a binary32 stream.
#include "join_pick.cuh"

const void* zo::join_half_float(const JoinPick& p) { return join_of<__half, float>(p); }
