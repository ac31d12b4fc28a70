// join_half.cu -- the join's kernels for fp16 blocks on an fp16 stream.
#include "join_pick.cuh"

const void* zo::join_half(const JoinPick& p) { return join_of<__half, __half>(p); }
