// join_float.cu -- the join's kernels for binary32 blocks.
#include "join_pick.cuh"

const void* zo::join_float(const JoinPick& p) { return join_of<float, float>(p); }
