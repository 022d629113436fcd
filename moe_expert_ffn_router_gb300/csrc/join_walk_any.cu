// moe_norm_join's walking kernels with types looked up at run time.
#include "join_walk.cuh"

namespace rvq {

rvq_status join_walk_any(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream) {
    return with_any_types(j, [&](auto t) { return walk<decltype(t)>(j, L, bwd, stream); });
}

}  // namespace rvq
