// moe_norm_join's walking kernels for f16 beside fp32.
#include "join_walk.cuh"

namespace rvq {

rvq_status join_walk_f16(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream) {
    return with_types<RVQ_F16>(j, [&](auto t) { return walk<decltype(t)>(j, L, bwd, stream); });
}

}  // namespace rvq
