// moe_norm_join's walking kernels for bf16 beside fp32.
#include "join_walk.cuh"

namespace rvq {

rvq_status join_walk_bf16(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream) {
    return with_types<RVQ_BF16>(j, [&](auto t) { return walk<decltype(t)>(j, L, bwd, stream); });
}

}  // namespace rvq
