// moe_norm_join_mx: moe_norm_join with the normed rows microscaled on the way out.
//
//   z = post_norm ? y r1 w_post : y,  h' = alpha h + gate z,  xn = h' r2 w_pre,
//   r = 1 / sqrt(mean of squares + eps); xn's blocks of 32 scaled and rounded
//
// Memory-bound: h and y in, h' and a byte (or half) per value out.  One block per row;
// a thread keeps its columns (groups of eight, a block's width apart) of h and y in
// registers, so a row is read once and two to four blocks per SM overlap one's loads
// with another's sums.  Four adjacent lanes hold a block of 32.
#include "join_common.cuh"
#include "mx.cuh"

namespace rvq {
namespace {

template <int V, int FMT, int HDT, int YDT>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512) mx_join_kernel(const MxJoinJob job) {
    __shared__ float red[2][32];
    const JoinJob &j = job.join;
    const int hdt = type_of<HDT>(j.hdt), ydt = type_of<YDT>(j.ydt);
    const int t = blockIdx.x;
    const int64_t row = (int64_t)t * j.d;
    const int tiles = mx_tiles(j.d);
    dependency_wait();
    dependents_may_start();
    float y[V][8], h[V][8], g[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[v][e] = h[v][e] = 0.f;
            g[v][e] = 1.f;
        }
        if (c < j.d) {
            ld8(j.y, ydt, row + c, y[v]);
            if (j.h) ld8(j.h, hdt, row + c, h[v]);
            if (j.gate_kind == MOE_GATE_FULL) ld8(j.gate, j.gdt, row + c, g[v]);
            if (j.gate_kind == MOE_GATE_CHANNEL) ld8(j.gate, j.gdt, c, g[v]);
        }
    }
    float gate = 1.f;
    if (j.gate_kind == MOE_GATE_TOKEN) gate = ld_elem(j.gate, j.gdt, t);
    if (j.gate_kind == MOE_GATE_SCALAR) gate = ld_elem(j.gate, j.gdt, 0);
    float r1 = 1.f;
    if (j.post_norm) {
        float s[1] = {0.f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += y[v][e] * y[v][e];
        block_sum(s, red[0]);
        r1 = 1.f / sqrtf(s[0] / (float)j.d + j.eps);
    }
    float s2[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
        if (c >= j.d) continue;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (j.w_post) ld8(j.w_post, j.wdt, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float z = j.post_norm ? y[v][e] * r1 * w[e] : y[v][e];
            const float gz = gate * g[v][e] * z;
            h[v][e] = j.h ? j.alpha * h[v][e] + gz : gz;
            s2[0] += h[v][e] * h[v][e];
        }
        if (j.h_out) st8(j.h_out, hdt, row + c, h[v]);
    }
    block_sum(s2, red[1]);
    const float r2 = 1.f / sqrtf(s2[0] / (float)j.d + j.eps);
    if (j.rstd && threadIdx.x == 0) {
        j.rstd[t] = r1;
        j.rstd[(int64_t)j.n + t] = r2;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (j.w_pre && c < j.d) ld8(j.w_pre, j.wdt, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = c < j.d ? w[e] * (h[v][e] * r2) : 0.f;
        if (j.xn && c < j.d) st8(j.xn, j.xdt, row + c, w);
        mx_put8<FMT>(w, job.codes, job.scales, t, c, tiles, c < tiles * kMxTile);
    }
}

template <int V, int FMT, int HDT, int YDT>
rvq_status launch(const MxJoinJob &job, cudaStream_t stream) {
    // whole half warps for the 128 columns of a word of scales
    const int groups = mx_tiles(job.join.d) * (kMxTile / 8);
    const int threads = ((groups + V - 1) / V + 31) / 32 * 32;
    RVQ_CUDA(launch_after(mx_join_kernel<V, FMT, HDT, YDT>, dim3((unsigned)job.join.n), threads, 0,
                          stream, job));
    return RVQ_OK;
}

template <int V, int FMT>
rvq_status by_types(const MxJoinJob &job, cudaStream_t stream) {
    const int h = job.join.hdt, y = job.join.ydt;
    if (h == RVQ_F32 && y == RVQ_F32) return launch<V, FMT, RVQ_F32, RVQ_F32>(job, stream);
    if (h == RVQ_F32 && y == RVQ_BF16) return launch<V, FMT, RVQ_F32, RVQ_BF16>(job, stream);
    if (h == RVQ_BF16 && y == RVQ_BF16) return launch<V, FMT, RVQ_BF16, RVQ_BF16>(job, stream);
    return launch<V, FMT, kAny, kAny>(job, stream);
}

template <int FMT>
rvq_status by_size(const MxJoinJob &job, cudaStream_t stream) {
    // up to 8192 columns a row fits a block of 1024 threads; with few rows that is the
    // shortest way through it
    if (job.join.d <= 8192 && job.join.n <= num_sms()) return by_types<1, FMT>(job, stream);
    if (job.join.d <= 8192) return by_types<2, FMT>(job, stream);
    return by_types<4, FMT>(job, stream);
}

}  // namespace

rvq_status launch_mx_join(const MxJoinJob &job, cudaStream_t stream) {
    return job.fmt == MOE_MX_F8 ? by_size<MOE_MX_F8>(job, stream)
                                : by_size<MOE_MX_F4>(job, stream);
}

}  // namespace rvq
