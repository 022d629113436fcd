// Elementwise gradients in front of the backward products of moe_linear and
// moe_gated_linear, with the bias gradients' sums over tokens.
//
// dp is rounded to 16 bits here, once: the products' operands are of one 16-bit type,
// and dp in two such parts would double their time.  It is the second of the two
// roundings of dx and dw (error against 64 bits 2.4e-3 in bf16, 1.7e-3 with the last
// rounding alone); bias gradients are summed before it.
//
// Memory-bound (4096 x 2048, gated: 117 MB in 20 us, 5.9 TB/s; 1777 x 4104 with GELU:
// 58 MB in 15 us): dout and the saved fp32 pre-activations are read once, dp is
// written once, 16 or 32 bytes per thread and access.  A block takes 32 rows x
// 256 columns (32 groups of eight columns x 8 row lanes, four rows each), so a
// bias gradient leaves one fp32 partial per 32 rows and column, added in row
// order.  The partials are added in a fixed order (no atomics: results repeat
// bit for bit) by idle warps of the products that follow, which hides them (whole
// training step, 757 x 2000 x 336: 24.0 us; with a launch of their own 26.0), or by a
// launch of their own where no such product is wanted.
#include "dense.cuh"

namespace rvq {
namespace {

constexpr int BW_LANES = 8;
static_assert(kBwdChunkRows % BW_LANES == 0, "rows of a chunk per lane");

// eight fp32 values; `wide`: at a multiple of 32 bytes, one load per lane.  A plain
// load, as of dout below: blocks may be resident while the kernel before still writes
// these values, and the read-only path is for data that no one writes meanwhile.
__device__ __forceinline__ void ld32(const float *p, int wide, float (&v)[8]) {
    if (wide) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                       "=f"(v[6]), "=f"(v[7])
                     : "l"(p));
    } else {
        ld8(p, RVQ_F32, 0, v);
    }
}

template <int MATS>
__global__ void __launch_bounds__(256) dense_bwd_kernel(const DenseBwdJob j) {
    __shared__ float red[BW_LANES][MATS][264];
    const int q = threadIdx.x & 31, lane = threadIdx.x >> 5;
    const int c = (blockIdx.y * 32 + q) * 8;
    const bool on = c < j.rows;
    dependency_wait();
    dependents_may_start();  // the products' blocks set up beside the last of these
    const bool sums = j.dbias[0] || j.dbias[1];
    float acc[2][8] = {};
    if (on) {
        // every load of the block's rows is issued before the first is used
        constexpr int R = kBwdChunkRows / BW_LANES;
        uint4 d_raw[R];
        float g[R][8], u[R][8];
        int64_t at[R];
        bool ok[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = blockIdx.x * kBwdChunkRows + i * BW_LANES + lane;
            ok[i] = t < j.n;
            at[i] = (int64_t)t * j.rows + c;
            if (!ok[i]) continue;
            d_raw[i] = *reinterpret_cast<const uint4 *>(
                reinterpret_cast<const uint16_t *>(j.dout) + (int64_t)t * j.ldd + c);
            if (j.pre[0]) ld32(j.pre[0] + at[i], j.wide, g[i]);
            if (MATS == 2) ld32(j.pre[1] + at[i], j.wide, u[i]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (!ok[i]) continue;
            float a[8], sl[8], d0[8], d1[8];
            unpack16(j.dt, d_raw[i].x, d0[0], d0[1]);
            unpack16(j.dt, d_raw[i].y, d0[2], d0[3]);
            unpack16(j.dt, d_raw[i].z, d0[4], d0[5]);
            unpack16(j.dt, d_raw[i].w, d0[6], d0[7]);
            if (j.pre[0]) act_group_both<MATS == 2>(j.act, g[i], a, sl);
            if (MATS == 2) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    d1[e] = d0[e] * a[e];
                    d0[e] = d0[e] * u[i][e] * sl[e];
                    acc[1][e] += d1[e];
                }
                if (j.dp[1]) st8(j.dp[1], j.dt, at[i], d1);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) d0[e] *= j.pre[0] ? j.alpha * sl[e] : j.alpha;
            }
            if (j.dp[0]) st8(j.dp[0], j.dt, at[i], d0);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[0][e] += d0[e];
        }
    }
    if (!sums) return;
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) red[lane][m][q * 8 + e] = acc[m][e];
    __syncthreads();
    const int col = blockIdx.y * 256 + threadIdx.x;
    if (col >= j.rows) return;
    for (int m = 0; m < MATS; ++m) {
        float s = 0.f;
#pragma unroll
        for (int l = 0; l < BW_LANES; ++l) s += red[l][m][threadIdx.x];
        j.part[((int64_t)blockIdx.x * MATS + m) * j.rows + col] = s;
    }
}

__global__ void __launch_bounds__(256) dense_bias_sum_kernel(const BiasSums s) {
    dependency_wait();
    add_bias_sums(s, (int)blockIdx.x * 8 + (threadIdx.x >> 5), (int)gridDim.x * 8, threadIdx.x & 31);
}

}  // namespace

rvq_status launch_dense_bwd(const DenseBwdJob &job, cudaStream_t stream) {
    const int chunks = dense_bwd_chunks(job.n);
    const dim3 grid((unsigned)chunks, (unsigned)((job.rows + 255) / 256));
    DenseBwdJob j = job;
    j.wide = (((uintptr_t)job.pre[0] | (uintptr_t)job.pre[1]) & 31) == 0;
    RVQ_CUDA(job.mats == 2 ? launch_after(dense_bwd_kernel<2>, grid, 256, 0, stream, j)
                           : launch_after(dense_bwd_kernel<1>, grid, 256, 0, stream, j));
    return RVQ_OK;
}

BiasSums bias_sums_of(const DenseBwdJob &job) {
    return {job.part, dense_bwd_chunks(job.n), job.mats, job.rows, job.dt,
            {job.dbias[0], job.dbias[1]}};
}

rvq_status launch_bias_sums(const BiasSums &s, cudaStream_t stream) {
    const int groups = s.mats * (s.rows / 8);  // a warp each
    RVQ_CUDA(launch_after(dense_bias_sum_kernel, (unsigned)((groups + 7) / 8), 256, 0, stream, s));
    return RVQ_OK;
}

}  // namespace rvq
