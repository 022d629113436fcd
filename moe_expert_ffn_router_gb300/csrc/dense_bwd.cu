// Elementwise gradients in front of the backward products of moe_linear and
// moe_gated_linear, with the bias gradients' sums over tokens.
//
// Memory-bound: dout and the saved fp32 pre-activations are read once, dp is
// written once, 16 or 32 bytes per thread and access.  A block takes 32 rows x
// 256 columns (32 groups of eight columns x 8 row lanes, four rows each), so a
// bias gradient leaves one fp32 partial per 32 rows and column, added in row
// order; a second launch adds the partials in chunk order (no atomics: results
// repeat bit for bit).
#include "dense.cuh"

namespace rvq {
namespace {

constexpr int BW_LANES = 8;
static_assert(kBwdChunkRows % BW_LANES == 0, "rows of a chunk per lane");

__global__ void __launch_bounds__(256) dense_bwd_kernel(const DenseBwdJob j) {
    __shared__ float red[BW_LANES][2][264];
    const int q = threadIdx.x & 31, lane = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + q) * 8;
    const bool on = c < j.rows;
    const bool sums = j.dbias[0] || j.dbias[1];
    float acc[2][8] = {};
    if (on) {
#pragma unroll
        for (int i = 0; i < kBwdChunkRows / BW_LANES; ++i) {
            const int t = blockIdx.y * kBwdChunkRows + i * BW_LANES + lane;
            if (t >= j.n) break;
            const int64_t at = (int64_t)t * j.rows + c;
            float g[8], a[8], sl[8], d0[8], d1[8];
            ld8(j.dout, j.dt, (int64_t)t * j.ldd + c, d0);
            if (j.pre[0]) {
                ld8(j.pre[0], RVQ_F32, at, g);
                act_group_both(j.act, g, a, sl);
            }
            if (j.mats == 2) {
                float u[8];
                ld8(j.pre[1], RVQ_F32, at, u);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    d1[e] = d0[e] * a[e];
                    d0[e] = d0[e] * u[e] * sl[e];
                    acc[1][e] += d1[e];
                }
                if (j.dp[1]) st8(j.dp[1], j.dt, at, d1);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) d0[e] *= j.pre[0] ? j.alpha * sl[e] : j.alpha;
            }
            if (j.dp[0]) st8(j.dp[0], j.dt, at, d0);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[0][e] += d0[e];
        }
    }
    if (!sums) return;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) red[lane][m][q * 8 + e] = acc[m][e];
    __syncthreads();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= j.rows) return;
    for (int m = 0; m < j.mats; ++m) {
        float s = 0.f;
#pragma unroll
        for (int l = 0; l < BW_LANES; ++l) s += red[l][m][threadIdx.x];
        j.part[((int64_t)blockIdx.y * j.mats + m) * j.rows + col] = s;
    }
}

__global__ void __launch_bounds__(256) dense_bias_sum_kernel(const DenseBwdJob j, int chunks) {
    const int col = blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (col >= j.rows || j.dbias[m] == nullptr) return;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < chunks; ++k) s += j.part[((int64_t)k * j.mats + m) * j.rows + col];
    st_elem(j.dbias[m], j.dt, col, s);
}

}  // namespace

rvq_status launch_dense_bwd(const DenseBwdJob &job, cudaStream_t stream) {
    const int chunks = dense_bwd_chunks(job.n);
    if (chunks > 65535) {
        set_error("dense gradient: %d tokens (at most %d)", job.n, 65535 * kBwdChunkRows);
        return RVQ_ENOTIMPL;
    }
    const dim3 grid((unsigned)((job.rows + 255) / 256), (unsigned)chunks);
    dense_bwd_kernel<<<grid, 256, 0, stream>>>(job);
    RVQ_LAUNCHED("dense_bwd");
    if (job.dbias[0] || job.dbias[1]) {
        dense_bias_sum_kernel<<<dim3((unsigned)((job.rows + 255) / 256), (unsigned)job.mats), 256, 0,
                                stream>>>(job, chunks);
        RVQ_LAUNCHED("dense_bias_sum");
    }
    return RVQ_OK;
}

}  // namespace rvq
