// Matrix products of the dense operators (shared expert, dense projections):
// every mode of DenseJob on fp32 multiply-adds.
//
// A block of 256 threads computes a 64 x 64 tile of the output (both
// accumulators of a gated product) from 16-deep slices staged in shared memory
// as fp32; each thread holds 4 x 4 sums.
#include "dense.cuh"

namespace rvq {
namespace {

constexpr int SG_T = 64, SG_K = 16;

// slice[k][i] = operand element (row r0 + i, depth k0 + k); zero past the ends
__device__ __forceinline__ void sg_load(float (*slice)[SG_T + 4], const void *p, int64_t ld, int t,
                                        int dt, int r0, int R, int k0, int K) {
    for (int e = threadIdx.x; e < SG_T * SG_K; e += 256) {
        const int k = t ? e / SG_T : e % SG_K, i = t ? e % SG_T : e / SG_K;
        const int r = r0 + i, kk = k0 + k;
        slice[k][i] = (r < R && kk < K)
                          ? ld_elem(p, dt, t ? (int64_t)kk * ld + r : (int64_t)r * ld + kk)
                          : 0.f;
    }
}

__global__ void __launch_bounds__(256) dense_simple_kernel(const DenseJob j) {
    __shared__ float sa[SG_K][SG_T + 4], sb[2][SG_K][SG_T + 4];
    const int which = j.mode == DG_PAIR_M ? (int)blockIdx.z : 0;
    const int m0 = blockIdx.y * SG_T, n0 = blockIdx.x * SG_T;
    const int tm = (threadIdx.x / 16) * 4, tn = (threadIdx.x % 16) * 4;
    float acc[2][4][4] = {};
    const int passes = j.mode == DG_SUM_K ? 2 : 1;
    for (int ps = 0; ps < passes; ++ps)
        for (int k0 = 0; k0 < j.K; k0 += SG_K) {
            __syncthreads();
            sg_load(sa, j.a[which + ps], j.lda, j.a_t, j.dt, m0, j.M, k0, j.K);
            sg_load(sb[0], j.b[ps], j.ldb, j.b_t, j.dt, n0, j.N, k0, j.K);
            if (j.mode == DG_GATED) sg_load(sb[1], j.b[1], j.ldb, j.b_t, j.dt, n0, j.N, k0, j.K);
            __syncthreads();
            for (int k = 0; k < SG_K; ++k)
                for (int q = 0; q < (j.mode == DG_GATED ? 2 : 1); ++q)
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            acc[q][a][b] += sa[k][tm + a] * sb[q][k][tn + b];
        }
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int m = m0 + tm + a, c = n0 + tn + b;
            if (m >= j.M || c >= j.N) continue;
            float v = acc[0][a][b] + (j.bias[0] ? ld_elem(j.bias[0], j.dt, c) : 0.f);
            if (j.pre[0]) j.pre[0][(int64_t)m * j.N + c] = v;
            v = act_value(j.act, v);
            if (j.mode == DG_GATED) {
                const float u = acc[1][a][b] + (j.bias[1] ? ld_elem(j.bias[1], j.dt, c) : 0.f);
                if (j.pre[1]) j.pre[1][(int64_t)m * j.N + c] = u;
                v *= u;
            } else {
                v *= j.alpha;
                if (j.residual) v += ld_elem(j.residual, j.rdt, (int64_t)m * j.ldr + c);
            }
            st_elem(j.out[which], j.odt, (int64_t)m * j.ldo + c, v);
        }
}

}  // namespace

rvq_status launch_dense_gemm(const DenseJob &job, cudaStream_t stream) {
    const dim3 grid((unsigned)((job.N + SG_T - 1) / SG_T), (unsigned)((job.M + SG_T - 1) / SG_T),
                    job.mode == DG_PAIR_M ? 2u : 1u);
    if (grid.y > 65535u) {
        set_error("dense product: %d rows", job.M);
        return RVQ_ENOTIMPL;
    }
    dense_simple_kernel<<<grid, 256, 0, stream>>>(job);
    RVQ_LAUNCHED("dense_simple");
    return RVQ_OK;
}

}  // namespace rvq
