// moe_norm_join: the norm after a block, its gate, the scaled residual and the
// norm before the next block, in one pass over the rows; and its gradients.
//
// Memory-bound (a few operations per byte): each row's values stay in
// registers between the sums and the outputs, so every input is read once and
// every output written once.  One block per row, V groups of eight columns per
// thread.  All sums are fp32: a thread's columns in order, then the warp's by
// shuffles, then the warps' in order.
#include "dense.cuh"

namespace rvq {
namespace {

// Sums of K values over the block; `red` is K * 32 floats.  Every thread gets
// the result.  A block calls it with alternating buffers, so one barrier per
// call is enough.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    const int warps = (blockDim.x + 31) >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) red[k * 32 + (threadIdx.x >> 5)] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = 0.f;
        for (int w = 0; w < warps; ++w) v[k] += red[k * 32 + w];
    }
}

__device__ __forceinline__ void ones8(float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
}

// the gate's values for eight columns of token t (1 without one)
__device__ __forceinline__ void gate8(const JoinJob &j, int t, int c, float (&g)[8]) {
    if (j.gate_kind == MOE_GATE_CHANNEL) {
        ld8(j.gate, j.gdt, c, g);
    } else if (j.gate_kind == MOE_GATE_FULL) {
        ld8(j.gate, j.gdt, (int64_t)t * j.d + c, g);
    } else {
        const float s = j.gate_kind == MOE_GATE_NONE
                            ? 1.f
                            : ld_elem(j.gate, j.gdt, j.gate_kind == MOE_GATE_TOKEN ? t : 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = s;
    }
}

template <int V>
__global__ void __launch_bounds__(1024) norm_join_kernel(const JoinJob j) {
    __shared__ float red[2][32];
    const int t = blockIdx.x;
    const int64_t row = (int64_t)t * j.d;
    float y[V][8], h[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[v][e] = h[v][e] = 0.f;
        if (c < j.d) {
            ld8(j.y, j.ydt, row + c, y[v]);
            if (j.h) ld8(j.h, j.hdt, row + c, h[v]);
        }
    }
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
        float g[8], w[8];
        gate8(j, t, c, g);
        ones8(w);
        if (j.w_post) ld8(j.w_post, j.wdt, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float z = j.post_norm ? y[v][e] * r1 * w[e] : y[v][e];
            h[v][e] = j.h ? j.alpha * h[v][e] + g[e] * z : g[e] * z;
            s2[0] += h[v][e] * h[v][e];
        }
        if (j.h_out) st8(j.h_out, j.hdt, row + c, h[v]);
    }
    if (j.xn == nullptr && j.rstd == nullptr) return;
    block_sum(s2, red[1]);
    const float r2 = 1.f / sqrtf(s2[0] / (float)j.d + j.eps);
    if (j.rstd && threadIdx.x == 0) {
        j.rstd[t] = r1;
        j.rstd[(int64_t)j.n + t] = r2;
    }
    if (j.xn == nullptr) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 8;
        if (c >= j.d) continue;
        float w[8];
        ones8(w);
        if (j.w_pre) ld8(j.w_pre, j.wdt, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= h[v][e] * r2;
        st8(j.xn, j.xdt, row + c, w);
    }
}

// Gradients.  A block walks over rows t = blockIdx.x, + gridDim.x, ... and
// keeps its column sums (dw_post, dw_pre, dgate per channel) in shared memory,
// each column owned by one thread.  With q = dxn w_pre, P = dh_out + r2 q and
// c = r2^3 / d the row's e = P - c S h_out, S = sum q h_out; the norm of y needs
// sum e gate z = sum P gate z - c S sum h_out gate z, so one reduction of three
// sums serves the row.
template <int V>
__global__ void __launch_bounds__(512) norm_join_bwd_kernel(const JoinJob j) {
    extern __shared__ __align__(16) float colsum[];  // [3][d], then 2 x 96 for the row sums
    float *red = colsum + 3 * j.d;
    const bool want[3] = {j.dw_post != nullptr, j.dw_pre != nullptr,
                          j.dgate != nullptr && j.gate_kind == MOE_GATE_CHANNEL};
    const bool row_gate = j.gate_kind == MOE_GATE_TOKEN || j.gate_kind == MOE_GATE_SCALAR;
    const float inv_d = 1.f / (float)j.d;
    float gate_sum = 0.f;
    for (int c = threadIdx.x; c < 3 * j.d; c += blockDim.x) colsum[c] = 0.f;
    __syncthreads();
    int flip = 0;
    for (int t = blockIdx.x; t < j.n; t += gridDim.x, flip ^= 1) {
        const int64_t row = (int64_t)t * j.d;
        const float r1 = j.post_norm ? j.rstd[t] : 1.f, r2 = j.rstd[(int64_t)j.n + t];
        float ho[V][8], y[V][8], P[V][8], dx[V][8];
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 8;
            if (c >= j.d) continue;
            float g[8], w[8];
            ld8(j.y, j.ydt, row + c, y[v]);
#pragma unroll
            for (int e = 0; e < 8; ++e) ho[v][e] = P[v][e] = dx[v][e] = 0.f;
            if (j.h) ld8(j.h, j.hdt, row + c, ho[v]);
            if (j.dh_out) ld8(j.dh_out, j.hdt, row + c, P[v]);
            if (j.dxn) ld8(j.dxn, j.xdt, row + c, dx[v]);
            gate8(j, t, c, g);
            ones8(w);
            if (j.w_post) ld8(j.w_post, j.wdt, c, w);
            float wp[8];
            ones8(wp);
            if (j.w_pre) ld8(j.w_pre, j.wdt, c, wp);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = j.post_norm ? y[v][e] * r1 * w[e] : y[v][e];
                ho[v][e] = j.h ? j.alpha * ho[v][e] + g[e] * z : g[e] * z;
                const float q = dx[v][e] * wp[e];
                P[v][e] += r2 * q;
                const float gz = row_gate ? z : g[e] * z;
                s[0] += q * ho[v][e];
                s[1] += P[v][e] * gz;
                s[2] += ho[v][e] * gz;
            }
        }
        block_sum(s, red + flip * 96);
        const float cS = r2 * r2 * r2 * inv_d * s[0];
        const float ez = s[1] - cS * s[2];  // sum e z (row gate) or sum e gate z
        float gr = 1.f;
        if (row_gate) {
            gr = ld_elem(j.gate, j.gdt, j.gate_kind == MOE_GATE_TOKEN ? t : 0);
            if (j.dgate && threadIdx.x == 0) {
                if (j.gate_kind == MOE_GATE_TOKEN)
                    st_elem(j.dgate, j.gdt, t, ez);
                else
                    gate_sum += ez;
            }
        }
        const float cy = r1 * r1 * inv_d * gr * ez;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 8;
            if (c >= j.d) continue;
            float g[8], w[8], o[8], dz[8];
            gate8(j, t, c, g);
            ones8(w);
            if (j.w_post) ld8(j.w_post, j.wdt, c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                P[v][e] -= cS * ho[v][e];
                o[e] = j.alpha * P[v][e];
                dz[e] = g[e] * P[v][e];
            }
            if (j.dh) st8(j.dh, j.hdt, row + c, o);
            if (j.dy) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = j.post_norm ? r1 * dz[e] * w[e] - y[v][e] * cy : dz[e];
                st8(j.dy, j.ydt, row + c, o);
            }
            if (j.dgate && (j.gate_kind == MOE_GATE_FULL || j.gate_kind == MOE_GATE_CHANNEL)) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = P[v][e] * (j.post_norm ? y[v][e] * r1 * w[e] : y[v][e]);
                if (j.gate_kind == MOE_GATE_FULL) {
                    st8(j.dgate, j.gdt, row + c, o);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) colsum[2 * j.d + c + e] += o[e];
                }
            }
            if (want[0])
#pragma unroll
                for (int e = 0; e < 8; ++e) colsum[c + e] += dz[e] * y[v][e] * r1;
            if (want[1])
#pragma unroll
                for (int e = 0; e < 8; ++e) colsum[j.d + c + e] += dx[v][e] * ho[v][e] * r2;
        }
    }
    float *part = j.part + (int64_t)blockIdx.x * 3 * j.d;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (want[k])
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = (v * blockDim.x + threadIdx.x) * 8;
                if (c >= j.d) continue;
#pragma unroll
                for (int e = 0; e < 8; e += 4)
                    *reinterpret_cast<float4 *>(part + k * j.d + c + e) =
                        *reinterpret_cast<const float4 *>(colsum + k * j.d + c + e);
            }
    if (threadIdx.x == 0) j.part[(int64_t)j.slots * 3 * j.d + blockIdx.x] = gate_sum;
}

// Adds the blocks' column sums in slot order: 32 columns x 8 slot lanes.
__global__ void __launch_bounds__(256) norm_join_sum_kernel(const JoinJob j) {
    __shared__ float red[8][33];
    const int k = blockIdx.y, q = threadIdx.x & 31, lane = threadIdx.x >> 5;
    void *dst = k == 0 ? j.dw_post : k == 1 ? j.dw_pre
                : j.gate_kind == MOE_GATE_CHANNEL ? j.dgate : nullptr;
    if (k < 3) {
        if (dst == nullptr) return;
        const int c = blockIdx.x * 32 + q;
        float s = 0.f;
        if (c < j.d)
            for (int i = lane; i < j.slots; i += 8) s += j.part[((int64_t)i * 3 + k) * j.d + c];
        red[lane][q] = s;
        __syncthreads();
        if (lane == 0 && c < j.d) {
            s = 0.f;
            for (int l = 0; l < 8; ++l) s += red[l][q];
            st_elem(dst, k == 2 ? j.gdt : j.wdt, c, s);
        }
    } else if (blockIdx.x == 0 && j.gate_kind == MOE_GATE_SCALAR && j.dgate) {
        if (threadIdx.x == 0) {
            float s = 0.f;
            for (int i = 0; i < j.slots; ++i) s += j.part[(int64_t)j.slots * 3 * j.d + i];
            st_elem(j.dgate, j.gdt, 0, s);
        }
    }
}

int threads_for(int d, int v) {
    const int t = (d / 8 + v - 1) / v;
    return (t + 31) / 32 * 32;
}

template <int V>
rvq_status launch_bwd(const JoinJob &j, cudaStream_t stream) {
    const size_t smem = ((size_t)3 * j.d + 2 * 96) * 4;
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(norm_join_bwd_kernel<V>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (3 * kJoinMaxD + 2 * 96) * 4));
        attr_done[dev] = 1;
    }
    norm_join_bwd_kernel<V><<<j.slots, threads_for(j.d, V), smem, stream>>>(j);
    RVQ_LAUNCHED("norm_join_bwd");
    return RVQ_OK;
}

}  // namespace

int join_bwd_slots(int n, int d) {
    (void)d;
    const int want = 2 * num_sms();
    return n < want ? n : want;
}

rvq_status launch_norm_join(const JoinJob &job, cudaStream_t stream) {
    const unsigned n = (unsigned)job.n;
    if (job.d <= 2048)
        norm_join_kernel<1><<<n, threads_for(job.d, 1), 0, stream>>>(job);
    else if (job.d <= 8192)
        norm_join_kernel<2><<<n, threads_for(job.d, 2), 0, stream>>>(job);
    else
        norm_join_kernel<4><<<n, threads_for(job.d, 4), 0, stream>>>(job);
    RVQ_LAUNCHED("norm_join");
    return RVQ_OK;
}

rvq_status launch_norm_join_bwd(const JoinJob &job, cudaStream_t stream) {
    if (job.d <= 4096)
        RVQ_TRY(launch_bwd<1>(job, stream));
    else if (job.d <= 8192)
        RVQ_TRY(launch_bwd<2>(job, stream));
    else
        RVQ_TRY(launch_bwd<4>(job, stream));
    const bool chan = job.dgate && (job.gate_kind == MOE_GATE_CHANNEL ||
                                    job.gate_kind == MOE_GATE_SCALAR);
    if (job.dw_post || job.dw_pre || chan) {
        norm_join_sum_kernel<<<dim3((unsigned)((job.d + 31) / 32), 4), 256, 0, stream>>>(job);
        RVQ_LAUNCHED("norm_join_sum");
    }
    return RVQ_OK;
}

}  // namespace rvq
