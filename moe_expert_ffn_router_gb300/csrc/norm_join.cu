// moe_norm_join: the norm after a block, its gate, the scaled residual and the
// norm before the next block, in one pass over the rows.
//
// Memory-bound (a few operations per byte): every input is read once and every
// output written once, so the design keeps bytes in flight.  Many rows: blocks
// walk over them with a ring of rows in shared memory (join_walk.cuh).  Few rows:
// one block per row, here.  All sums are fp32: a thread's columns in order, then
// the warp's by shuffles, then the warps' in order.
#include "join_common.cuh"

namespace rvq {
namespace {

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

// Few rows: one block per row, loads straight to registers.
template <int V>
__global__ void __launch_bounds__(1024) join_row_kernel(const JoinJob j) {
    __shared__ float red[2][32];
    const int t = blockIdx.x;
    const int64_t row = (int64_t)t * j.d;
    dependency_wait();
    dependents_may_start();
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

// Adds the blocks' sums: 32 columns (a quad per thread) x up to 128 lanes, a lane's
// blocks in order, then the lanes in a fixed order.
__global__ void __launch_bounds__(1024) join_sum_kernel(const JoinJob j) {
    __shared__ float red[32][32];
    const int k = blockIdx.y, q = threadIdx.x & 7, lane = threadIdx.x >> 3, lanes = blockDim.x >> 3;
    void *dst = k == 0 ? j.dw_post : k == 1 ? j.dw_pre
                : j.gate_kind == MOE_GATE_CHANNEL ? j.dgate : nullptr;
    dependency_wait();
    const bool scalar = k == 2 && j.gate_kind == MOE_GATE_SCALAR && j.dgate && blockIdx.x == 0;
    if (scalar) {
        if (threadIdx.x == 0) {
            float s = 0.f;
#pragma unroll 8
            for (int i = 0; i < j.slots; ++i) s += j.part[(int64_t)j.slots * 3 * j.d + i];
            st_elem(j.dgate, j.gdt, 0, s);
        }
        return;
    }
    if (dst == nullptr) return;
    const int c = blockIdx.x * 32 + q * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < j.d) {
        const float *p = j.part + (int64_t)k * j.d + c;
#pragma unroll 8
        for (int i = lane; i < j.slots; i += lanes) {
            const float4 o = *reinterpret_cast<const float4 *>(p + (int64_t)i * 3 * j.d);
            s = make_float4(s.x + o.x, s.y + o.y, s.z + o.z, s.w + o.w);
        }
    }
#pragma unroll
    for (int o = 8; o < 32; o *= 2) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
        s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
        s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
    }
    if ((threadIdx.x & 31) < 8) *reinterpret_cast<float4 *>(&red[threadIdx.x >> 5][q * 4]) = s;
    __syncthreads();
    const int col = blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x < 32 && col < j.d) {
        float t = 0.f;
#pragma unroll 8
        for (int w = 0; w < lanes / 4; ++w) t += red[w][threadIdx.x];
        st_elem(dst, k == 2 ? j.gdt : j.wdt, col, t);
    }
}

}  // namespace

int join_bwd_slots(int n, int d) {
    const int most = join_bwd_blocks(d) * num_sms();
    return n < most ? n : most;
}

rvq_status launch_norm_join(const JoinJob &job, cudaStream_t stream) {
    if (job.n <= 2 * num_sms()) {
        const unsigned n = (unsigned)job.n;
        if (job.d <= 8192)
            RVQ_CUDA(launch_after(join_row_kernel<1>, n, join_threads(job.d, 8, 1), 0, stream, job));
        else
            RVQ_CUDA(launch_after(join_row_kernel<2>, n, join_threads(job.d, 8, 2), 0, stream, job));
        return RVQ_OK;
    }
    JoinJob j = job;
    return join_walk(j, false, stream);
}

rvq_status launch_norm_join_bwd(const JoinJob &job, cudaStream_t stream) {
    JoinJob j = job;
    RVQ_TRY(join_walk(j, true, stream));
    const bool gate = j.dgate && (j.gate_kind == MOE_GATE_CHANNEL || j.gate_kind == MOE_GATE_SCALAR);
    if (j.dw_post || j.dw_pre || gate) {
        // the blocks' sums over rows, in order (no atomics: results repeat)
        const int lanes = j.slots < 256 ? 32 : 128;
        RVQ_CUDA(launch_after(join_sum_kernel, dim3((unsigned)((j.d + 31) / 32), 3), 8 * lanes, 0,
                              stream, j));
    }
    return RVQ_OK;
}

}  // namespace rvq
