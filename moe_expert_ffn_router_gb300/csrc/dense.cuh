// Internal declarations of the dense (unquantised) operators beside the routed
// experts: moe_linear, moe_gated_linear and their gradients (dense_api.cu,
// dense_gemm.cu, dense_bwd.cu) and moe_norm_join (norm_join.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"

namespace rvq {

// ---------------------------------------------------------------- launches
// The dense operators' kernels are launched programmatically: a kernel's blocks
// may start as those of the kernel before it on the stream end, and touch memory
// only after dependency_wait(), which waits for that kernel's end.  Only short
// kernels call dependents_may_start() (those for few rows, and the elementwise
// gradients, whose products then start 1 to 2 us sooner): waiting blocks of the next
// kernel hold shared memory, and with the walking kernels of moe_norm_join that cost
// more than the launch (forward and gradients of 4099 x 2048: 70 us, 54 us without).
__device__ __forceinline__ void dependency_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void dependents_may_start() {
    asm volatile("griddepcontrol.launch_dependents;");
}

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- elements
// Scalars and groups of eight of the three element types, as fp32.
__device__ __forceinline__ float ld_elem(const void *p, int dt, int64_t i) {
    if (dt == RVQ_F32) return reinterpret_cast<const float *>(p)[i];
    const uint16_t b = reinterpret_cast<const uint16_t *>(p)[i];
    if (dt == RVQ_BF16) return __uint_as_float((uint32_t)b << 16);
    return __half2float(__ushort_as_half(b));
}

__device__ __forceinline__ void st_elem(void *p, int dt, int64_t i, float v) {
    if (dt == RVQ_F32)
        reinterpret_cast<float *>(p)[i] = v;
    else if (dt == RVQ_BF16)
        reinterpret_cast<uint16_t *>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        reinterpret_cast<uint16_t *>(p)[i] = __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ uint32_t pack16(int dt, float lo, float hi) {
    if (dt == RVQ_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void unpack16(int dt, uint32_t w, float &lo, float &hi) {
    if (dt == RVQ_BF16) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        lo = f.x;
        hi = f.y;
    }
}

// eight consecutive elements at a 16-byte aligned place
__device__ __forceinline__ void ld8(const void *p, int dt, int64_t i, float (&v)[8]) {
    if (dt == RVQ_F32) {
        const float4 *q = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 q = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(p) + i);
        unpack16(dt, q.x, v[0], v[1]);
        unpack16(dt, q.y, v[2], v[3]);
        unpack16(dt, q.z, v[4], v[5]);
        unpack16(dt, q.w, v[6], v[7]);
    }
}

__device__ __forceinline__ void st8(void *p, int dt, int64_t i, const float (&v)[8]) {
    if (dt == RVQ_F32) {
        float4 *q = reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p) + i) =
            make_uint4(pack16(dt, v[0], v[1]), pack16(dt, v[2], v[3]), pack16(dt, v[4], v[5]),
                       pack16(dt, v[6], v[7]));
    }
}

// four consecutive elements at a place that is a multiple of four
__device__ __forceinline__ void ld4(const void *p, int dt, int64_t i, float (&v)[4]) {
    if (dt == RVQ_F32) {
        const float4 q = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
        const uint2 q = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + i);
        unpack16(dt, q.x, v[0], v[1]);
        unpack16(dt, q.y, v[2], v[3]);
    }
}

__device__ __forceinline__ void st4(void *p, int dt, int64_t i, const float (&v)[4]) {
    if (dt == RVQ_F32)
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + i) =
            make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p) + i) =
            make_uint2(pack16(dt, v[0], v[1]), pack16(dt, v[2], v[3]));
}

// ------------------------------------------------------------- activations
// 1 / (1 + exp(-v)) from the hardware exponential and reciprocal: relative
// error below 2^-22 + |v| 2^-23 (the argument's rounding), 0 and 1 at the ends.
__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// argument of the sigmoid that the tanh form of GELU multiplies v with:
// (1 + tanh(t)) / 2 = sigmoid(2 t), t = sqrt(2/pi) (v + 0.044715 v^3)
__device__ __forceinline__ float gelu_tanh_arg(float v) {
    return 1.5957691216057308f * (v + 0.044715f * v * v * v);
}

// Normal distribution function of v and exp(-v^2 / 2), of one exponential: the tail
// beyond |v| is e^(-v^2 / 2) t p(t), t = 1 / (1 + 0.3 |v|), with p fitted to the tail's
// ratio to the exponential in relative error (degree 7, Lawson's reweighted least
// squares over |v| <= 14: 1.5e-7, and 4.3e-7 with the evaluation in fp32), so a
// negative v keeps its relative accuracy as far as fp32 reaches.  erff and expf made
// the gradients of GELU compute-bound.
__device__ __forceinline__ float normal_cdf(float v, float &e) {
    e = __expf(-0.5f * v * v);
    const float t = __fdividef(1.f, 1.f + 0.3f * fabsf(v));
    float p = 3.567477157e-2f;
    p = p * t - 0.1572030725f;
    p = p * t + 0.2063534899f;
    p = p * t - 5.368363016e-2f;
    p = p * t + 0.1285616198f;
    p = p * t + 9.991349398e-2f;
    p = p * t + 0.1207539558f;
    p = p * t + 0.1196292988f;
    const float q = p * t * e;  // the tail beyond |v|
    return v < 0.f ? q : 1.f - q;
}

template <int ACT>
__device__ __forceinline__ float act_value_of(float v) {
    if (ACT == MOE_ACT_RELU) return v > 0.f ? v : (v != v ? v : 0.f);
    if (ACT == MOE_ACT_SILU) return __fdividef(v, 1.f + __expf(-v));
    if (ACT == MOE_ACT_GELU) {
        float e;
        return v * normal_cdf(v, e);
    }
    if (ACT == MOE_ACT_GELU_TANH) return __fdividef(v, 1.f + __expf(-gelu_tanh_arg(v)));
    return v;
}

template <int ACT>
__device__ __forceinline__ float act_slope_of(float v) {
    if (ACT == MOE_ACT_RELU) return v > 0.f ? 1.f : 0.f;
    if (ACT == MOE_ACT_SILU) {
        const float s = sigmoid_f(v);
        return s * (1.f + v * (1.f - s));
    }
    if (ACT == MOE_ACT_GELU) {
        float e;
        const float c = normal_cdf(v, e);
        return c + v * 0.39894228040143268f * e;
    }
    if (ACT == MOE_ACT_GELU_TANH) {
        // beyond |v| = 16 the slope is 0 or 1 to fp32, and v * v * v may overflow
        if (v >= 16.f) return 1.f;
        if (v <= -16.f) return 0.f;
        const float s = sigmoid_f(gelu_tanh_arg(v));
        return s + v * s * (1.f - s) * 1.5957691216057308f * (1.f + 3.f * 0.044715f * v * v);
    }
    return 1.f;
}

// one branch per group of values, not per value
template <int ACT, int N>
__device__ __forceinline__ void act_values(float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = act_value_of<ACT>(v[e]);
}

template <int N>
__device__ __forceinline__ void act_group(int act, float (&v)[N]) {
    switch (act) {
        case MOE_ACT_RELU: act_values<MOE_ACT_RELU>(v); break;
        case MOE_ACT_SILU: act_values<MOE_ACT_SILU>(v); break;
        case MOE_ACT_GELU: act_values<MOE_ACT_GELU>(v); break;
        case MOE_ACT_GELU_TANH: act_values<MOE_ACT_GELU_TANH>(v); break;
        default: break;
    }
}

// v -> (act(v), act'(v)); the value only if wanted
template <int ACT, bool VALUE, int N>
__device__ __forceinline__ void act_both(const float (&v)[N], float (&a)[N], float (&s)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (VALUE) a[e] = act_value_of<ACT>(v[e]);
        s[e] = act_slope_of<ACT>(v[e]);
    }
}

template <bool VALUE, int N>
__device__ __forceinline__ void act_group_both(int act, const float (&v)[N], float (&a)[N],
                                               float (&s)[N]) {
    switch (act) {
        case MOE_ACT_RELU: act_both<MOE_ACT_RELU, VALUE>(v, a, s); break;
        case MOE_ACT_SILU: act_both<MOE_ACT_SILU, VALUE>(v, a, s); break;
        case MOE_ACT_GELU: act_both<MOE_ACT_GELU, VALUE>(v, a, s); break;
        case MOE_ACT_GELU_TANH: act_both<MOE_ACT_GELU_TANH, VALUE>(v, a, s); break;
        default: act_both<MOE_ACT_NONE, VALUE>(v, a, s); break;
    }
}

// --------------------------------------------------------------------- GEMM
// One product, or two that share an operand or an output, for one launch:
//   PLAIN   out0[m][n] = sum_k A0[m][k] B0[n][k]
//   GATED   g = A0 B0^T, u = A0 B1^T; out0 = act(g + bias0) * (u + bias1)
//   SUM_K   out0 = A0 B0^T + A1 B1^T
//   PAIR_M  out0 = A0 B0^T, out1 = A1 B0^T
// An operand is stored K-contiguous ([rows][K]) or, with *_t set, as its
// transpose ([K][rows]).  out0 = residual + alpha * act(product + bias0) in the
// other modes.  pre (fp32, contiguous [M][N]) receives product + bias.
enum DgMode { DG_PLAIN = 0, DG_GATED = 1, DG_SUM_K = 2, DG_PAIR_M = 3 };
struct DenseJob {
    int mode;
    int M, N, K;
    int a_t, b_t;
    const void *a[2];
    int64_t lda;
    const void *b[2];
    int64_t ldb;
    int dt;                 // of A, B and the biases: RVQ_BF16 or RVQ_F16
    const void *bias[2];
    int act;
    float alpha;
    const void *residual;
    int rdt;
    int64_t ldr;
    void *out[2];
    int odt;
    int64_t ldo;
    float *pre[2];
    uint32_t *status;       // the workspace's status block
    float *partial;         // dense_gemm_partial_bytes of workspace
};
size_t dense_gemm_partial_bytes(const DenseJob &job);  // grows with M, N and K
rvq_status launch_dense_gemm(const DenseJob &job, cudaStream_t stream);
// Sums of a bias gradient still to be added: dbias[m][col] (NULL: not wanted) from
// the fp32 partials part[chunk][m][col].
struct BiasSums {
    const float *part;
    int chunks, mats, rows, dt;
    void *dbias[2];
    __host__ __device__ bool wanted() const { return dbias[0] || dbias[1]; }
};
// Two products without a common output (not GATED; one dt), in one launch where
// that is faster; one whose out[0] is NULL is not wanted.  Adds the bias gradients
// along with them.
rvq_status launch_dense_gemm_two(const DenseJob &x, const DenseJob &y, const BiasSums &sums,
                                 cudaStream_t stream);
// rvq_selftest_dense_plan's answer for one product or the two of a gradient
void dense_plan_of(const DenseJob &x, const DenseJob *y, int32_t (&out)[7]);
// launch_dense_gemm for few tokens as the rows of A: the weights streamed past the
// batch (dense_stream.cu)
constexpr int kStreamMaxTokens = 192;
bool dense_stream_fits(const DenseJob &job);
rvq_status launch_dense_stream(const DenseJob &job, cudaStream_t stream);

// Gradient of the gated product (mats = 2) or of an activation (mats = 1):
//   mats 2: dp0 = dout * pre1 * act'(pre0), dp1 = dout * act(pre0)
//   mats 1: dp0 = alpha * dout * act'(pre0)      (pre0 NULL: act' = 1)
// dp (16-bit [n][rows] each, NULL: not written) and, with dbias[i] set, the
// partial sums over the n rows (fp32 [chunks][mats][rows] in part), which
// launch_dense_gemm_two or launch_bias_sums adds.
struct DenseBwdJob {
    int mats, n, rows, act;
    float alpha;
    const void *dout;
    int64_t ldd;
    int dt;
    const float *pre[2];
    void *dp[2];
    void *dbias[2];
    float *part;
    int wide;               // pre starts on 32 bytes (rows are multiples of eight)
};
constexpr int kBwdChunkRows = 32;  // rows per partial of a bias gradient
inline int dense_bwd_chunks(int n) { return (n + kBwdChunkRows - 1) / kBwdChunkRows; }
rvq_status launch_dense_bwd(const DenseBwdJob &job, cudaStream_t stream);
// Adds the partials of bias gradients: eight columns per warp and turn, the chunks
// dealt to four lanes each, whose sums are added in a fixed order.
__device__ __forceinline__ void add_bias_sums(const BiasSums &s, int warp, int warps, int lane) {
    const int col = lane & 7, first = lane >> 3;
    const int groups = s.rows / 8;
    const int64_t step = (int64_t)s.mats * s.rows;
    for (int i = warp; i < s.mats * groups; i += warps) {
        const int m = i / groups, c = (i - m * groups) * 8 + col;
        if (s.dbias[m] == nullptr) continue;
        const float *p = s.part + (int64_t)m * s.rows + c;
        float sum = 0.f;
#pragma unroll 8
        for (int k = first; k < s.chunks; k += 4) sum += p[k * step];
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (first == 0) st_elem(s.dbias[m], s.dt, c, sum);
    }
}

BiasSums bias_sums_of(const DenseBwdJob &job);
rvq_status launch_bias_sums(const BiasSums &s, cudaStream_t stream);

// ---------------------------------------------------------------- norm join
struct JoinJob {
    int n, d;
    float eps, alpha;
    const void *h, *y, *gate, *w_post, *w_pre;
    int hdt, ydt, gdt, wdt;
    int gate_kind, post_norm;
    void *h_out, *xn;
    int xdt;
    float *rstd;            // [2][n]: of y (1 without a post norm), of h_out
    // gradients
    const void *dh_out, *dxn;
    void *dh, *dy, *dgate, *dw_post, *dw_pre;
    float *part;            // [slots][3][d] column sums, then [slots] scalar sums
    int slots;              // blocks of the gradient kernel
};
constexpr int kJoinMaxD = 16384;
int join_bwd_slots(int n, int d);  // at most, for the workspace
rvq_status launch_norm_join(const JoinJob &job, cudaStream_t stream);
rvq_status launch_norm_join_bwd(const JoinJob &job, cudaStream_t stream);

}  // namespace rvq
