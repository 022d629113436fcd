// moe_norm_join_mx: moe_norm_join with the normed rows microscaled on the way out.
//
//   z = post_norm ? y r1 w_post : y,  h' = alpha h + gate z,  xn = h' r2 w_pre,
//   r = 1 / sqrt(mean of squares + eps); xn's blocks of 32 scaled and rounded
//
// Memory-bound: h and y in, h' and a byte (or half) per value out.  Few rows, and types
// without an instance below: one block per row, a thread's columns (groups of eight, a
// block's width apart) in registers; four adjacent lanes hold a block of 32.  Many rows:
// blocks walk over them; a row is copied into shared memory (cp.async) while the one
// before is worked on in registers, so one place is enough and two blocks or more share
// an SM, whose sums and round trips overlap (a ring of two or three rows, one block of
// fp32 7168 per SM, took 44 and 53 us for 2048 rows where this takes 34).  A thread's
// groups are of four columns, eight adjacent lanes hold a block of 32 and a warp the 128
// columns of a word of scales.
//
// Measured (GB300, 8 bits out): 2048 x 7168 fp32 with a post norm and a channel gate 34 us
// (191 MB, 5.6 TB/s), fp32 stream and bf16 block 28.7 (5.6), all bf16 28.7 (3.6: issue, 45
// instructions per value and lane); 1531 x 2040 bf16 7.7; 64 x 7168 3.6.
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

// Four columns of a row per lane, whole warps together: the codes at `codes`, and the word
// of scales of the warp's 128 columns at `scales`.
template <int FMT>
__device__ __forceinline__ void mx_put4(const Four &x, uint8_t *codes, uint8_t *scales, bool on) {
    constexpr uint32_t kAbs = 0x7FFFFFFFu;
    uint32_t top = max(max(__float_as_uint(x.a.x) & kAbs, __float_as_uint(x.a.y) & kAbs),
                       max(__float_as_uint(x.b.x) & kAbs, __float_as_uint(x.b.y) & kAbs));
#pragma unroll
    for (int o = 1; o < 8; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t byte = mx_byte<FMT>(top);
    const Four q = x * four(mx_inverse(byte));
    if (FMT == MOE_MX_F8) {
        const uint32_t w = byte == 255 ? 0u : e4m3x4(q.a.x, q.a.y, q.b.x, q.b.y);
        if (on) *reinterpret_cast<uint32_t *>(codes) = w;
    } else {
        const float v[8] = {q.a.x, q.a.y, q.b.x, q.b.y, 0.f, 0.f, 0.f, 0.f};
        const uint16_t w = byte == 255 ? (uint16_t)0 : (uint16_t)e2m1x8(v);
        if (on) *reinterpret_cast<uint16_t *>(codes) = w;
    }
    uint32_t word = byte << (threadIdx.x & 24);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    word |= __shfl_xor_sync(0xffffffffu, word, 16);
    if (on && (threadIdx.x & 31) == 0) *reinterpret_cast<uint32_t *>(scales) = word;
}

// The sum of v over a block of up to 16 warps, in the warps' order; `red`: 16 floats, of
// which those of absent warps are 0.
__device__ __forceinline__ float sum_of_block(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 p = reinterpret_cast<const float4 *>(red)[i];
        s = (((s + p.x) + p.y) + p.z) + p.w;
    }
    return s;
}

// Where a walking block keeps things in shared memory (bytes): a row on its way in, and the
// gains; `pad` columns long, zeros past the last.
struct MxRow {
    int pad;               // columns
    int h, gate;           // places in the row, after y
    int zero;              // a row of zeros for an absent h
    int out, in;           // gains: w_post (times a channel gate, then fp32), w_pre
    int out_dt, total;
};

MxRow row_layout(const JoinJob &j) {
    MxRow L = {};
    const auto bytes = [&](int dt) { return L.pad * (dt == RVQ_F32 ? 4 : 2); };
    L.pad = join_threads(j.d, 4, 4) * 16;
    L.h = bytes(j.ydt);
    L.gate = L.h + (j.h ? bytes(j.hdt) : 0);
    L.zero = L.gate + (j.gate_kind == MOE_GATE_FULL ? bytes(j.gdt) : 0);
    L.out = L.zero + (j.h ? 0 : bytes(j.hdt));
    L.out_dt = j.gate_kind == MOE_GATE_CHANNEL ? (int)RVQ_F32 : j.wdt;
    L.in = L.out + bytes(L.out_dt);
    L.total = L.in + bytes(j.wdt);
    return L;
}

// Zeros past the rows' ends, an absent h, and the gains, four columns at a time; rows
// already in flight are not touched.  (d and pad are multiples of eight.)
template <int W, int GATE>
__device__ __forceinline__ void fill_row(uint8_t *smem, const JoinJob &j, const MxRow &L) {
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    const int c0 = threadIdx.x * 4, step = blockDim.x * 4;
    for (int i = j.d + c0; i < L.pad; i += step) {
        st4(smem, j.ydt, i, zero);
        if (j.h) st4(smem + L.h, j.hdt, i, zero);
        if (GATE == 2) st4(smem + L.gate, j.gdt, i, zero);
    }
    for (int i = c0; i < (L.out - L.zero) / 4; i += step) st4(smem + L.zero, RVQ_F32, i, zero);
#pragma unroll 4
    for (int i = c0; i < L.pad; i += step) {
        const float x = i < j.d ? 1.f : 0.f;
        float a[4] = {x, x, x, x}, b[4] = {x, x, x, x}, g[4] = {x, x, x, x};
        if (i < j.d && j.w_post) ld4(j.w_post, W, i, a);
        if (i < j.d && j.w_pre) ld4(j.w_pre, W, i, b);
        if (GATE == 1 && i < j.d) ld4(j.gate, j.gdt, i, g);
        if (GATE == 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] *= g[e];
        st4(smem + L.out, GATE == 1 ? (int)RVQ_F32 : W, i, a);
        st4(smem + L.in, W, i, b);
    }
}

// GATE 0: one value per row or none, 1: per channel, 2: full, of h's type.
template <int H, int Y, int W, int GATE>
__global__ void __launch_bounds__(512, 2) mx_join_walk_kernel(const MxJoinJob job, const MxRow L) {
    constexpr int V = 4;
    constexpr bool FULL = GATE == 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[4][16];
    const JoinJob &j = job.join;
    const int tiles = mx_tiles(j.d), G = gridDim.x;
    const bool has_h = j.h != nullptr;
    const float inv_d = 1.f / (float)j.d, alpha = has_h ? j.alpha : 0.f;
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t at_h = at + (has_h ? L.h : L.zero);
    const auto fetch = [&](int t) {
        if (t < j.n) {
            const int64_t row = (int64_t)t * j.d;
            fetch_row<V, Y>(at, j.y, j.ydt, row, j.d);
            if (has_h) fetch_row<V, H>(at + L.h, j.h, j.hdt, row, j.d);
            if (FULL) fetch_row<V, H>(at + L.gate, j.gate, j.gdt, row, j.d);
        }
        cp_commit();
    };
    // places of absent warps are added too; a block may have fewer threads than places
    for (int i = threadIdx.x; i < 64; i += blockDim.x) red[i >> 4][i & 15] = 0.f;
    int t = blockIdx.x;
    dependency_wait();
    fetch(t);
    fill_row<W, GATE>(smem, j, L);
    float g_next = 1.f;
    if (j.gate_kind == MOE_GATE_SCALAR) g_next = ld_elem(j.gate, j.gdt, 0);
    if (j.gate_kind == MOE_GATE_TOKEN && t < j.n) g_next = ld_elem(j.gate, j.gdt, t);
    int flip = 0;
    for (; t < j.n; t += G, flip ^= 2) {
        cp_wait<0>();
        __syncthreads();  // this row has arrived everywhere
        const float gt = g_next;
        const int64_t row = (int64_t)t * j.d;
        Four y[V], h[V], g[FULL ? V : 1];
        Four q = four(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            lds4<Y>(at, c, j.ydt, y[v]);
            lds4<H>(at_h, c, j.hdt, h[v]);
            if (FULL) lds4<H>(at + L.gate, c, j.gdt, g[v]);
            q = fma4(y[v], y[v], q);
        }
        __syncthreads();  // and is read everywhere: the next one takes its place
        fetch(t + G);
        if (j.gate_kind == MOE_GATE_TOKEN && t + G < j.n) g_next = ld_elem(j.gate, j.gdt, t + G);
        float r1 = 1.f;
        if (j.post_norm) {
            r1 = 1.f / sqrtf(sum_of_block(sum4(q), red[flip]) * inv_d + j.eps);
        }
        q = four(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            Four w;
            lds4<GATE == 1 ? (int)RVQ_F32 : W>(at + L.out, c, 0, w);
            Four z = y[v] * four(r1) * w;
            if (FULL) z = g[v] * z;
            h[v] = fma4(four(gt), z, four(alpha) * h[v]);
            q = fma4(h[v], h[v], q);
            put4<H>(j.h_out, row + c, j.h_out != nullptr && c < j.d, j.hdt, h[v]);
        }
        const float r2 = 1.f / sqrtf(sum_of_block(sum4(q), red[flip + 1]) * inv_d + j.eps);
        if (j.rstd && threadIdx.x == 0) {
            j.rstd[t] = r1;
            j.rstd[(int64_t)j.n + t] = r2;
        }
        uint8_t *codes = job.codes + (int64_t)t * tiles * (job.fmt == MOE_MX_F8 ? 128 : 64);
        uint8_t *scales = job.scales + mx_scale_at(t, 0, tiles);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = v * blockDim.x + threadIdx.x, c = 4 * i;
            Four w;
            lds4<W>(at + L.in, c, 0, w);
            const Four x = c < j.d ? h[v] * four(r2) * w : four(0.f);
            put4<kAny>(j.xn, row + c, j.xn != nullptr && c < j.d, j.xdt, x);
            const bool on = c < tiles * kMxTile;
            uint8_t *sc = scales + (i >> 5) * kMxTileBytes;
            if (job.fmt == MOE_MX_F8)
                mx_put4<MOE_MX_F8>(x, codes + c, sc, on);
            else
                mx_put4<MOE_MX_F4>(x, codes + c / 2, sc, on);
        }
    }
    cp_wait<0>();
}

// Walking blocks, as many as an SM holds at once.
template <int H, int Y, int W, int GATE>
rvq_status walk(const MxJoinJob &job, cudaStream_t stream) {
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    constexpr auto K = mx_join_walk_kernel<H, Y, W, GATE>;
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax));
        attr_done[dev] = 1;
    }
    const int threads = join_threads(job.join.d, 4, 4);
    const MxRow L = row_layout(job.join);
    int per = 0;
    RVQ_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, K, threads, (size_t)L.total));
    const int blocks = (per < 1 ? 1 : per) * num_sms(), n = job.join.n;
    RVQ_CUDA(launch_after(K, (unsigned)(n < blocks ? n : blocks), (unsigned)threads, (size_t)L.total,
                          stream, job, L));
    return RVQ_OK;
}

// Whether blocks walk over the rows: more rows than the row kernel holds at once, long or
// many enough to pay for the setup (walked and a block per row, fp32 stream, bf16 block, post
// norm, past L2: 2048 x 512 4.9 and 5.1 us; 2048 x 1536 9.1 and 11.5; 4200 x 512 7.8 and
// 7.1, 8192 x 512 10.8 and 12.8; 20000 x 72 18.1 and 20.8; 2048 x 7168 32.9 and 45.4; rows
// that L2 holds, 2048 x 512 4.4 and 3.5); one fits with its gains, and the types have an
// instance (fp32 or bf16 rows and gains, a full gate of h's type).
bool walks(const JoinJob &j) {
    return j.n > 2 * num_sms() && (j.d > 1024 || j.n > 4096) && j.d <= 8192 && j.hdt != RVQ_F16 &&
           j.ydt != RVQ_F16 && j.wdt != RVQ_F16 &&
           (j.gate_kind != MOE_GATE_FULL || j.gdt == j.hdt) && row_layout(j).total <= kSmemMax;
}

template <int H, int Y, int W>
rvq_status walk_gate(const MxJoinJob &job, cudaStream_t stream) {
    if (job.join.gate_kind == MOE_GATE_FULL) return walk<H, Y, W, 2>(job, stream);
    if (job.join.gate_kind == MOE_GATE_CHANNEL) return walk<H, Y, W, 1>(job, stream);
    return walk<H, Y, W, 0>(job, stream);
}

template <int H, int Y>
rvq_status walk_gains(const MxJoinJob &job, cudaStream_t stream) {
    return job.join.wdt == RVQ_F32 ? walk_gate<H, Y, RVQ_F32>(job, stream)
                                   : walk_gate<H, Y, RVQ_BF16>(job, stream);
}

rvq_status walk_types(const MxJoinJob &job, cudaStream_t stream) {
    const bool h32 = job.join.hdt == RVQ_F32, y32 = job.join.ydt == RVQ_F32;
    if (h32 && y32) return walk_gains<RVQ_F32, RVQ_F32>(job, stream);
    if (h32) return walk_gains<RVQ_F32, RVQ_BF16>(job, stream);
    if (y32) return walk_gains<RVQ_BF16, RVQ_F32>(job, stream);
    return walk_gains<RVQ_BF16, RVQ_BF16>(job, stream);
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
    if (walks(job.join))
        return walk_types(job, stream);
    return job.fmt == MOE_MX_F8 ? by_size<MOE_MX_F8>(job, stream)
                                : by_size<MOE_MX_F4>(job, stream);
}

}  // namespace rvq
