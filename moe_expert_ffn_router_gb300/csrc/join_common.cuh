// Shared parts of moe_norm_join and its gradients (norm_join.cu, join_walk.cuh):
// sums over a block, a ring of rows in shared memory, and the launch of blocks
// that walk over the rows.
//
// A walking block's thread owns the same columns of every row: groups of four,
// a block's width apart, so that a warp's accesses are contiguous for every
// type.  The next row is copied into a ring of two while one is worked on
// (cp.async).  Inner loops have no branches: a type is a template parameter, an
// absent tensor is a row of zeros.  With types looked up at run time every
// load's latency was exposed: 56 us against 36 us for 2048 rows of 7168 (fp32 h
// and y, bf16 xn).
//
// Measured (GB300): forward of 2048 x 7168 36 us (fp32 h and y, bf16 xn: 206 MB,
// 5.7 TB/s) and 26 us (bf16: 118 MB, 4.5 TB/s), of 4099 x 2048 (bf16) 16 us; forward and
// gradients 126, 82 and 45 us.  The forward call is bound by memory; the gradients
// by issue and latency (57 % of the issue slots with 16 warps an SM; the sums over
// rows hold up to 48 registers a thread), of long fp32 rows by copies that wait
// for the row before, where two rows do not fit (join_ring): past 6144 columns with
// fp32 gains and a 16-bit xn, 7168 with 16-bit gains too.
#pragma once

#include <type_traits>

#include "dense.cuh"

namespace rvq {

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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------- groups of four values
// DT: an rvq_dtype, or kAny (the type is looked up in dt).
constexpr int kAny = -1;

// Four fp32 values as two pairs: the arithmetic runs on packed pairs (half the
// instructions; the gradients' kernel issues more than it loads).
struct Four {
    float2 a, b;
};
__device__ __forceinline__ Four four(float x) {
    return {make_float2(x, x), make_float2(x, x)};
}
__device__ __forceinline__ Four operator*(const Four &x, const Four &y) {
    return {__fmul2_rn(x.a, y.a), __fmul2_rn(x.b, y.b)};
}
__device__ __forceinline__ Four fma4(const Four &x, const Four &y, const Four &z) {
    return {__ffma2_rn(x.a, y.a, z.a), __ffma2_rn(x.b, y.b, z.b)};
}
__device__ __forceinline__ float sum4(const Four &x) {
    return (x.a.x + x.a.y) + (x.b.x + x.b.y);
}

template <int DT>
__device__ __forceinline__ int type_of(int dt) {
    return DT == kAny ? dt : DT;
}

__device__ __forceinline__ int esize(int dt) { return dt == RVQ_F32 ? 4 : 2; }

__device__ __forceinline__ void widen4(uint2 r, int dt, Four &v) {
    unpack16(dt, r.x, v.a.x, v.a.y);
    unpack16(dt, r.y, v.b.x, v.b.y);
}

// four values at element i of a row in shared memory (byte address `at`)
template <int DT>
__device__ __forceinline__ void lds4(uint32_t at, int i, int dt, Four &v) {
    const int t = type_of<DT>(dt);
    if (t == RVQ_F32) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.a.x), "=f"(v.a.y), "=f"(v.b.x), "=f"(v.b.y)
                     : "r"(at + i * 4)
                     : "memory");
    } else {
        uint2 r;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(r.x), "=r"(r.y)
                     : "r"(at + i * 2)
                     : "memory");
        widen4(r, t, v);
    }
}

// four values in global memory; `none` when off
template <int DT>
__device__ __forceinline__ void ldg4(const void *p, int64_t i, bool on, int dt, float none,
                                     Four &v) {
    float t[4] = {none, none, none, none};
    if (on) ld4(p, type_of<DT>(dt), i, t);
    v = {make_float2(t[0], t[1]), make_float2(t[2], t[3])};
}

template <int DT>
__device__ __forceinline__ void put4(void *p, int64_t i, bool on, int dt, const Four &v) {
    const float t[4] = {v.a.x, v.a.y, v.b.x, v.b.y};
    if (on) st4(p, type_of<DT>(dt), i, t);
}

// ------------------------------------------------------------ the ring of rows

// Where a walking block keeps things in shared memory (bytes).  Every row and
// vector is `pad` columns long, the block's threads times their columns; what
// lies past d is zero, so inner loops need no test of the column.
struct JoinSmem {
    int pad;
    int y, h, dh, dx, gate, row;  // places in a ring slot; a slot's size
    int stages;                   // ring depth: 2, 1, or 0 (rows are read from global memory)
    int zero;                     // after the ring: a row of zeros for absent tensors
    int chan;                     // a channel gate
    int w_post, w_pre;            // gains (1 for absent ones), with a ring
    int total;
};

// A row of a tensor into its place in the ring: 16 bytes per thread and copy, so
// what a thread reads later has been copied by others (half the copies of 8 bytes
// each of its own columns; the copies' issue was what bounded the gradients).
template <int V, int DT>
__device__ __forceinline__ void fetch_row(uint32_t slot, const void *p, int dt, int64_t row, int d) {
    const int t = type_of<DT>(dt);
    const char *src = reinterpret_cast<const char *>(p) + row * esize(t);
    const int n16 = d * esize(t) / 16;
#pragma unroll
    for (int v = 0; v < (DT == kAny || DT == RVQ_F32 ? V : (V + 1) / 2); ++v) {
        const int i = v * blockDim.x + threadIdx.x;
        if (i < n16) cp_async16(slot + i * 16, src + i * 16);
    }
}

// four values of a row: in the ring (or the row of zeros), or, for kAny
// instances without a ring, in global memory
template <int DT>
__device__ __forceinline__ void row4(int stages, uint32_t at, const void *p, int64_t row, int i, int d,
                                     int dt, Four &v) {
    if (DT == kAny && stages == 0)
        ldg4<DT>(p, row + i, p != nullptr && i < d, dt, 0.f, v);
    else
        lds4<DT>(at, i, dt, v);
}

// four gains: in shared memory, or (no ring) in global memory
template <int DT>
__device__ __forceinline__ void gain4(int stages, uint32_t at, const void *p, int i, int d, int dt,
                                      Four &v) {
    if (DT == kAny && stages == 0)
        ldg4<DT>(p, i, p != nullptr && i < d, dt, 1.f, v);
    else
        lds4<DT>(at, i, dt, v);
}

// Zeros past the rows' ends (and the row of zeros), gains, a channel gate; none of
// it is written by the copies of rows, which are in flight already.
__device__ __forceinline__ void fill_smem(uint8_t *smem, const JoinJob &j, const JoinSmem &L,
                                          bool bwd) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const auto pad = [&](int at, int dt) {
        const int e = esize(dt), n16 = (L.pad - j.d) * e / 16;  // d and pad are multiples of 8
        for (int i = threadIdx.x; i < n16; i += blockDim.x)
            reinterpret_cast<uint4 *>(smem + at + j.d * e)[i] = zero;
    };
    if (L.pad > j.d)
        for (int s = 0; s < L.stages; ++s) {
            const int slot = s * L.row;
            pad(slot + L.y, j.ydt);
            if (j.h) pad(slot + L.h, j.hdt);
            if (bwd && j.dh_out) pad(slot + L.dh, j.hdt);
            if (bwd && j.dxn) pad(slot + L.dx, j.xdt);
            if (j.gate_kind == MOE_GATE_FULL) pad(slot + L.gate, j.gdt);
        }
    for (int i = threadIdx.x; i < (L.chan - L.zero) / 16; i += blockDim.x)
        reinterpret_cast<uint4 *>(smem + L.zero)[i] = zero;
    const uint32_t one = j.wdt == RVQ_F32 ? 0x3F800000u : j.wdt == RVQ_BF16 ? 0x3F803F80u : 0x3C003C00u;
    const auto gain = [&](int at, const void *src) {
        if (L.stages == 0) return;
        pad(at, j.wdt);
        const int n16 = j.d * esize(j.wdt) / 16;
        for (int i = threadIdx.x; i < n16; i += blockDim.x)
            reinterpret_cast<uint4 *>(smem + at)[i] =
                src ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(one, one, one, one);
    };
    gain(L.w_post, j.w_post);
    gain(L.w_pre, j.w_pre);
    if (j.gate_kind == MOE_GATE_CHANNEL) {
        pad(L.chan, RVQ_F32);
        for (int i = threadIdx.x * 4; i < j.d; i += blockDim.x * 4) {
            float g[4];
            ld4(j.gate, j.gdt, i, g);
            *reinterpret_cast<float4 *>(smem + L.chan + i * 4) = make_float4(g[0], g[1], g[2], g[3]);
        }
    }
    __syncthreads();
}

// Types of an instance: h (and h_out, dh, dh_out), y (and dy), xn (and dxn),
// gains, and a full gate.  GATE 0: one value per row, 1: per channel, 2: full.
template <int V_, int H_, int Y_, int X_, int W_, int G_, int GATE_>
struct JoinTypes {
    static constexpr int V = V_, H = H_, Y = Y_, X = X_, W = W_, G = G_, GATE = GATE_;
};

// Blocks per SM of the gradients' kernel, at most: the partial sums to add grow
// with the blocks, so only as many as give an SM 512 threads.
inline int join_bwd_blocks(int d) {
    const int b = 512 / (((d / 4 + 3) / 4 + 31) / 32 * 32);
    return b < 4 ? 4 : b;
}
// Whether a thread of the gradients' kernel takes two groups of columns instead of
// four, for twice the warps: where the rows' bytes leave an SM few blocks, or a block
// few warps, or there is a row per SM at most (forward and gradients, four and two:
// fp32 2000 x 2048 39.5 and 31.8 us, 1500 x 4096 57.3 and 49.2; bf16 3000 x 1000 28.6
// and 27.0, 100 x 2048 11.0 and 10.1, but 4099 x 2048 40.0 and 42.2).  Past 4096
// columns the registers of so many threads do not suffice.
inline bool join_bwd_narrow(const JoinJob &j) {
    return j.d <= 4096 && (j.hdt == RVQ_F32 || j.d <= 1024 || j.n <= num_sms());
}
constexpr int kSmemMax = 225 << 10;  // of a block, beside its static part

inline int join_threads(int d, int group, int v) {
    const int t = (d / group + v - 1) / v;
    return (t + 31) / 32 * 32;
}

inline JoinSmem join_layout(const JoinJob &j, bool bwd, int st, int v) {
    JoinSmem L = {};
    L.pad = join_threads(j.d, 4, v) * v * 4;
    const auto row = [&](const void *p, int dt) { return p ? L.pad * (dt == RVQ_F32 ? 4 : 2) : 0; };
    int at = 0;
    L.y = at;
    at += row(j.y, j.ydt);
    L.h = at;
    at += row(j.h, j.hdt);
    L.dh = at;
    at += bwd ? row(j.dh_out, j.hdt) : 0;
    L.dx = at;
    at += bwd ? row(j.dxn, j.xdt) : 0;
    L.gate = at;
    at += j.gate_kind == MOE_GATE_FULL ? row(j.gate, j.gdt) : 0;
    L.row = at;
    L.stages = st;
    at *= st;
    L.zero = at;
    if (st > 0 && (!j.h || (bwd && (!j.dh_out || !j.dxn)))) at += L.pad * 4;
    L.chan = at;
    at += j.gate_kind == MOE_GATE_CHANNEL ? L.pad * 4 : 0;
    if (st > 0) {
        L.w_post = at;
        at += row(&L, j.wdt);
        L.w_pre = at;
        at += row(&L, j.wdt);
    }
    L.total = at;
    return L;
}

// Two rows, one (then a block's copies and its work take turns), or (rows of more
// than 8192 fp32 columns) none.  A third row cost more than it hid, in blocks per
// SM and in the wait for the first rows (gradients of 2048 x 7168 68 us with
// three, 60 us with two).
inline JoinSmem join_ring(const JoinJob &j, bool bwd, int v) {
    for (int st = 2; st > 0; --st) {
        const JoinSmem L = join_layout(j, bwd, st, v);
        if (L.total <= kSmemMax) return L;
    }
    return join_layout(j, bwd, 0, v);
}

// Walking blocks of kernel K: as many as an SM holds at once, up to `most`.
template <auto K>
 rvq_status launch_walk(JoinJob &j, const JoinSmem &L, int threads, int most, cudaStream_t stream) {
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax));
        attr_done[dev] = 1;
    }
    int per = 0;
    RVQ_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, K, threads, (size_t)L.total));
    if (per > most) per = most;
    if (per < 1) per = 1;
    const int blocks = per * num_sms();
    j.slots = j.n < blocks ? j.n : blocks;
    RVQ_CUDA(launch_after(K, (unsigned)j.slots, (unsigned)threads, (size_t)L.total, stream, j, L));
    return RVQ_OK;
}

// Whether a typed instance serves a job: rows of up to 8192 columns (they fit the
// ring), every 16-bit tensor of type s16, an fp32 xn beside an fp32 h only, and a
// full gate of h's type.
inline bool join_typed(const JoinJob &j, const JoinSmem &L, int s16) {
    const auto fits = [&](int dt) { return dt == RVQ_F32 || dt == s16; };
    return j.d <= 8192 && L.stages > 0 && fits(j.hdt) && fits(j.ydt) && fits(j.xdt) &&
           fits(j.wdt) && (j.xdt != RVQ_F32 || j.hdt == RVQ_F32) &&
           (j.gate_kind != MOE_GATE_FULL || j.gdt == j.hdt);
}

// Calls f(JoinTypes<...>()) for the typed instance of a job.
template <int S16, class F>
rvq_status with_types(const JoinJob &j, F &&f) {
    using C0 = std::integral_constant<int, S16>;
    using C1 = std::integral_constant<int, (int)RVQ_F32>;
    const auto gate = [&](auto H, auto Y, auto X, auto W) {
        if (j.gate_kind == MOE_GATE_FULL)
            return f(JoinTypes<4, H.value, Y.value, X.value, W.value, H.value, 2>());
        if (j.gate_kind == MOE_GATE_CHANNEL)
            return f(JoinTypes<4, H.value, Y.value, X.value, W.value, RVQ_F32, 1>());
        return f(JoinTypes<4, H.value, Y.value, X.value, W.value, RVQ_F32, 0>());
    };
    const auto pick_w = [&](auto H, auto Y, auto X) {
        return j.wdt == RVQ_F32 ? gate(H, Y, X, C1()) : gate(H, Y, X, C0());
    };
    const auto pick_x = [&](auto H, auto Y) {
        if constexpr (H.value == (int)RVQ_F32)
            if (j.xdt == RVQ_F32) return pick_w(H, Y, C1());
        return pick_w(H, Y, C0());
    };
    const auto pick_y = [&](auto H) {
        return j.ydt == RVQ_F32 ? pick_x(H, C1()) : pick_x(H, C0());
    };
    return j.hdt == RVQ_F32 ? pick_y(C1()) : pick_y(C0());
}

constexpr int kAnyV = 8;

template <class F>
rvq_status with_any_types(const JoinJob &j, F &&f) {
    if (j.gate_kind == MOE_GATE_FULL)
        return f(JoinTypes<kAnyV, kAny, kAny, kAny, kAny, kAny, 2>());
    if (j.gate_kind == MOE_GATE_CHANNEL)
        return f(JoinTypes<kAnyV, kAny, kAny, kAny, kAny, kAny, 1>());
    return f(JoinTypes<kAnyV, kAny, kAny, kAny, kAny, kAny, 0>());
}

// the walking kernels by 16-bit type (one translation unit each)
rvq_status join_walk_bf16(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);
rvq_status join_walk_f16(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);
rvq_status join_walk_any(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);

inline rvq_status join_walk(JoinJob &j, bool bwd, cudaStream_t stream) {
    // types of absent tensors do not matter: take those of the others
    if (!(j.w_post || j.w_pre || j.dw_post || j.dw_pre)) j.wdt = RVQ_F32;
    if (!(bwd ? j.dxn : j.xn)) j.xdt = j.hdt;
    const JoinSmem L = join_ring(j, bwd, 4);
    if (join_typed(j, L, RVQ_BF16)) return join_walk_bf16(j, L, bwd, stream);
    if (join_typed(j, L, RVQ_F16)) return join_walk_f16(j, L, bwd, stream);
    return join_walk_any(j, join_ring(j, bwd, kAnyV), bwd, stream);
}

}  // namespace rvq
