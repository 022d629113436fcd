// Shared parts of moe_norm_join (norm_join.cu) and its gradients
// (norm_join_bwd.cu): sums over a block, a ring of rows in shared memory, and
// the launch of blocks that walk over the rows.
//
// A walking block's thread owns the same columns of every row: groups of four,
// a block's width apart, so that a warp's accesses are contiguous for every
// type.  It copies them ahead into the ring (cp.async, one or two rows in flight
// while one is worked on) and reads only what it copied itself: the ring needs
// no barrier.  Inner loops have no branches: a type is a template parameter
// (16-bit formats differ by a select), an absent tensor or column is a
// predicated load with a neutral value.  With a branch per load (types chosen at
// run time) every load's latency was exposed: 65 us against 34 us for 2048 rows
// of 7168 (fp32 h and y, bf16 xn).
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
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------- groups of four values
// DT: an rvq_dtype, or kAny (the type is looked up in dt).
constexpr int kAny = -1;

template <int DT>
__device__ __forceinline__ int type_of(int dt) {
    return DT == kAny ? dt : DT;
}

__device__ __forceinline__ int esize(int dt) { return dt == RVQ_F32 ? 4 : 2; }

__device__ __forceinline__ void widen4(uint2 r, int dt, float (&v)[4]) {
    unpack16(dt, r.x, v[0], v[1]);
    unpack16(dt, r.y, v[2], v[3]);
}

// four values at element i of a row in shared memory (byte address `at`)
template <int DT>
__device__ __forceinline__ void lds4(uint32_t at, int i, int dt, float (&v)[4]) {
    const int t = type_of<DT>(dt);
    if (t == RVQ_F32) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
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
                                     float (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = none;
    if (on) ld4(p, type_of<DT>(dt), i, v);
}

template <int DT>
__device__ __forceinline__ void put4(void *p, int64_t i, bool on, int dt, const float (&v)[4]) {
    if (on) st4(p, type_of<DT>(dt), i, v);
}

// ------------------------------------------------------------ the ring of rows

// Where a walking block keeps things in shared memory (bytes).  Every row and
// vector is `pad` columns long, the block's threads times their columns; what
// lies past d is zero, so inner loops need no test of the column.
struct JoinSmem {
    int pad;
    int y, h, dh, dx, gate, row;  // places in a ring slot; a slot's size
    int stages;                   // ring depth (0: rows are read from global memory)
    int zero;                     // after the ring: a row of zeros for absent tensors
    int chan;                     // a channel gate
    int w_post, w_pre;            // gains (1 for absent ones); -1: read from global memory
    int total;
};

template <int V, int DT>
__device__ __forceinline__ void fetch_row(uint32_t slot, const void *p, int dt, int64_t row, int d) {
    const bool f32 = type_of<DT>(dt) == RVQ_F32;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * blockDim.x + threadIdx.x) * 4;
        if (c < d) {
            if (f32)
                cp_async16(slot + c * 4, reinterpret_cast<const float *>(p) + row + c);
            else
                cp_async8(slot + c * 2, reinterpret_cast<const uint16_t *>(p) + row + c);
        }
    }
}

// the oldest row's copies are done, with a ring of `stages` rows
__device__ __forceinline__ void wait_row(int stages) {
    if (stages == 3)
        cp_wait<2>();
    else
        cp_wait<1>();
}

// four values of a row: in the ring (or the row of zeros), or, for kAny
// instances without a ring, in global memory
template <int DT>
__device__ __forceinline__ void row4(int stages, uint32_t at, const void *p, int64_t row, int i, int d,
                                     int dt, float (&v)[4]) {
    if (DT == kAny && stages == 0)
        ldg4<DT>(p, row + i, p != nullptr && i < d, dt, 0.f, v);
    else
        lds4<DT>(at, i, dt, v);
}

// four gains: in shared memory (SHARED 1), in global memory (0), or as `at` says
template <int DT, int SHARED>
__device__ __forceinline__ void gain4(int at, uint32_t base, const void *p, int i, int d, int dt,
                                      float (&v)[4]) {
    if (SHARED == 1 || (SHARED == kAny && at >= 0))
        lds4<DT>(base + at, i, dt, v);
    else
        ldg4<DT>(p, i, p != nullptr && i < d, dt, 1.f, v);
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
        if (at < 0) return;
        pad(at, j.wdt);
        const int n16 = j.d * esize(j.wdt) / 16;
        for (int i = threadIdx.x; i < n16; i += blockDim.x)
            reinterpret_cast<uint4 *>(smem + at)[i] =
                src ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(one, one, one, one);
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
// SHARED: gains in shared memory (1), global (0), or as the layout says (kAny).
template <int V_, int H_, int Y_, int X_, int W_, int G_, int GATE_, int SHARED_>
struct JoinTypes {
    static constexpr int V = V_, H = H_, Y = Y_, X = X_, W = W_, G = G_, GATE = GATE_,
                         SHARED = SHARED_;
};

constexpr int kBwdBlocksPerSm = 4;   // the partial sums to add grow with the blocks
constexpr int kSmemMax = 225 << 10;  // of a block, beside its static part

inline int join_threads(int d, int group, int v) {
    const int t = (d / group + v - 1) / v;
    return (t + 31) / 32 * 32;
}

inline JoinSmem join_layout(const JoinJob &j, bool bwd, int st, int v, bool gains) {
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
    L.w_post = L.w_pre = -1;
    if (gains) {
        L.w_post = at;
        at += row(&L, j.wdt);
        L.w_pre = at;
        at += row(&L, j.wdt);
    }
    L.total = at;
    return L;
}

// Three rows and the gains, two rows and the gains, two rows alone, or (rows too
// long for shared memory) none.
inline JoinSmem join_ring(const JoinJob &j, bool bwd, int v) {
    for (int i = 0; i < 3; ++i) {
        const JoinSmem L = join_layout(j, bwd, i == 0 ? 3 : 2, v, i < 2);
        if (L.total <= kSmemMax) return L;
    }
    return join_layout(j, bwd, 0, v, false);
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

// Whether a typed instance serves a job: rows of up to 8192 columns that fit the
// ring, a 16-bit xn, every 16-bit tensor of its type, a full gate of h's type,
// and, for gains left in global memory, fp32 h and gains (shorter types fit).
inline bool join_typed(const JoinJob &j, const JoinSmem &L) {
    const int s16 = j.xdt;
    const auto fits = [&](int dt) { return dt == RVQ_F32 || dt == s16; };
    return s16 != RVQ_F32 && j.d <= 8192 && L.stages > 0 && fits(j.hdt) && fits(j.ydt) &&
           fits(j.wdt) && (j.gate_kind != MOE_GATE_FULL || j.gdt == j.hdt) &&
           (L.w_pre >= 0 || (j.hdt == RVQ_F32 && j.wdt == RVQ_F32));
}

// Calls f(JoinTypes<...>()) for the typed instance of a job.
template <int S16, class F>
rvq_status with_types(const JoinJob &j, const JoinSmem &L, F &&f) {
    using C0 = std::integral_constant<int, S16>;
    using C1 = std::integral_constant<int, (int)RVQ_F32>;
    const auto gate = [&](auto H, auto Y, auto W, auto G) {
        if (j.gate_kind == MOE_GATE_FULL)
            return f(JoinTypes<4, H.value, Y.value, S16, W.value, H.value, 2, G.value>());
        if (j.gate_kind == MOE_GATE_CHANNEL)
            return f(JoinTypes<4, H.value, Y.value, S16, W.value, RVQ_F32, 1, G.value>());
        return f(JoinTypes<4, H.value, Y.value, S16, W.value, RVQ_F32, 0, G.value>());
    };
    using Shared = std::integral_constant<int, 1>;
    using Global = std::integral_constant<int, 0>;
    const auto pick_w = [&](auto H, auto Y) {
        if (j.wdt != RVQ_F32) return gate(H, Y, C0(), Shared());
        if constexpr (H.value == (int)RVQ_F32)
            if (L.w_pre < 0) return gate(H, Y, C1(), Global());
        return gate(H, Y, C1(), Shared());
    };
    const auto pick_y = [&](auto H) {
        return j.ydt == RVQ_F32 ? pick_w(H, C1()) : pick_w(H, C0());
    };
    return j.hdt == RVQ_F32 ? pick_y(C1()) : pick_y(C0());
}

constexpr int kAnyV = 8;

template <class F>
rvq_status with_any_types(const JoinJob &j, F &&f) {
    if (j.gate_kind == MOE_GATE_FULL)
        return f(JoinTypes<kAnyV, kAny, kAny, kAny, kAny, kAny, 2, kAny>());
    if (j.gate_kind == MOE_GATE_CHANNEL)
        return f(JoinTypes<kAnyV, kAny, kAny, kAny, kAny, kAny, 1, kAny>());
    return f(JoinTypes<kAnyV, kAny, kAny, kAny, kAny, kAny, 0, kAny>());
}

// the walking kernels by 16-bit type (one translation unit each)
rvq_status join_walk_bf16(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);
rvq_status join_walk_f16(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);
rvq_status join_walk_any(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);

inline rvq_status join_walk(JoinJob &j, bool bwd, cudaStream_t stream) {
    // types of absent tensors do not matter: take those of the others
    if (!(j.w_post || j.w_pre || j.dw_post || j.dw_pre)) j.wdt = RVQ_F32;
    if (!(bwd ? j.dxn : j.xn)) j.xdt = j.hdt != RVQ_F32 ? j.hdt : j.ydt != RVQ_F32 ? j.ydt : RVQ_BF16;
    const JoinSmem L = join_ring(j, bwd, 4);
    if (!join_typed(j, L)) return join_walk_any(j, join_ring(j, bwd, kAnyV), bwd, stream);
    return j.xdt == RVQ_BF16 ? join_walk_bf16(j, L, bwd, stream) : join_walk_f16(j, L, bwd, stream);
}

}  // namespace rvq
