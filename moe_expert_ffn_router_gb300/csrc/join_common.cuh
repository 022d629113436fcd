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

// four values at element i of a row in shared memory (byte address `at`); zeros
// when off
template <int DT>
__device__ __forceinline__ void lds4(uint32_t at, int i, bool on, int dt, float (&v)[4]) {
    const int t = type_of<DT>(dt);
    if (t == RVQ_F32) {
        asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %5, 0;\nmov.f32 %0, 0f00000000;\nmov.f32 %1, "
            "0f00000000;\nmov.f32 %2, 0f00000000;\nmov.f32 %3, 0f00000000;\n@p ld.shared.v4.f32 "
            "{%0, %1, %2, %3}, [%4];\n}\n"
            : "=&f"(v[0]), "=&f"(v[1]), "=&f"(v[2]), "=&f"(v[3])
            : "r"(at + i * 4), "r"((int)on)
            : "memory");
    } else {
        uint2 r;
        asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %3, 0;\nmov.b32 %0, 0;\nmov.b32 %1, 0;\n@p "
            "ld.shared.v2.b32 {%0, %1}, [%2];\n}\n"
            : "=&r"(r.x), "=&r"(r.y)
            : "r"(at + i * 2), "r"((int)on)
            : "memory");
        widen4(r, t, v);
    }
}

// four values in global memory; zeros when off
template <int DT>
__device__ __forceinline__ void ldg4(const void *p, int64_t i, bool on, int dt, float (&v)[4]) {
    const int t = type_of<DT>(dt);
    v[0] = v[1] = v[2] = v[3] = 0.f;
    if (on) ld4(p, t, i, v);
}

// a gain: 1 without one
struct Gain {
    const void *p;
    uint32_t at;   // shared memory
    bool have, shared;
};

template <int DT>
__device__ __forceinline__ void gain4(const Gain &g, int i, bool on, int dt, float (&v)[4]) {
    const int t = type_of<DT>(dt);
    if (t == RVQ_F32) {
        float4 r = make_float4(1.f, 1.f, 1.f, 1.f);
        if (g.have && on && !g.shared)
            r = __ldg(reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(g.p) + i));
        if (g.have && on && g.shared)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
                         : "r"(g.at + i * 4)
                         : "memory");
        v[0] = r.x;
        v[1] = r.y;
        v[2] = r.z;
        v[3] = r.w;
    } else {
        const uint32_t one = t == RVQ_BF16 ? 0x3F803F80u : 0x3C003C00u;
        uint2 r = make_uint2(one, one);
        if (g.have && on && !g.shared)
            r = __ldg(reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(g.p) + i));
        if (g.have && on && g.shared)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(r.x), "=r"(r.y)
                         : "r"(g.at + i * 2)
                         : "memory");
        widen4(r, t, v);
    }
}

template <int DT>
__device__ __forceinline__ void put4(void *p, int64_t i, bool on, int dt, const float (&v)[4]) {
    if (on) st4(p, type_of<DT>(dt), i, v);
}

// ------------------------------------------------------------ the ring of rows

// Where a walking block keeps things in shared memory (bytes; rows and vectors
// are multiples of 16 bytes since d % 8 == 0).
struct JoinSmem {
    int y, h, dh, dx, gate, row;  // places in a ring slot; a slot's size
    int stages;                   // ring depth (0: rows are read from global memory)
    int chan;                     // after the ring: a channel gate
    int w_post, w_pre;            // gains; -1: read from global memory
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

// four values of a row: in the ring, or (kAny instances without a ring) global
template <int DT>
__device__ __forceinline__ void row4(int stages, uint32_t at, const void *p, int64_t row, int i,
                                     bool on, int dt, float (&v)[4]) {
    if (DT == kAny && stages == 0)
        ldg4<DT>(p, row + i, on, dt, v);
    else
        lds4<DT>(at, i, on, dt, v);
}

__device__ __forceinline__ Gain keep_gain(uint8_t *smem, int at, const void *src, int dt, int d) {
    Gain g;
    g.p = src;
    g.at = 0;
    g.have = src != nullptr;
    g.shared = at >= 0;
    if (g.have && g.shared) {
        const int n16 = d * esize(dt) / 16;
        for (int i = threadIdx.x; i < n16; i += blockDim.x)
            reinterpret_cast<uint4 *>(smem + at)[i] = reinterpret_cast<const uint4 *>(src)[i];
        g.at = (uint32_t)__cvta_generic_to_shared(smem + at);
    }
    return g;
}

// a channel gate: in shared memory as fp32
__device__ __forceinline__ uint32_t keep_gate(uint8_t *smem, int at, const void *src, int dt,
                                              int d) {
    float *to = reinterpret_cast<float *>(smem + at);
    for (int i = threadIdx.x; i < d; i += blockDim.x) to[i] = ld_elem(src, dt, i);
    return (uint32_t)__cvta_generic_to_shared(to);
}

// Types of an instance: h (and h_out, dh, dh_out), y (and dy), xn (and dxn),
// gains, and a full gate.  GATE 0: one value per row, 1: per channel, 2: full.
template <int V_, int H_, int Y_, int X_, int W_, int G_, int GATE_>
struct JoinTypes {
    static constexpr int V = V_, H = H_, Y = Y_, X = X_, W = W_, G = G_, GATE = GATE_;
};

constexpr int kBwdBlocksPerSm = 4;   // the partial sums to add grow with the blocks
constexpr int kSmemMax = 225 << 10;  // of a block, beside its static part

inline int join_threads(int d, int group, int v) {
    const int t = (d / group + v - 1) / v;
    return (t + 31) / 32 * 32;
}

inline JoinSmem join_layout(const JoinJob &j, bool bwd, int st) {
    const auto size = [&](const void *p, int dt) { return p ? j.d * (dt == RVQ_F32 ? 4 : 2) : 0; };
    JoinSmem L = {};
    int at = 0;
    L.y = at;
    at += size(j.y, j.ydt);
    L.h = at;
    at += size(j.h, j.hdt);
    L.dh = at;
    at += bwd ? size(j.dh_out, j.hdt) : 0;
    L.dx = at;
    at += bwd ? size(j.dxn, j.xdt) : 0;
    L.gate = at;
    at += j.gate_kind == MOE_GATE_FULL ? size(j.gate, j.gdt) : 0;
    L.row = at;
    L.stages = st;
    at *= st;
    L.chan = at;
    at += j.gate_kind == MOE_GATE_CHANNEL ? j.d * 4 : 0;
    int *const place[2] = {&L.w_post, &L.w_pre};
    const int bytes[2] = {size(j.w_post, j.wdt), size(j.w_pre, j.wdt)};
    for (int i = 0; i < 2; ++i) {
        *place[i] = at + bytes[i] <= kSmemMax ? at : -1;
        if (*place[i] >= 0) at += bytes[i];
    }
    L.total = at;
    return L;
}

// Three rows, or two, or (rows too long for shared memory) none.  Gains are kept
// in shared memory where that costs no row.
inline JoinSmem join_ring(const JoinJob &j, bool bwd) {
    for (int st = 3; st > 1; --st) {
        const JoinSmem L = join_layout(j, bwd, st);
        if (L.total <= kSmemMax) return L;
    }
    return join_layout(j, bwd, 0);
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
    K<<<j.slots, threads, (size_t)L.total, stream>>>(j, L);
    RVQ_LAUNCHED("norm_join");
    return RVQ_OK;
}

// Calls f(JoinTypes<...>()) for the instance of a job's types with S16 as its
// 16-bit type: rows of up to 8192 columns that fit the ring, a 16-bit xn, every
// 16-bit tensor of one type, and a full gate of h's type.  Anything else takes
// the instance that looks types up.
inline bool join_typed(const JoinJob &j, const JoinSmem &L) {
    const int s16 = j.xdt;
    const auto fits = [&](const void *p, int dt) { return !p || dt == RVQ_F32 || dt == s16; };
    return s16 != RVQ_F32 && j.d <= 8192 && L.stages > 0 && fits(j.y, j.hdt) && fits(j.y, j.ydt) &&
           (!(j.w_post || j.w_pre || j.dw_post || j.dw_pre) || fits(j.y, j.wdt)) &&
           (j.gate_kind != MOE_GATE_FULL || j.gdt == j.hdt);
}

template <int S16, class F>
rvq_status with_types(const JoinJob &j, F &&f) {
    using C0 = std::integral_constant<int, S16>;
    using C1 = std::integral_constant<int, (int)RVQ_F32>;
    const auto gate = [&](auto H, auto Y, auto W) {
        if (j.gate_kind == MOE_GATE_FULL)
            return f(JoinTypes<4, H.value, Y.value, S16, W.value, H.value, 2>());
        if (j.gate_kind == MOE_GATE_CHANNEL)
            return f(JoinTypes<4, H.value, Y.value, S16, W.value, RVQ_F32, 1>());
        return f(JoinTypes<4, H.value, Y.value, S16, W.value, RVQ_F32, 0>());
    };
    const auto pick_w = [&](auto H, auto Y) {
        return j.wdt == RVQ_F32 ? gate(H, Y, C1()) : gate(H, Y, C0());
    };
    const auto pick_y = [&](auto H) {
        return j.ydt == RVQ_F32 ? pick_w(H, C1()) : pick_w(H, C0());
    };
    return j.hdt == RVQ_F32 ? pick_y(C1()) : pick_y(C0());
}

template <class F>
rvq_status with_any_types(const JoinJob &j, F &&f) {
    if (j.gate_kind == MOE_GATE_FULL) return f(JoinTypes<8, kAny, kAny, kAny, kAny, kAny, 2>());
    if (j.gate_kind == MOE_GATE_CHANNEL)
        return f(JoinTypes<8, kAny, kAny, kAny, kAny, kAny, 1>());
    return f(JoinTypes<8, kAny, kAny, kAny, kAny, kAny, 0>());
}

// the walking kernels by 16-bit type (one translation unit each)
rvq_status join_walk_bf16(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);
rvq_status join_walk_f16(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);
rvq_status join_walk_any(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream);

inline rvq_status join_walk(JoinJob &j, bool bwd, cudaStream_t stream) {
    const JoinSmem L = join_ring(j, bwd);
    if (!join_typed(j, L)) return join_walk_any(j, L, bwd, stream);
    return j.xdt == RVQ_BF16 ? join_walk_bf16(j, L, bwd, stream) : join_walk_f16(j, L, bwd, stream);
}

}  // namespace rvq
