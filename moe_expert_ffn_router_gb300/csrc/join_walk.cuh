// The kernels of moe_norm_join and its gradients whose blocks walk over the rows,
// for every instance of their types; join_walk_*.cu compile them.
#pragma once

#include "join_common.cuh"

namespace rvq {
namespace {

template <class T>
__global__ void __launch_bounds__(512) join_ring_kernel(const JoinJob j, const JoinSmem L) {
    constexpr int V = T::V;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[4][32];
    const bool has_h = j.h != nullptr;
    const float inv_d = 1.f / (float)j.d, alpha = has_h ? j.alpha : 0.f;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem);
    const auto fetch = [&](int t, int s) {
        if (t < j.n) {
            const uint32_t slot = ring + s * L.row;
            const int64_t row = (int64_t)t * j.d;
            fetch_row<V, T::Y>(slot + L.y, j.y, j.ydt, row, j.d);
            if (has_h) fetch_row<V, T::H>(slot + L.h, j.h, j.hdt, row, j.d);
            if (T::GATE == 2) fetch_row<V, T::G>(slot + L.gate, j.gate, j.gdt, row, j.d);
        }
        cp_commit();
    };
    const int G = gridDim.x, S = L.stages;
    int t = blockIdx.x;
    dependency_wait();
    if (S) fetch(t, 0);
    fill_smem(smem, j, L, false);
    float g_next = 1.f;
    if (j.gate_kind == MOE_GATE_SCALAR) g_next = ld_elem(j.gate, j.gdt, 0);
    if (j.gate_kind == MOE_GATE_TOKEN && t < j.n) g_next = ld_elem(j.gate, j.gdt, t);
    int slot_i = 0, flip = 0;
    for (; t < j.n; t += G, flip ^= 2) {
        if (S == 1 && t >= G) {  // the one row's place is free
            __syncthreads();
            fetch(t, 0);
        }
        if (S) {
            // this row has arrived everywhere, and the row before is read
            cp_wait<0>();
            __syncthreads();
        }
        if (S == 2) fetch(t + G, slot_i ^ 1);
        const float gt = g_next;
        if (j.gate_kind == MOE_GATE_TOKEN && t + G < j.n) g_next = ld_elem(j.gate, j.gdt, t + G);
        const uint32_t slot = ring + slot_i * L.row;
        if (S == 2) slot_i ^= 1;
        const int64_t row = (int64_t)t * j.d;
        const uint32_t at_h = has_h ? slot + L.h : ring + L.zero;
        Four y[V], h[V];
        float s1[1], s2[1];
        Four q = four(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            row4<T::Y>(S, slot + L.y, j.y, row, c, j.d, j.ydt, y[v]);
            row4<T::H>(S, at_h, j.h, row, c, j.d, j.hdt, h[v]);
            q = fma4(y[v], y[v], q);
        }
        float r1 = 1.f;
        if (j.post_norm) {
            s1[0] = sum4(q);
            block_sum(s1, red[flip]);
            r1 = 1.f / sqrtf(s1[0] * inv_d + j.eps);
        }
        q = four(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            Four g = four(gt), w;
            if (T::GATE == 1) lds4<RVQ_F32>(ring + L.chan, c, RVQ_F32, g);
            if (T::GATE == 2) row4<T::G>(S, slot + L.gate, j.gate, row, c, j.d, j.gdt, g);
            gain4<T::W>(S, ring + L.w_post, j.w_post, c, j.d, j.wdt, w);
            h[v] = fma4(g, y[v] * four(r1) * w, four(alpha) * h[v]);
            q = fma4(h[v], h[v], q);
            put4<T::H>(j.h_out, row + c, j.h_out != nullptr && c < j.d, j.hdt, h[v]);
        }
        s2[0] = sum4(q);
        block_sum(s2, red[flip + 1]);
        const float r2 = 1.f / sqrtf(s2[0] * inv_d + j.eps);
        if (j.rstd && threadIdx.x == 0) {
            j.rstd[t] = r1;
            j.rstd[(int64_t)j.n + t] = r2;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            Four w;
            gain4<T::W>(S, ring + L.w_pre, j.w_pre, c, j.d, j.wdt, w);
            put4<T::X>(j.xn, row + c, j.xn != nullptr && c < j.d, j.xdt, h[v] * four(r2) * w);
        }
    }
    cp_wait<0>();
}

// Gradients.  With q = dxn w_pre, P = dh_out + r2 q and c = r2^3 / d a row has
// e = P - c S h_out, S = sum q h_out; the norm of y needs sum e gate z = sum P
// gate z - c S sum h_out gate z, so one reduction of three sums serves the row.
// The second pass over the row reads the ring again.  The sums over rows
// (dw_post, dw_pre, dgate per channel) stay in registers while a block walks:
// one fp32 partial per block, column and sum.
template <class T>
__global__ void __launch_bounds__(512) join_bwd_kernel(const JoinJob j, const JoinSmem L) {
    constexpr int V = T::V;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][96];
    const bool has_h = j.h != nullptr, has_dh = j.dh_out != nullptr, has_dx = j.dxn != nullptr;
    const float inv_d = 1.f / (float)j.d, alpha = has_h ? j.alpha : 0.f;
    constexpr int SUMS = T::GATE == 1 ? 3 : 2;  // dw_post, dw_pre, dgate per channel
    Four acc[SUMS][V];
    float gate_sum = 0.f;
#pragma unroll
    for (int k = 0; k < SUMS; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[k][v] = four(0.f);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem);
    const auto fetch = [&](int t, int s) {
        if (t < j.n) {
            const uint32_t slot = ring + s * L.row;
            const int64_t row = (int64_t)t * j.d;
            fetch_row<V, T::Y>(slot + L.y, j.y, j.ydt, row, j.d);
            if (has_h) fetch_row<V, T::H>(slot + L.h, j.h, j.hdt, row, j.d);
            if (has_dh) fetch_row<V, T::H>(slot + L.dh, j.dh_out, j.hdt, row, j.d);
            if (has_dx) fetch_row<V, T::X>(slot + L.dx, j.dxn, j.xdt, row, j.d);
            if (T::GATE == 2) fetch_row<V, T::G>(slot + L.gate, j.gate, j.gdt, row, j.d);
        }
        cp_commit();
    };
    const int G = gridDim.x, S = L.stages;
    int t = blockIdx.x;
    dependency_wait();
    if (S) fetch(t, 0);
    fill_smem(smem, j, L, true);
    float r1n = 1.f, r2n = 1.f, gn = 1.f;
    const auto scalars = [&](int u) {
        if (u >= j.n) return;
        if (j.post_norm) r1n = j.rstd[u];
        r2n = j.rstd[(int64_t)j.n + u];
        if (j.gate_kind == MOE_GATE_TOKEN) gn = ld_elem(j.gate, j.gdt, u);
    };
    if (j.gate_kind == MOE_GATE_SCALAR) gn = ld_elem(j.gate, j.gdt, 0);
    scalars(t);
    int slot_i = 0, flip = 0;
    for (; t < j.n; t += G, flip ^= 1) {
        if (S == 1 && t >= G) {  // the one row's place is free
            __syncthreads();
            fetch(t, 0);
        }
        if (S) {
            // this row has arrived everywhere, and the row before is read
            cp_wait<0>();
            __syncthreads();
        }
        if (S == 2) fetch(t + G, slot_i ^ 1);
        const float r1 = r1n, r2 = r2n, gt = gn;
        scalars(t + G);
        const uint32_t slot = ring + slot_i * L.row;
        if (S == 2) slot_i ^= 1;
        const int64_t row = (int64_t)t * j.d;
        const uint32_t at_h = has_h ? slot + L.h : ring + L.zero;
        const uint32_t at_dh = has_dh ? slot + L.dh : ring + L.zero;
        const uint32_t at_dx = has_dx ? slot + L.dx : ring + L.zero;
        const Four R1 = four(r1), R2 = four(r2), AL = four(alpha);
        // a group's y r1, z, h_out, q, P, dxn, gate, w_post (zeros past the row)
        struct Group {
            Four yr, z, ho, q, P, dx, g, w;
        };
        const auto group = [&](int c) {
            Group u;
            Four y, h, dh, wp;
            row4<T::Y>(S, slot + L.y, j.y, row, c, j.d, j.ydt, y);
            row4<T::H>(S, at_h, j.h, row, c, j.d, j.hdt, h);
            row4<T::H>(S, at_dh, j.dh_out, row, c, j.d, j.hdt, dh);
            row4<T::X>(S, at_dx, j.dxn, row, c, j.d, j.xdt, u.dx);
            u.g = four(gt);
            if (T::GATE == 1) lds4<RVQ_F32>(ring + L.chan, c, RVQ_F32, u.g);
            if (T::GATE == 2) row4<T::G>(S, slot + L.gate, j.gate, row, c, j.d, j.gdt, u.g);
            gain4<T::W>(S, ring + L.w_post, j.w_post, c, j.d, j.wdt, u.w);
            gain4<T::W>(S, ring + L.w_pre, j.w_pre, c, j.d, j.wdt, wp);
            u.yr = y * R1;
            u.z = u.yr * u.w;
            u.ho = fma4(u.g, u.z, AL * h);
            u.q = u.dx * wp;
            u.P = fma4(R2, u.q, dh);
            return u;
        };
        Four s0 = four(0.f), sA = four(0.f), sB = four(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Group u = group((v * blockDim.x + threadIdx.x) * 4);
            const Four gz = T::GATE == 0 ? u.z : u.g * u.z;
            s0 = fma4(u.q, u.ho, s0);
            sA = fma4(u.P, gz, sA);
            sB = fma4(u.ho, gz, sB);
        }
        float s[3] = {sum4(s0), sum4(sA), sum4(sB)};
        block_sum(s, red[flip]);
        // r2 s[0] is of the order of d: in this order no factor leaves fp32 where c S
        // does not (r2^3 alone does for rows of 1e-13 or 1e13)
        const float cS = r2 * (r2 * (r2 * s[0] * inv_d));
        const float ez = s[1] - cS * s[2];  // sum e z (one gate per row) or sum e gate z
        if (T::GATE == 0 && j.dgate && threadIdx.x == 0) {
            if (j.gate_kind == MOE_GATE_TOKEN)
                st_elem(j.dgate, j.gdt, t, ez);
            else
                gate_sum += ez;
        }
        // dy = r1 (dz w_post - y r1 mean(...)): mean = (sum e gate z) / d
        const float cy = j.post_norm ? inv_d * (T::GATE == 0 ? gt * ez : ez) : 0.f;
        const Four NS = four(-cS), NY = four(-cy);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            const Group u = group(c);
            const Four e = fma4(NS, u.ho, u.P);
            put4<T::H>(j.dh, row + c, j.dh != nullptr && c < j.d, j.hdt, AL * e);
            const Four dz = u.g * e;
            put4<T::Y>(j.dy, row + c, j.dy != nullptr && c < j.d, j.ydt,
                       R1 * fma4(NY, u.yr, dz * u.w));
            acc[0][v] = fma4(dz, u.yr, acc[0][v]);
            acc[1][v] = fma4(u.dx, u.ho * R2, acc[1][v]);
            if (T::GATE == 1) acc[SUMS - 1][v] = fma4(e, u.z, acc[SUMS - 1][v]);
            if (T::GATE == 2)
                put4<T::G>(j.dgate, row + c, j.dgate != nullptr && c < j.d, j.gdt, e * u.z);
        }
    }
    cp_wait<0>();
    float *part = j.part + (int64_t)blockIdx.x * 3 * j.d;
    const bool want[3] = {j.dw_post != nullptr, j.dw_pre != nullptr,
                          T::GATE == 1 && j.dgate != nullptr};
#pragma unroll
    for (int k = 0; k < SUMS; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            put4<RVQ_F32>(part, (int64_t)k * j.d + c, want[k] && c < j.d, RVQ_F32, acc[k][v]);
        }
    if (threadIdx.x == 0) j.part[(int64_t)j.slots * 3 * j.d + blockIdx.x] = gate_sum;
}

constexpr int kFwdBlocksPerSm = 16;

template <class T>
rvq_status walk(JoinJob &j, const JoinSmem &L, bool bwd, cudaStream_t stream) {
    const int threads = join_threads(j.d, 4, T::V);
    if constexpr (T::V == 4) {
        if (bwd && join_bwd_narrow(j)) {
            using U = JoinTypes<2, T::H, T::Y, T::X, T::W, T::G, T::GATE>;
            return launch_walk<join_bwd_kernel<U>>(j, join_ring(j, true, 2), join_threads(j.d, 4, 2),
                                                   join_bwd_blocks(j.d), stream);
        }
    }
    if (bwd) return launch_walk<join_bwd_kernel<T>>(j, L, threads, join_bwd_blocks(j.d), stream);
    return launch_walk<join_ring_kernel<T>>(j, L, threads, kFwdBlocksPerSm, stream);
}

}  // namespace
}  // namespace rvq
