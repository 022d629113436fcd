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
    for (int s = 0; s + 1 < S; ++s) fetch(t + s * G, s);
    fill_smem(smem, j, L, false);
    float g_next = 1.f;
    if (j.gate_kind == MOE_GATE_SCALAR) g_next = ld_elem(j.gate, j.gdt, 0);
    if (j.gate_kind == MOE_GATE_TOKEN && t < j.n) g_next = ld_elem(j.gate, j.gdt, t);
    int slot_i = 0, flip = 0;
    for (; t < j.n; t += G, flip ^= 2) {
        if (S) {
            fetch(t + (S - 1) * G, slot_i == 0 ? S - 1 : slot_i - 1);
            wait_row(S);
        }
        const float gt = g_next;
        if (j.gate_kind == MOE_GATE_TOKEN && t + G < j.n) g_next = ld_elem(j.gate, j.gdt, t + G);
        const uint32_t slot = ring + slot_i * L.row;
        slot_i = slot_i + 1 >= S ? 0 : slot_i + 1;
        const int64_t row = (int64_t)t * j.d;
        const uint32_t at_h = has_h ? slot + L.h : ring + L.zero;
        float y[V][4], h[V][4];
        float s1[1] = {0.f}, s2[1] = {0.f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            row4<T::Y>(S, slot + L.y, j.y, row, c, j.d, j.ydt, y[v]);
            row4<T::H>(S, at_h, j.h, row, c, j.d, j.hdt, h[v]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s1[0] += y[v][e] * y[v][e];
        }
        float r1 = 1.f;
        if (j.post_norm) {
            block_sum(s1, red[flip]);
            r1 = 1.f / sqrtf(s1[0] * inv_d + j.eps);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            float g[4] = {gt, gt, gt, gt}, w[4];
            if (T::GATE == 1) lds4<RVQ_F32>(ring + L.chan, c, RVQ_F32, g);
            if (T::GATE == 2) row4<T::G>(S, slot + L.gate, j.gate, row, c, j.d, j.gdt, g);
            gain4<T::W, T::SHARED>(L.w_post, ring, j.w_post, c, j.d, j.wdt, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[v][e] = alpha * h[v][e] + g[e] * (y[v][e] * r1 * w[e]);
                s2[0] += h[v][e] * h[v][e];
            }
            put4<T::H>(j.h_out, row + c, j.h_out != nullptr && c < j.d, j.hdt, h[v]);
        }
        block_sum(s2, red[flip + 1]);
        const float r2 = 1.f / sqrtf(s2[0] * inv_d + j.eps);
        if (j.rstd && threadIdx.x == 0) {
            j.rstd[t] = r1;
            j.rstd[(int64_t)j.n + t] = r2;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            float w[4];
            gain4<T::W, T::SHARED>(L.w_pre, ring, j.w_pre, c, j.d, j.wdt, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] *= h[v][e] * r2;
            put4<T::X>(j.xn, row + c, j.xn != nullptr && c < j.d, j.xdt, w);
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
    float acc[3][V][4], gate_sum = 0.f;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[k][v][e] = 0.f;
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
    for (int s = 0; s + 1 < S; ++s) fetch(t + s * G, s);
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
        if (S) {
            fetch(t + (S - 1) * G, slot_i == 0 ? S - 1 : slot_i - 1);
            wait_row(S);
        }
        const float r1 = r1n, r2 = r2n, gt = gn;
        scalars(t + G);
        const uint32_t slot = ring + slot_i * L.row;
        slot_i = slot_i + 1 >= S ? 0 : slot_i + 1;
        const int64_t row = (int64_t)t * j.d;
        const uint32_t at_h = has_h ? slot + L.h : ring + L.zero;
        const uint32_t at_dh = has_dh ? slot + L.dh : ring + L.zero;
        const uint32_t at_dx = has_dx ? slot + L.dx : ring + L.zero;
        // a group's y, h_out, P, dxn, q, gate, z, w_post (zeros past the row)
        const auto group = [&](int c, float (&y)[4], float (&ho)[4], float (&P)[4], float (&dx)[4],
                               float (&q)[4], float (&g)[4], float (&z)[4], float (&w)[4]) {
            float wp[4];
            row4<T::Y>(S, slot + L.y, j.y, row, c, j.d, j.ydt, y);
            row4<T::H>(S, at_h, j.h, row, c, j.d, j.hdt, ho);
            row4<T::H>(S, at_dh, j.dh_out, row, c, j.d, j.hdt, P);
            row4<T::X>(S, at_dx, j.dxn, row, c, j.d, j.xdt, dx);
            g[0] = g[1] = g[2] = g[3] = gt;
            if (T::GATE == 1) lds4<RVQ_F32>(ring + L.chan, c, RVQ_F32, g);
            if (T::GATE == 2) row4<T::G>(S, slot + L.gate, j.gate, row, c, j.d, j.gdt, g);
            gain4<T::W, T::SHARED>(L.w_post, ring, j.w_post, c, j.d, j.wdt, w);
            gain4<T::W, T::SHARED>(L.w_pre, ring, j.w_pre, c, j.d, j.wdt, wp);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[e] = y[e] * r1 * w[e];
                ho[e] = alpha * ho[e] + g[e] * z[e];
                q[e] = dx[e] * wp[e];
                P[e] += r2 * q[e];
            }
        };
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            float y[4], ho[4], P[4], dx[4], q[4], g[4], z[4], w[4];
            group(c, y, ho, P, dx, q, g, z, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float gz = T::GATE == 0 ? z[e] : g[e] * z[e];
                s[0] += q[e] * ho[e];
                s[1] += P[e] * gz;
                s[2] += ho[e] * gz;
            }
        }
        block_sum(s, red[flip]);
        const float cS = r2 * r2 * r2 * inv_d * s[0];
        const float ez = s[1] - cS * s[2];  // sum e z (one gate per row) or sum e gate z
        if (T::GATE == 0 && j.dgate && threadIdx.x == 0) {
            if (j.gate_kind == MOE_GATE_TOKEN)
                st_elem(j.dgate, j.gdt, t, ez);
            else
                gate_sum += ez;
        }
        const float cy = j.post_norm ? r1 * r1 * inv_d * (T::GATE == 0 ? gt * ez : ez) : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * blockDim.x + threadIdx.x) * 4;
            float y[4], ho[4], P[4], dx[4], q[4], g[4], z[4], w[4], o[4];
            group(c, y, ho, P, dx, q, g, z, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                P[e] -= cS * ho[e];
                o[e] = alpha * P[e];
            }
            put4<T::H>(j.dh, row + c, j.dh != nullptr && c < j.d, j.hdt, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float dz = g[e] * P[e], ze = P[e] * z[e];
                o[e] = r1 * dz * w[e] - y[e] * cy;
                acc[0][v][e] += dz * y[e] * r1;
                acc[1][v][e] += dx[e] * ho[e] * r2;
                acc[2][v][e] += ze;
                P[e] = ze;
            }
            put4<T::Y>(j.dy, row + c, j.dy != nullptr && c < j.d, j.ydt, o);
            if (T::GATE == 2) put4<T::G>(j.dgate, row + c, j.dgate != nullptr && c < j.d, j.gdt, P);
        }
    }
    cp_wait<0>();
    float *part = j.part + (int64_t)blockIdx.x * 3 * j.d;
    const bool want[3] = {j.dw_post != nullptr, j.dw_pre != nullptr,
                          T::GATE == 1 && j.dgate != nullptr};
#pragma unroll
    for (int k = 0; k < 3; ++k)
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
    if (bwd) return launch_walk<join_bwd_kernel<T>>(j, L, threads, kBwdBlocksPerSm, stream);
    return launch_walk<join_ring_kernel<T>>(j, L, threads, kFwdBlocksPerSm, stream);
}

}  // namespace
}  // namespace rvq
