// Ways of an epilogue warp's values, one row per lane, into whole rows in memory: shared
// by the tiled products (dense_gemm.cu, mx_gemm.cu).
#pragma once

#include "dense.cuh"

namespace rvq {

// An epilogue warp's staging turns values held one row per lane into whole rows
// in memory: 32 rows of eight 16-byte groups, group j of row r at r * 8 + (j ^
// (r & 7)), conflict-free both ways.
__device__ __forceinline__ void turn_in(uint32_t turn, int lane, const float (&v)[32]) {
    __syncwarp();  // the rows before are read
#pragma unroll
    for (int j = 0; j < 8; ++j)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                         turn + lane * 128 + ((j ^ (lane & 7)) << 4)),
                     "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]), "f"(v[4 * j + 3])
                     : "memory");
    __syncwarp();
}

__device__ __forceinline__ void turn_out(uint32_t turn, int r, int j, float (&v)[4]) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(turn + r * 128 + ((j ^ (r & 7)) << 4))
                 : "memory");
}

// The residual of a 32 x 32 group, as turn_rows() wants it: row 4 i + lane / 8,
// columns 4 (lane % 8) ..; all loads in flight at once.
struct Residual {
    uint4 r[8];
    __device__ __forceinline__ void load(const void *p, int dt, int64_t ld, int lane, int row, int rows,
                                         int col, int width) {
        const int j = lane & 7, r0 = lane >> 3;
        const bool f32 = dt == RVQ_F32;
        const char *q = reinterpret_cast<const char *>(p) +
                        ((int64_t)(row + r0) * ld + col + 4 * j) * (f32 ? 4 : 2);
        const int64_t step = 4 * ld * (f32 ? 4 : 2);
        const bool on = p != nullptr && 4 * j < width;
#pragma unroll
        for (int i = 0; i < 8; ++i, q += step) {
            r[i] = make_uint4(0u, 0u, 0u, 0u);
            if (on && f32 && row + 4 * i + r0 < rows) r[i] = *reinterpret_cast<const uint4 *>(q);
            if (on && !f32 && row + 4 * i + r0 < rows) {
                const uint2 t = *reinterpret_cast<const uint2 *>(q);
                r[i].x = t.x;
                r[i].y = t.y;
            }
        }
    }
};

// The staged 32 x `width` values (plus a residual) to rows at (row, col): 128 (fp32)
// or 64 (16-bit) contiguous bytes per row, four rows per instruction.
// Everything is read before the first store: a test per row between loads and
// stores exposed each load's latency.
__device__ __forceinline__ void turn_rows(uint32_t turn, int lane, void *p, int dt, int64_t ld,
                                          int row, int rows, int col, int width,
                                          const Residual *res, int rdt) {
    const int j = lane & 7, r0 = lane >> 3;
    const bool on = 4 * j < width;
    float v[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_out(turn, 4 * i + r0, j, v[i]);
    if (res) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float b[4];
            if (rdt == RVQ_F32) {
                b[0] = __uint_as_float(res->r[i].x);
                b[1] = __uint_as_float(res->r[i].y);
                b[2] = __uint_as_float(res->r[i].z);
                b[3] = __uint_as_float(res->r[i].w);
            } else {
                unpack16(rdt, res->r[i].x, b[0], b[1]);
                unpack16(rdt, res->r[i].y, b[2], b[3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] += b[e];
        }
    }
    const int64_t at = (int64_t)(row + r0) * ld + col + 4 * j;
    if (dt == RVQ_F32) {
        float *q = reinterpret_cast<float *>(p) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, q += 4 * ld)
            if (on && row + 4 * i + r0 < rows)
                *reinterpret_cast<float4 *>(q) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
    } else {
        uint16_t *q = reinterpret_cast<uint16_t *>(p) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, q += 4 * ld)
            if (on && row + 4 * i + r0 < rows)
                *reinterpret_cast<uint2 *>(q) =
                    make_uint2(pack16(dt, v[i][0], v[i][1]), pack16(dt, v[i][2], v[i][3]));
    }
}

// 32 values per lane, one row per lane, to 16-bit rows without a residual:
// rounded first, so half as much goes through the staging (32 rows of four
// 16-byte groups, group j of row r at r * 4 + (j ^ (r / 2 & 3))).
__device__ __forceinline__ void rows_16_plain(uint32_t turn, int lane, void *p, int dt, int64_t ld,
                                              int row, int rows, int col, int width,
                                              const float (&v)[32]) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = pack16(dt, v[2 * e], v[2 * e + 1]);
    __syncwarp();  // the rows before are read
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         turn + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)),
                     "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                     : "memory");
    __syncwarp();
    const int j = lane & 3, r0 = lane >> 2;
    uint4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + r0;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(o[i].x), "=r"(o[i].y), "=r"(o[i].z), "=r"(o[i].w)
                     : "r"(turn + r * 64 + ((j ^ ((r >> 1) & 3)) << 4))
                     : "memory");
    }
    uint16_t *q = reinterpret_cast<uint16_t *>(p) + (int64_t)(row + r0) * ld + col + 8 * j;
#pragma unroll
    for (int i = 0; i < 4; ++i, q += 8 * ld)
        if (8 * j < width && row + 8 * i + r0 < rows) *reinterpret_cast<uint4 *>(q) = o[i];
}

}  // namespace rvq
