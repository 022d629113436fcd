// Internal declarations of the microscaled operators: quantisation (mx_quant.cu), the
// norm join with a microscaled output (mx_join.cu) and the products (mx_gemm.cu,
// mx_stream.cu); their host side is mx_api.cu.
//
// A microscaled matrix: blocks of 32 values along a row share a scale 2^(byte - 127).
// Codes are row-major, columns padded with zeros to a multiple of 128: e4m3 a byte
// each, e2m1 two to a byte, the lower column in the lower half.  Scale bytes lie in
// tiles of 128 rows x 4 blocks (512 bytes), a tile as the tensor cores take it: byte
// (row % 32) * 16 + (row / 32 % 4) * 4 + block % 4; tiles of the same rows follow one
// another.  A row's four scales of 128 columns are one aligned word.
#pragma once

#include "dense.cuh"

namespace rvq {

constexpr int kMxBlock = 32;
constexpr int kMxTile = 128;       // rows of a tile of scales; columns it covers
constexpr int kMxTileBytes = 512;

__host__ __device__ inline int mx_tiles(int v) { return (v + kMxTile - 1) / kMxTile; }
inline int64_t mx_pitch(int fmt, int cols) {
    return (int64_t)mx_tiles(cols) * (fmt == MOE_MX_F8 ? kMxTile : kMxTile / 2);
}

// Place of the four scales of row `row`, columns 128 t ..; tiles = mx_tiles(cols).
__device__ __forceinline__ int64_t mx_scale_at(int row, int t, int tiles) {
    const uint32_t r = (uint32_t)row;
    return ((int64_t)(r / kMxTile) * tiles + t) * kMxTileBytes + (r % 32) * 16 + (r / 32 % 4) * 4;
}

// 2^(byte - 127); 255 is NaN
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// Scale byte of a block from the largest of its magnitudes' bits: the power of two
// that takes it below twice the format's largest power of two (2^8, 2^2), at least
// 2^-127; 255 where one is not finite.
template <int FMT>
__device__ __forceinline__ uint32_t mx_byte(uint32_t top) {
    const uint32_t e = top >> 23, lead = FMT == MOE_MX_F8 ? 8 : 2;
    return e == 255 ? 255 : e > lead ? e - lead : 0;
}

// 1 / scale, a normal number for every byte below 255; 0 for 255
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return __uint_as_float(byte == 255 ? 0u : (254u - byte) << 23);
}

__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    return m;
}

// Eight values over their scale, rounded to even, ends at the format's largest.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Four adjacent lanes hold a block of 32 values, eight each (column `c` of row `row`):
// the codes and, four blocks (16 lanes) at a time, the scales.  All lanes of the half
// warp take part; what lies behind the matrix is zero in v.  `on`: the lane's columns
// are within the padded row.
template <int FMT>
__device__ __forceinline__ void mx_put8(const float (&v)[8], uint8_t *codes, uint8_t *scales,
                                        int row, int c, int tiles, bool on) {
    uint32_t top = top8(v);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t byte = mx_byte<FMT>(top);
    const float inv = mx_inverse(byte);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = byte == 255 ? 0.f : v[e] * inv;
    if (on) {
        const int64_t at = (int64_t)row * tiles * kMxTile + c;
        if (FMT == MOE_MX_F8)
            *reinterpret_cast<uint2 *>(codes + at) =
                make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
        else
            *reinterpret_cast<uint32_t *>(codes + at / 2) = e2m1x8(q);
    }
    // bytes of lanes 0, 4, 8, 12 of the half warp
    uint32_t word = byte << (8 * ((threadIdx.x >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (on && (threadIdx.x & 15) == 0)
        *reinterpret_cast<uint32_t *>(scales + mx_scale_at(row, c / kMxTile, tiles)) = word;
}

struct MxQuantJob {
    const void *x;
    int64_t ldx;
    int xdt;
    int rows, cols, fmt;
    uint8_t *codes, *scales;
};
rvq_status launch_mx_quantize(const MxQuantJob &job, cudaStream_t stream);

struct MxDequantJob {
    const uint8_t *codes, *scales;
    int rows, cols, fmt;
    void *out;
    int64_t ldo;
    int odt;
};
rvq_status launch_mx_dequantize(const MxDequantJob &job, cudaStream_t stream);

// moe_norm_join with xn microscaled too (join.xn may be NULL)
struct MxJoinJob {
    JoinJob join;
    int fmt;
    uint8_t *codes, *scales;
};
rvq_status launch_mx_join(const MxJoinJob &job, cudaStream_t stream);

}  // namespace rvq
