// moe_mx_quantize and moe_mx_dequantize: between 16- or 32-bit matrices and
// microscaled ones.
//
// Memory-bound: 2 or 4 bytes read and 1.03 or 0.53 written per value.  A lane holds
// eight values (16 or 32 bytes), a half warp the 128 columns that share a word of
// scales, so the largest magnitude of a block is two shuffles away and every store is
// whole words.  Blocks of 256 threads take kUnits runs of 16 half warps, all of
// whose loads are in flight before the first is used.
#include "mx.cuh"

namespace rvq {
namespace {

constexpr int kUnits = 4;

// 128 columns of a row
struct Unit {
    int row, tile, c;
    bool in;  // this lane's eight columns are the matrix's
};

__device__ __forceinline__ Unit unit_at(uint32_t u, uint32_t units, int tiles, int cols) {
    Unit r;
    const uint32_t row = u / (uint32_t)tiles;
    r.row = (int)row;
    r.tile = (int)(u - row * (uint32_t)tiles);
    r.c = r.tile * kMxTile + (int)(threadIdx.x & 15) * 8;
    r.in = u < units && r.c < cols;
    return r;
}

template <int FMT, int XDT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantJob j, int tiles,
                                                          uint32_t units) {
    dependency_wait();
    dependents_may_start();
    const uint32_t first = blockIdx.x * (16 * kUnits) + (threadIdx.x >> 4);
    float v[kUnits][8];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_at(first + 16 * i, units, tiles, j.cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
        if (u.in) ld8(j.x, XDT, (int64_t)u.row * j.ldx + u.c, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_at(first + 16 * i, units, tiles, j.cols);
        mx_put8<FMT>(v[i], j.codes, j.scales, u.row, u.c, tiles, first + 16 * i < units);
    }
}

template <int FMT>
__device__ __forceinline__ void widen8(uint2 q, float (&v)[8]) {
    uint32_t h[4];
    if (FMT == MOE_MX_F8) {
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                : "=r"(h[i])
                : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
    } else {
        asm("{\n.reg .b8 a, b, c, d;\n"
            "mov.b32 {a, b, c, d}, %4;\n"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(q.x));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack16(RVQ_F16, h[i], v[2 * i], v[2 * i + 1]);
}

template <int FMT>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const MxDequantJob j, int tiles,
                                                            uint32_t units) {
    dependency_wait();
    dependents_may_start();
    const uint32_t first = blockIdx.x * (16 * kUnits) + (threadIdx.x >> 4);
    uint2 q[kUnits];
    uint32_t s[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_at(first + 16 * i, units, tiles, j.cols);
        q[i] = make_uint2(0u, 0u);
        s[i] = 0u;
        if (!u.in) continue;
        const int64_t at = (int64_t)u.row * tiles * kMxTile + u.c;
        if (FMT == MOE_MX_F8)
            q[i] = *reinterpret_cast<const uint2 *>(j.codes + at);
        else
            q[i].x = *reinterpret_cast<const uint32_t *>(j.codes + at / 2);
        s[i] = j.scales[mx_scale_at(u.row, u.tile, tiles) + (u.c / kMxBlock & 3)];
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const Unit u = unit_at(first + 16 * i, units, tiles, j.cols);
        if (!u.in) continue;
        float v[8];
        widen8<FMT>(q[i], v);
        const float scale = mx_scale(s[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
        st8(j.out, j.odt, (int64_t)u.row * j.ldo + u.c, v);
    }
}

unsigned blocks_of(uint32_t units) { return (units + 16 * kUnits - 1) / (16 * kUnits); }

template <int FMT>
rvq_status quantize(const MxQuantJob &job, int tiles, uint32_t units, cudaStream_t stream) {
    const dim3 grid(blocks_of(units));
    if (job.xdt == RVQ_F32)
        RVQ_CUDA(launch_after(mx_quantize_kernel<FMT, RVQ_F32>, grid, 256, 0, stream, job, tiles, units));
    else if (job.xdt == RVQ_BF16)
        RVQ_CUDA(launch_after(mx_quantize_kernel<FMT, RVQ_BF16>, grid, 256, 0, stream, job, tiles, units));
    else
        RVQ_CUDA(launch_after(mx_quantize_kernel<FMT, RVQ_F16>, grid, 256, 0, stream, job, tiles, units));
    return RVQ_OK;
}

}  // namespace

rvq_status launch_mx_quantize(const MxQuantJob &job, cudaStream_t stream) {
    const int tiles = mx_tiles(job.cols);
    const uint32_t units = (uint32_t)job.rows * (uint32_t)tiles;
    return job.fmt == MOE_MX_F8 ? quantize<MOE_MX_F8>(job, tiles, units, stream)
                                : quantize<MOE_MX_F4>(job, tiles, units, stream);
}

rvq_status launch_mx_dequantize(const MxDequantJob &job, cudaStream_t stream) {
    const int tiles = mx_tiles(job.cols);
    const uint32_t units = (uint32_t)job.rows * (uint32_t)tiles;
    const dim3 grid(blocks_of(units));
    if (job.fmt == MOE_MX_F8)
        RVQ_CUDA(launch_after(mx_dequantize_kernel<MOE_MX_F8>, grid, 256, 0, stream, job, tiles, units));
    else
        RVQ_CUDA(launch_after(mx_dequantize_kernel<MOE_MX_F4>, grid, 256, 0, stream, job, tiles, units));
    return RVQ_OK;
}

}  // namespace rvq
