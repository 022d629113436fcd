// moe_mx_quantize and moe_mx_dequantize: between 16- or 32-bit matrices and
// microscaled ones.
//
// Memory-bound: 2 or 4 bytes read and 1.03 or 0.53 written per value.  A lane holds
// eight values (16 or 32 bytes), a half warp the 128 columns that share a word of
// scales, so the largest magnitude of a block is two shuffles away and every store is
// whole words.  Blocks of 256 threads take up to four runs of 16 half warps, all of
// whose loads are in flight before the first is used.
//
// Measured (GB300): 8192 x 7168 fp32 to 8 bits 42.8 us (6.9 TB/s, the copy rate), bf16 35
// (5.0; bound by issue), back to bf16 27 (6.5); one row of 7168 1.3.
#include "mx.cuh"

namespace rvq {
namespace {

constexpr int kMost = 4;  // units of a thread

// 128 columns of a row: unit u is of row u / tiles.  One division per thread: its next
// unit is 16 further, `down` rows and `right` tiles.
struct Units {
    int tiles, down, right;
    uint32_t count;
};
struct Unit {
    int row, tile;
    __device__ __forceinline__ Unit(uint32_t u, const Units &k)
        : row((int)(u / (uint32_t)k.tiles)), tile((int)(u - (uint32_t)row * (uint32_t)k.tiles)) {}
    __device__ __forceinline__ void next(const Units &k) {
        row += k.down;
        tile += k.right;
        if (tile >= k.tiles) {
            tile -= k.tiles;
            ++row;
        }
    }
    // this lane's first column
    __device__ __forceinline__ int c() const {
        return tile * kMxTile + (int)(threadIdx.x & 15) * 8;
    }
};

template <int FMT, int XDT, int kUnits>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const MxQuantJob j,
                                                          const Units k) {
    dependency_wait();
    dependents_may_start();
    const uint32_t first = blockIdx.x * (16 * kUnits) + (threadIdx.x >> 4);
    // as they lie in memory: widening a unit at once would wait for its load before the
    // next one's
    constexpr int W = XDT == RVQ_F32 ? 2 : 1;
    uint4 raw[kUnits][W];
    Unit u(first, k);
#pragma unroll
    for (int i = 0; i < kUnits; ++i, u.next(k)) {
        const bool in = first + 16 * i < k.count && u.c() < j.cols;
        const char *p = reinterpret_cast<const char *>(j.x) +
                        ((int64_t)u.row * j.ldx + u.c()) * (XDT == RVQ_F32 ? 4 : 2);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            raw[i][w] = make_uint4(0u, 0u, 0u, 0u);
            if (in) raw[i][w] = reinterpret_cast<const uint4 *>(p)[w];
        }
    }
    u = Unit(first, k);
#pragma unroll
    for (int i = 0; i < kUnits; ++i, u.next(k)) {
        float v[8];
        const uint32_t w[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                               raw[i][W - 1].x, raw[i][W - 1].y, raw[i][W - 1].z, raw[i][W - 1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (XDT == RVQ_F32)
                v[e] = __uint_as_float(w[e]);
            else if (e % 2 == 0)
                unpack16(XDT, w[e / 2], v[e], v[e + 1]);
        mx_put8<FMT>(v, j.codes, j.scales, u.row, u.c(), k.tiles, first + 16 * i < k.count);
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

template <int FMT, int kUnits>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const MxDequantJob j,
                                                            const Units k) {
    dependency_wait();
    dependents_may_start();
    const uint32_t first = blockIdx.x * (16 * kUnits) + (threadIdx.x >> 4);
    uint2 q[kUnits];
    uint32_t s[kUnits];
    Unit u(first, k);
#pragma unroll
    for (int i = 0; i < kUnits; ++i, u.next(k)) {
        q[i] = make_uint2(0u, 0u);
        s[i] = 0u;
        if (first + 16 * i >= k.count || u.c() >= j.cols) continue;
        const int64_t at = (int64_t)u.row * k.tiles * kMxTile + u.c();
        if (FMT == MOE_MX_F8)
            q[i] = *reinterpret_cast<const uint2 *>(j.codes + at);
        else
            q[i].x = *reinterpret_cast<const uint32_t *>(j.codes + at / 2);
        s[i] = j.scales[mx_scale_at(u.row, u.tile, k.tiles) + (u.c() / kMxBlock & 3)];
    }
    u = Unit(first, k);
#pragma unroll
    for (int i = 0; i < kUnits; ++i, u.next(k)) {
        if (first + 16 * i >= k.count || u.c() >= j.cols) continue;
        float v[8];
        widen8<FMT>(q[i], v);
        const float scale = mx_scale(s[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
        st8(j.out, j.odt, (int64_t)u.row * j.ldo + u.c(), v);
    }
}

Units units_of(int rows, int cols) {
    Units k;
    k.tiles = mx_tiles(cols);
    k.down = 16 / k.tiles;
    k.right = 16 % k.tiles;
    k.count = (uint32_t)rows * (uint32_t)k.tiles;
    return k;
}

unsigned blocks_of(uint32_t units, int each) { return (units + 16 * each - 1) / (16 * each); }

// One unit per thread where more would leave SMs idle (one row of 7168: 2.5 us with four,
// 1.7 with one).
bool few(const Units &k) { return k.count <= (uint32_t)num_sms() * 16 * kMost; }

template <int FMT, int XDT>
rvq_status quantize_as(const MxQuantJob &job, cudaStream_t stream) {
    const Units k = units_of(job.rows, job.cols);
    if (few(k))
        RVQ_CUDA(launch_after(mx_quantize_kernel<FMT, XDT, 1>, blocks_of(k.count, 1), 256, 0, stream,
                              job, k));
    else
        RVQ_CUDA(launch_after(mx_quantize_kernel<FMT, XDT, kMost>, blocks_of(k.count, kMost), 256, 0,
                              stream, job, k));
    return RVQ_OK;
}

template <int FMT>
rvq_status quantize(const MxQuantJob &job, cudaStream_t stream) {
    if (job.xdt == RVQ_F32) return quantize_as<FMT, RVQ_F32>(job, stream);
    if (job.xdt == RVQ_BF16) return quantize_as<FMT, RVQ_BF16>(job, stream);
    return quantize_as<FMT, RVQ_F16>(job, stream);
}

template <int FMT>
rvq_status dequantize(const MxDequantJob &job, cudaStream_t stream) {
    const Units k = units_of(job.rows, job.cols);
    if (few(k))
        RVQ_CUDA(launch_after(mx_dequantize_kernel<FMT, 1>, blocks_of(k.count, 1), 256, 0, stream,
                              job, k));
    else
        RVQ_CUDA(launch_after(mx_dequantize_kernel<FMT, kMost>, blocks_of(k.count, kMost), 256, 0,
                              stream, job, k));
    return RVQ_OK;
}

}  // namespace

rvq_status launch_mx_quantize(const MxQuantJob &job, cudaStream_t stream) {
    return job.fmt == MOE_MX_F8 ? quantize<MOE_MX_F8>(job, stream)
                                : quantize<MOE_MX_F4>(job, stream);
}

rvq_status launch_mx_dequantize(const MxDequantJob &job, cudaStream_t stream) {
    return job.fmt == MOE_MX_F8 ? dequantize<MOE_MX_F8>(job, stream)
                                : dequantize<MOE_MX_F4>(job, stream);
}

}  // namespace rvq
