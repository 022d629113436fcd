// Tensor-core helpers of the microscaled products (mx_gemm.cu, mx_stream.cu).  Inline
// PTX; sm_100 family.
//
// A slice of an operand is 128 bytes of shared memory deep (one 128-byte swizzled row):
//   kind::mxf4       both operands e2m1, packed: 256 columns, four MMAs 64 deep
//   kind::mxf8f6f4   e4m3, or e2m1 in a byte's room each (16 values, 8 bytes of them
//                    and 8 of padding, as TMA unpacks them): 128 columns, four MMAs 32
//                    deep
// Scales: a tile of 128 rows x 4 blocks (512 bytes) is copied as it lies into four
// columns of tensor memory (column r / 32, lane r % 32, byte = block, for all four
// groups of 32 lanes).  A slice has one tile (mxf8f6f4) or two (mxf4) per 128 rows.
// MMAs read the bytes of their blocks: one, or two at place 0 or 2.
#pragma once

#include "dense_tc.cuh"
#include "mx.cuh"

namespace rvq {

// Shared-memory descriptor of a tile of scales: 32 rows of 16 bytes, no swizzle, 8-row
// groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)1u << 16;
    d |= (uint64_t)(128u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    return d;
}

template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
    if (CTAS == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
                     "l"(scale_desc(saddr))
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
                     "l"(scale_desc(saddr))
                     : "memory");
}

// Instruction descriptor but for the places of the scales: formats 0 = e4m3, 5 = e2m1
// (mxf8f6f4) or 1 = e2m1 (mxf4); scales e8m0; both operands K-major.
inline uint32_t mx_idesc(bool f4, int afmt, int bfmt, int M, int N) {
    const uint32_t a = f4 ? 1u : afmt == MOE_MX_F8 ? 0u : 5u;
    const uint32_t b = f4 ? 1u : bfmt == MOE_MX_F8 ? 0u : 5u;
    return (a << 7) | (b << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t scale_places(uint32_t id) { return (id << 4) | (id << 29); }

template <int CTAS, bool F4>
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t sa, uint32_t sb, uint32_t acc) {
#define RVQ_MX_MMA(CTA, KIND)                                                                   \
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"                                    \
                 "tcgen05.mma.cta_group::" CTA ".kind::" KIND                                   \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),                             \
                 "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)                         \
                 : "memory")
    if (CTAS == 1 && F4) RVQ_MX_MMA("1", "mxf4.block_scale.scale_vec::2X");
    if (CTAS == 1 && !F4) RVQ_MX_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
    if (CTAS == 2 && F4) RVQ_MX_MMA("2", "mxf4.block_scale.scale_vec::2X");
    if (CTAS == 2 && !F4) RVQ_MX_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
#undef RVQ_MX_MMA
}

// Bytes that TMA counts for `rows` rows of a slice: a 4-bit operand in a byte's room
// each counts as it lies in memory.
__host__ __device__ __forceinline__ uint32_t slice_bytes(bool f4, int fmt, int rows) {
    return (uint32_t)rows * (f4 || fmt == MOE_MX_F8 ? 128u : 64u);
}

// Tensor maps (mx_gemm.cu): boxes of one slice x box_rows rows of codes; of one
// slice's tiles x box_tiles (groups of 128 rows) of scales.  `f4`: for kind::mxf4.
rvq_status encode_codes(CUtensorMap *map, const uint8_t *codes, int rows, int cols, int fmt,
                        bool f4, int box_rows);
rvq_status encode_scales(CUtensorMap *map, const uint8_t *scales, int rows, int cols, bool f4,
                         int box_tiles);

// A product of microscaled matrices: out = residual + alpha act(x w0^T + bias0), or
// (mats 2) act(x w0^T + bias0) * (x w1^T + bias1), in odt, or microscaled (codes).
struct MxJob {
    int mats, n, rows, cols;
    const uint8_t *x, *xs;
    int xfmt;
    const uint8_t *w[2], *ws[2];
    int wfmt;
    const float *bias[2];
    int act;
    float alpha;
    const void *residual;
    int rdt;
    int64_t ldr;
    void *out;
    int odt;
    int64_t ldo;
    uint8_t *codes, *scales;  // microscaled output instead of out
    int ofmt;
    uint32_t *status;
    bool f4() const { return xfmt == MOE_MX_F4 && wfmt == MOE_MX_F4; }
};
rvq_status launch_mx_product(const MxJob &job, cudaStream_t stream);

// How a product's weights are streamed: CTAs that share a tile's depth, tiles (of 128
// weight rows, up to 128 tokens), slices of the whole depth, and whether two CTAs fit an
// SM.
struct MxStreamPlan {
    int split, slices;
    long long tiles;
    bool two;
};
MxStreamPlan plan_mx_stream(const MxJob &job);
rvq_status launch_mx_stream(const MxJob &job, cudaStream_t stream);
// Whether tiles of CTA pairs take the product (n, rows, cols, mats and formats of job).
bool mx_by_tiles(const MxJob &job);

}  // namespace rvq
