// Products of microscaled matrices: tensor maps and the choice of a kernel.
#include "mx_tc.cuh"

#include <cudaTypedefs.h>

namespace rvq {

static rvq_status encode(CUtensorMap *map, CUtensorMapDataType type, const void *p, uint64_t inner,
                         uint64_t outer, uint64_t pitch, uint32_t box_inner, uint32_t box_outer,
                         CUtensorMapSwizzle swizzle) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn =
        reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder_entry());
    if (fn == nullptr) {
        set_error("microscaled product: cuTensorMapEncodeTiled is not available");
        return RVQ_ECUDA;
    }
    const cuuint64_t dims[2] = {inner, outer}, pitches[1] = {pitch};
    const cuuint32_t box[2] = {box_inner, box_outer}, step[2] = {1u, 1u};
    const CUresult r = fn(map, type, 2, const_cast<void *>(p), dims, pitches, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("microscaled product: cuTensorMapEncodeTiled failed (%d)", (int)r);
        return RVQ_ECUDA;
    }
    return RVQ_OK;
}

rvq_status encode_codes(CUtensorMap *map, const uint8_t *codes, int rows, int cols, int fmt,
                        bool f4, int box_rows) {
    const uint64_t pitch = (uint64_t)mx_pitch(fmt, cols);
    // packed e2m1 of a mixed product: a byte's room each in shared memory
    if (fmt == MOE_MX_F4 && !f4)
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, codes, 2 * pitch, (uint64_t)rows,
                      pitch, 128, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, pitch, (uint64_t)rows, pitch, 128,
                  (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

rvq_status encode_scales(CUtensorMap *map, const uint8_t *scales, int rows, int cols, bool f4,
                         int box_tiles) {
    const uint64_t words = (uint64_t)mx_tiles(cols) * (kMxTileBytes / 4);
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, words, (uint64_t)mx_tiles(rows),
                  words * 4, f4 ? 256 : 128, (uint32_t)box_tiles, CU_TENSOR_MAP_SWIZZLE_NONE);
}

rvq_status launch_mx_product(const MxJob &job, cudaStream_t stream) {
    return launch_mx_stream(job, stream);
}

}  // namespace rvq
