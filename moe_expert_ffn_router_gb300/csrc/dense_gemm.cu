// Matrix products of the dense operators (shared expert, dense projections)
// on the tensor cores: every mode of DenseJob in one persistent kernel.
//
// Compute-bound at prefill and training sizes (2 M N K operations against
// (M K + N K + M N) elements), so the design feeds tcgen05.mma without a pause:
//  * A pair of CTAs (a cluster of two) owns a 256 x tile_n output tile: CTA r
//    holds rows 128 r .. 128 r + 127 of A and half of B's rows, the leader's
//    one thread issues cta_group::2 MMAs on both halves.  Pairing halves the
//    shared memory and L2 traffic of B per operation.
//  * Both operands arrive by TMA in 64-deep slices (one 128-byte swizzled row
//    of 16-bit elements), seven 32 KB stages per CTA; the slices of both CTAs
//    complete on the leader's barrier.
//  * A transposed operand (stored [K][rows]) is loaded as it lies, in boxes of
//    64 rows x 64 deep, and read through MN-major descriptors, so the gradients
//    need no transposed copies.
//  * Accumulators are fp32 in tensor memory, two of up to 256 columns: eight
//    warps per CTA write one tile out while the next one is multiplied.
//  * A gated product loads its gate half from B0 (leader) and its up half from
//    B1 (follower), so both projections of an output lie in one accumulator row
//    and act(g) * u is formed in registers.
// Rows, columns and depth past the ends are zero-filled by TMA and not stored.
// Each output is rounded once, from fp32.  Every wait is bounded (1 s).
#include "dense_tc.cuh"

#include <cudaTypedefs.h>

namespace rvq {
namespace {

constexpr int DG_BM = 128;   // rows of A per CTA
constexpr int DG_BK = 64;    // depth of a slice
constexpr int DG_ST = 7;     // stages
constexpr int DG_ABYTES = DG_BM * DG_BK * 2;
constexpr int DG_STAGE = 2 * DG_ABYTES;     // A, and up to 128 rows of B
constexpr int DG_SMEM = DG_ST * DG_STAGE + 256;
constexpr int DG_EPI_WARPS = 8;
constexpr int DG_THREADS = 32 * (4 + DG_EPI_WARPS);
constexpr int DG_ACC = 256;  // TMEM columns per accumulator
constexpr int DG_GROUP = 8;  // M tiles walked together (operand reuse in L2)
static_assert(DG_SMEM <= 232448, "shared memory of a CTA");

struct GemmArgs {
    int mode, M, N, a_t, b_t;
    int kb;              // slices of one product
    int tile_n, half;    // columns of an accumulator; rows of B per CTA
    int mt, nt;          // output tiles (M tiles of both problems for PAIR_M)
    uint32_t idesc;
    int dt, act, rdt, odt;
    int wide;            // rows of out (1) and pre (2) start on 32 bytes
    float alpha;
    const void *bias[2], *residual;
    int64_t ldr, ldo;
    void *out[2];
    float *pre[2];
    uint32_t *status;
};

__device__ __forceinline__ void arrive_cluster(uint32_t mbar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mbar)
                 : "memory");
}

// box at (col, row) into this CTA's shared memory, counted on the leader's barrier
__device__ __forceinline__ void tma_pair(uint32_t dst, const CUtensorMap *tm, int col, int row,
                                         uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(col), "r"(row), "r"(mbar)
        : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

// arrives on the barrier at this offset in both CTAs once the MMAs issued so
// far are done
__device__ __forceinline__ void commit_pair(uint32_t mbar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(mbar),
        "h"((uint16_t)3)
        : "memory");
}

// output tile t -> (m tile, n tile): groups of DG_GROUP M tiles, N inside
__device__ __forceinline__ void tile_at(const GemmArgs &g, int t, int &m, int &n) {
    const int grp = t / (DG_GROUP * g.nt);
    const int first = grp * DG_GROUP;
    const int rows = min(DG_GROUP, g.mt - first);
    const int r = t - grp * DG_GROUP * g.nt;
    m = first + r % rows;
    n = r / rows;
}

// 32 bytes of one lane: one whole sector per lane and instruction
__device__ __forceinline__ void st32(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 16 (or the first 8) consecutive outputs; `wide`: rows start on 32 bytes
__device__ __forceinline__ void store16(void *p, int dt, int64_t at, const float (&v)[16], int cols,
                                        bool wide) {
    if (cols == 16 && wide) {
        uint32_t w[8];
        if (dt == RVQ_F32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[8 * h + e]);
                st32(reinterpret_cast<float *>(p) + at + 8 * h, w);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack16(dt, v[2 * e], v[2 * e + 1]);
            st32(reinterpret_cast<uint16_t *>(p) + at, w);
        }
        return;
    }
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        lo[e] = v[e];
        hi[e] = v[8 + e];
    }
    st8(p, dt, at, lo);
    if (cols == 16) st8(p, dt, at + 8, hi);
}

__device__ __forceinline__ void add_bias16(const void *bias, int dt, int c, int cols,
                                           float (&v)[16]) {
    if (bias == nullptr) return;
    float b[8];
    ld8(bias, dt, c, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += b[e];
    if (cols == 16) {
        ld8(bias, dt, c + 8, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 + e] += b[e];
    }
}

template <bool GATED>
__global__ void __launch_bounds__(DG_THREADS, 1) dense_gemm_kernel(
    const __grid_constant__ CUtensorMap ma0, const __grid_constant__ CUtensorMap ma1,
    const __grid_constant__ CUtensorMap mb0, const __grid_constant__ CUtensorMap mb1,
    const __grid_constant__ GemmArgs g) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int tiles = g.mt * g.nt;
    const int mt1 = g.mode == DG_PAIR_M ? g.mt / 2 : g.mt;  // M tiles of one problem
    const int slices = g.mode == DG_SUM_K ? 2 * g.kb : g.kb;
    uint8_t *bars = smem + DG_ST * DG_STAGE;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * DG_ST,
                   accfull0 = empty0 + 8 * DG_ST, accempty0 = accfull0 + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 8 * (2 * DG_ST + 4));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < DG_ST; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accfull0 + 8 * b, 1);
            mbar_init(accempty0 + 8 * b, 2 * DG_EPI_WARPS);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        // one CTA per SM (shared memory), so the allocation never waits
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tslot)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();  // the peer's barriers and TMEM are ready too
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tslot;

    if (warp == 0) {
        // producer: this CTA's rows of A and of B for every slice
        const int bboxes = g.b_t ? (g.half + 63) / 64 : 1;
        const uint32_t bytes = DG_ABYTES + (g.b_t ? bboxes * 8192 : g.half * 128);
        int it = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
            int m, n;
            tile_at(g, t, m, n);
            const bool second = m >= mt1;
            const int m0 = (second ? m - mt1 : m) * 2 * DG_BM + (int)rank * DG_BM;
            const int n0 = GATED ? n * g.half : n * g.tile_n + (int)rank * g.half;
            for (int k = 0; k < slices; ++k, ++it) {
                const int s = it % DG_ST;
                if (it >= DG_ST && !warp_wait(empty0 + 8 * s, ((it / DG_ST) - 1) & 1, abort_flag,
                                              g.status)) {
                    ok = false;
                    break;
                }
                const bool k2 = k >= g.kb;
                const int kx = (k2 ? k - g.kb : k) * DG_BK;
                const CUtensorMap *ta = (second || k2) ? &ma1 : &ma0;
                const CUtensorMap *tb = (GATED ? rank == 1 : k2) ? &mb1 : &mb0;
                const uint32_t st = smem_u32(smem + s * DG_STAGE), sb = st + DG_ABYTES;
                const uint32_t bar = cluster_addr(full0 + 8 * s, 0);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * bytes);
                    if (g.a_t) {
                        tma_pair(st, ta, m0, kx, bar);
                        tma_pair(st + 8192, ta, m0 + 64, kx, bar);
                    } else {
                        tma_pair(st, ta, kx, m0, bar);
                    }
                    if (g.b_t) {
                        tma_pair(sb, tb, n0, kx, bar);
                        if (bboxes > 1) tma_pair(sb + 8192, tb, n0 + 64, kx, bar);
                    } else {
                        tma_pair(sb, tb, kx, n0, bar);
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp == 1 && rank == 0) {
        // issuer: four 16-deep MMAs per slice
        const uint32_t da = g.a_t ? 2048u >> 4 : 2u, db = g.b_t ? 2048u >> 4 : 2u;
        int it = 0, done = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs, ++done) {
            const int buf = done & 1;
            if (done >= 2 && !warp_wait(accempty0 + 8 * buf, ((done >> 1) - 1) & 1, abort_flag,
                                             g.status))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + (uint32_t)(buf * DG_ACC);
            for (int k = 0; k < slices; ++k, ++it) {
                const int s = it % DG_ST;
                if (!warp_wait(full0 + 8 * s, (it / DG_ST) & 1, abort_flag, g.status)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t st = smem_u32(smem + s * DG_STAGE);
                const uint64_t a = operand_desc(st, g.a_t),
                               b = operand_desc(st + DG_ABYTES, g.b_t);
                if (elect_one()) {
#pragma unroll
                    for (int q = 0; q < DG_BK / 16; ++q)
                        mma_pair(acc, a + q * da, b + q * db, g.idesc, (k > 0 || q > 0) ? 1u : 0u);
                    commit_pair(empty0 + 8 * s);
                }
                __syncwarp();
            }
            if (elect_one()) commit_pair(accfull0 + 8 * buf);
            __syncwarp();
        }
    } else if (warp >= 4) {
        // epilogue: lanes 32 q .. 32 q + 31 of the accumulator, every other
        // group of 16 columns
        const int q = warp & 3, par = (warp - 4) >> 2;
        const int units = (GATED ? g.half : g.tile_n) / 16;
        int done = 0;
        for (int t = pair; t < tiles; t += pairs, ++done) {
            int m, n;
            tile_at(g, t, m, n);
            const bool second = m >= mt1;
            const int row = (second ? m - mt1 : m) * 2 * DG_BM + (int)rank * DG_BM + 32 * q + lane;
            const int buf = done & 1;
            if (!warp_wait(accfull0 + 8 * buf, (done >> 1) & 1, abort_flag, g.status)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + (uint32_t)(buf * DG_ACC) + ((uint32_t)(32 * q) << 16);
            void *out = g.out[second ? 1 : 0];
            for (int u = par; u < units; u += 2) {
                uint32_t r0[16], r1[16];
                tmem_ld16(acc + 16 * u, r0);
                if (GATED) tmem_ld16(acc + g.half + 16 * u, r1);
                tmem_wait();
                const int c = n * (GATED ? g.half : g.tile_n) + 16 * u;
                const int cols = min(16, g.N - c);
                if (row < g.M && cols > 0) {
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r0[e]);
                    add_bias16(g.bias[0], g.dt, c, cols, v);
                    if (g.pre[0]) store16(g.pre[0], RVQ_F32, (int64_t)row * g.N + c, v, cols,
                                              g.wide & 2);
                    act_group(g.act, v);
                    if (GATED) {
                        float w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __uint_as_float(r1[e]);
                        add_bias16(g.bias[1], g.dt, c, cols, w);
                        if (g.pre[1]) store16(g.pre[1], RVQ_F32, (int64_t)row * g.N + c, w, cols,
                                                  g.wide & 2);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] *= w[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] *= g.alpha;
                        add_bias16(g.residual ? (const char *)g.residual +
                                                    (int64_t)row * g.ldr * (g.rdt == RVQ_F32 ? 4 : 2)
                                              : nullptr,
                                   g.rdt, c, cols, v);
                    }
                    store16(out, g.odt, (int64_t)row * g.ldo + c, v, cols, g.wide & 1);
                }
                __syncwarp();
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_cluster(cluster_addr(accempty0 + 8 * buf, 0));
        }
    }
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        // copies and MMAs still in flight end well within this time
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 2000000ull) __nanosleep(1000);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();  // the peer no longer needs this CTA's shared memory or TMEM
    if (warp == 2) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
}

// Columns of an accumulator: the width with the least (waves of CTA pairs) x
// (time of a slice), where a slice costs its MMAs (2 tile_n cycles) or, for
// narrow tiles, its operand fill ((128 + tile_n / 2) rows of 128 bytes at about
// 72 bytes per cycle and SM).
int choose_tile_n(const DenseJob &j, int mt, int pairs) {
    int best = 0;
    double cost = 1e300;
    for (int tn = 256; tn >= 64; tn -= 32) {
        if (j.b_t && tn != 256 && tn != 128) continue;  // whole 64-row boxes per CTA
        const int per = j.mode == DG_GATED ? tn / 2 : tn;
        const long long tiles = (long long)mt * ((j.N + per - 1) / per);
        const double waves = (double)((tiles + pairs - 1) / pairs);
        const double fill = (128.0 + tn / 2) * 128.0 / 72.0;
        const double c = waves * (2.0 * tn > fill ? 2.0 * tn : fill);
        if (c < cost * 0.999) {
            cost = c;
            best = tn;
        }
    }
    return best;
}

}  // namespace

rvq_status encode_operand(CUtensorMap *map, const void *p, int rows, int K, int64_t ld, int t, int dt,
                          int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode =
        reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder_entry());
    if (encode == nullptr) {
        set_error("dense product: cuTensorMapEncodeTiled is not available");
        return RVQ_ECUDA;
    }
    const cuuint64_t dims[2] = {(cuuint64_t)(t ? rows : K), (cuuint64_t)(t ? K : rows)};
    const cuuint64_t pitch[1] = {(cuuint64_t)ld * 2u};
    const cuuint32_t box[2] = {64u, (cuuint32_t)(t ? 64 : box_rows)};
    const cuuint32_t step[2] = {1u, 1u};
    const CUresult r =
        encode(map, dt == RVQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               2, const_cast<void *>(p), dims, pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("dense product: cuTensorMapEncodeTiled failed (%d)", (int)r);
        return RVQ_ECUDA;
    }
    return RVQ_OK;
}

rvq_status launch_dense_gemm(const DenseJob &job, cudaStream_t stream) {
    if (dense_stream_fits(job)) return launch_dense_stream(job, stream);
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(dense_gemm_kernel<false>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, DG_SMEM));
        RVQ_CUDA(cudaFuncSetAttribute(dense_gemm_kernel<true>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, DG_SMEM));
        attr_done[dev] = 1;
    }
    const bool gated = job.mode == DG_GATED;
    const int pairs_max = num_sms() / 2;
    GemmArgs g = {};
    g.mode = job.mode;
    g.M = job.M;
    g.N = job.N;
    g.a_t = job.a_t;
    g.b_t = job.b_t;
    g.kb = (job.K + DG_BK - 1) / DG_BK;
    g.mt = (job.M + 2 * DG_BM - 1) / (2 * DG_BM) * (job.mode == DG_PAIR_M ? 2 : 1);
    g.tile_n = choose_tile_n(job, g.mt, pairs_max);
    g.half = g.tile_n / 2;
    const int per = gated ? g.half : g.tile_n;
    g.nt = (job.N + per - 1) / per;
    const long long tiles = (long long)g.mt * g.nt;
    if (tiles > 0x7fffffffll / DG_GROUP) {
        set_error("dense product: %lld output tiles", tiles);
        return RVQ_ENOTIMPL;
    }
    const uint32_t fmt = job.dt == RVQ_BF16 ? 1u : 0u;
    g.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)job.a_t << 15) |
              ((uint32_t)job.b_t << 16) | ((uint32_t)(g.tile_n >> 3) << 17) |
              ((uint32_t)(2 * DG_BM >> 4) << 24);
    g.dt = job.dt;
    g.act = job.act;
    g.rdt = job.rdt;
    g.odt = job.odt;
    g.alpha = job.alpha;
    g.residual = job.residual;
    g.ldr = job.ldr;
    g.ldo = job.ldo;
    for (int i = 0; i < 2; ++i) {
        g.bias[i] = job.bias[i];
        g.out[i] = job.out[i];
        g.pre[i] = job.pre[i];
    }
    g.status = job.status;
    const int64_t oe = job.odt == RVQ_F32 ? 4 : 2;
    const uintptr_t outs = (uintptr_t)job.out[0] | (uintptr_t)job.out[1] |
                           (uintptr_t)(job.ldo * oe) | (uintptr_t)(per * oe);
    const uintptr_t pres = (uintptr_t)job.pre[0] | (uintptr_t)job.pre[1] | (uintptr_t)(per * 4);
    g.wide = ((outs & 31) == 0 ? 1 : 0) | ((pres & 31) == 0 ? 2 : 0);
    CUtensorMap ma[2], mb[2];
    for (int i = 0; i < 2; ++i) {
        if (i == 1 && job.a[1] == nullptr)
            ma[1] = ma[0];
        else
            RVQ_TRY(encode_operand(&ma[i], job.a[i], job.M, job.K, job.lda, job.a_t, job.dt, DG_BM));
        if (i == 1 && job.b[1] == nullptr)
            mb[1] = mb[0];
        else
            RVQ_TRY(encode_operand(&mb[i], job.b[i], job.N, job.K, job.ldb, job.b_t, job.dt, g.half));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs_max ? tiles : pairs_max)));
    cfg.blockDim = dim3(DG_THREADS);
    cfg.dynamicSmemBytes = DG_SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (gated)
        RVQ_CUDA(cudaLaunchKernelEx(&cfg, dense_gemm_kernel<true>, ma[0], ma[1], mb[0], mb[1], g));
    else
        RVQ_CUDA(cudaLaunchKernelEx(&cfg, dense_gemm_kernel<false>, ma[0], ma[1], mb[0], mb[1], g));
    RVQ_LAUNCHED("dense_gemm");
    return RVQ_OK;
}

}  // namespace rvq
