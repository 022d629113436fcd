// The forward products of the dense operators for few tokens (decode batches):
// moe_linear and moe_gated_linear as a stream of the weights.
//
// Memory-bound: rows x cols weights are read once and a handful of tokens are
// multiplied with each, so the weights take the place of the M operand (128 of
// their rows fill the tensor core's lanes, whatever the batch) and the tokens
// are the N operand, padded to a multiple of 16.
//  * A CTA multiplies a tile of 128 weight rows (64 gate rows and the 64 up rows
//    beside them for a gated product) with all tokens over one part of the
//    depth; a cluster of up to 8 CTAs splits the depth, so that even a matrix
//    of few rows keeps the memory system busy.
//  * Weights and tokens arrive by TMA in 64-deep slices through a ring of about
//    96 KB per CTA, two CTAs per SM (one of about 190 KB from 80 tokens on);
//    one thread issues the MMAs.
//  * The partial tiles (fp32) go to shared memory, and each CTA of the cluster
//    adds its share of the rows over the cluster in rank order (distributed
//    shared memory): no workspace, no atomics, results repeat bit for bit.
// Every wait is bounded (1 s).
#include "dense_tc.cuh"

namespace rvq {
namespace {

constexpr int DS_ROWS = 128;
constexpr int DS_BK = 64;
constexpr int DS_ABYTES = DS_ROWS * DS_BK * 2;
constexpr int DS_THREADS = 256;
constexpr int DS_MAX_ST = 10;
constexpr int DS_PITCH = DS_ROWS + 4;  // floats between tokens of a partial tile

struct StreamArgs {
    int n, rows, kb;      // tokens, rows of one matrix, 64-deep slices
    int npad;             // tokens padded to a multiple of 16
    int stages, split;    // ring depth; CTAs of a cluster
    uint32_t cols;        // TMEM columns
    uint32_t idesc;
    int dt, act, rdt, odt;
    float alpha;
    const void *bias[2], *residual;
    int64_t ldr, ldo;
    void *out;
    float *pre[2];
    uint32_t *status;
};

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *tm, int col, int row,
                                         uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(col), "r"(row), "r"(mbar)
        : "memory");
}

__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

template <bool GATED>
__global__ void __launch_bounds__(DS_THREADS, 2) dense_stream_kernel(
    const __grid_constant__ CUtensorMap mw0, const __grid_constant__ CUtensorMap mw1,
    const __grid_constant__ CUtensorMap mx, const __grid_constant__ StreamArgs g) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int TR = GATED ? DS_ROWS / 2 : DS_ROWS;  // rows of one matrix in a tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int tile = blockIdx.x / g.split;
    const int r0 = tile * TR;
    const int k0 = (int)((int64_t)g.kb * rank / g.split);
    const int k1 = (int)((int64_t)g.kb * (rank + 1) / g.split);
    const int stage = DS_ABYTES + g.npad * DS_BK * 2;
    __shared__ __align__(8) uint64_t bars[2 * DS_MAX_ST + 1];
    __shared__ uint32_t tslot;
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * DS_MAX_ST,
                   accfull = empty0 + 8 * DS_MAX_ST;
    if (threadIdx.x == 0) {
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(accfull, 1);
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        // an SM holds at most two such CTAs (shared memory), 256 columns each
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tslot)),
                     "r"(g.cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tslot;

    if (warp == 0) {
        for (int k = k0, it = 0; k < k1; ++k, ++it) {
            const int s = it % g.stages;
            if (it >= g.stages && !warp_wait(empty0 + 8 * s, ((it / g.stages) - 1) & 1, abort_flag,
                                             g.status))
                break;
            const uint32_t st = smem_u32(smem + s * stage), bar = full0 + 8 * s;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar, (uint32_t)stage);
                tma_load(st, &mw0, k * DS_BK, r0, bar);
                if (GATED) tma_load(st + DS_ABYTES / 2, &mw1, k * DS_BK, r0, bar);
                tma_load(st + DS_ABYTES, &mx, k * DS_BK, 0, bar);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        for (int k = k0, it = 0; k < k1; ++k, ++it) {
            const int s = it % g.stages;
            if (!warp_wait(full0 + 8 * s, (it / g.stages) & 1, abort_flag, g.status)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t st = smem_u32(smem + s * stage);
            const uint64_t a = operand_desc(st, 0), b = operand_desc(st + DS_ABYTES, 0);
            if (elect_one()) {
#pragma unroll
                for (int q = 0; q < DS_BK / 16; ++q)
                    mma_one(tmem, a + 2 * q, b + 2 * q, g.idesc, (it > 0 || q > 0) ? 1u : 0u);
                mma_commit(empty0 + 8 * s);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(accfull);
        __syncwarp();
    }
    // the partial tile, [token][row], over the ring (its last slice is consumed)
    warp_wait(accfull, 0, abort_flag, g.status);
    __syncthreads();
    const bool ok = !*abort_flag;  // no wait of this CTA is left that could raise it
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    float *part = reinterpret_cast<float *>(smem);
    if (ok) {
        const int q = warp & 3;
        for (int c = (warp >> 2) * 16; c < g.npad; c += 32) {
            uint32_t r[16];
            tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)c, r);
            tmem_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c + e < g.n) part[(c + e) * DS_PITCH + 32 * q + lane] = __uint_as_float(r[e]);
        }
    }
    __syncthreads();
    if (*abort_flag) {
        // copies and MMAs still in flight end well within this time
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 2000000ull) __nanosleep(1000);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();  // every partial tile of the cluster is in place
    if (ok) {
        const int quads = TR / 4 / g.split;  // groups of four rows this CTA finishes
        for (int i = threadIdx.x; i < g.n * quads; i += DS_THREADS) {
            const int t = i / quads, qr = (rank * quads + i % quads) * 4;
            const int r = r0 + qr;
            if (r >= g.rows) continue;
            const uint32_t at = smem_u32(part + t * DS_PITCH + qr);
            float v[4] = {}, u[4] = {};
            for (int p = 0; p < g.split; ++p) {
                const uint32_t a = cluster_addr(at, (uint32_t)p);
                const float4 x = ld_cluster4(a);
                v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
                if (GATED) {
                    const float4 y = ld_cluster4(a + TR * 4);
                    u[0] += y.x; u[1] += y.y; u[2] += y.z; u[3] += y.w;
                }
            }
            float b[4];
            if (g.bias[0]) {
                ld4(g.bias[0], g.dt, r, b);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += b[e];
            }
            if (g.pre[0]) st4(g.pre[0], RVQ_F32, (int64_t)t * g.rows + r, v);
            act_group(g.act, v);
            if (GATED) {
                if (g.bias[1]) {
                    ld4(g.bias[1], g.dt, r, b);
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[e] += b[e];
                }
                if (g.pre[1]) st4(g.pre[1], RVQ_F32, (int64_t)t * g.rows + r, u);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= u[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= g.alpha;
                if (g.residual) {
                    ld4(g.residual, g.rdt, (int64_t)t * g.ldr + r, b);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += b[e];
                }
            }
            st4(g.out, g.odt, (int64_t)t * g.ldo + r, v);
        }
    }
    cluster_sync();  // the peers' tiles stay in place until read
    if (warp == 2) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.cols));
    }
}

constexpr int kRingSmall = 96 << 10, kRingLarge = 190 << 10;
constexpr int kSmallTokens = 80;  // up to here two CTAs share an SM

}  // namespace

bool dense_stream_fits(const DenseJob &j) {
    return (j.mode == DG_PLAIN || j.mode == DG_GATED) && !j.a_t && !j.b_t &&
           j.M <= kStreamMaxTokens;
}

rvq_status launch_dense_stream(const DenseJob &job, cudaStream_t stream) {
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(dense_stream_kernel<false>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kRingLarge));
        RVQ_CUDA(cudaFuncSetAttribute(dense_stream_kernel<true>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kRingLarge));
        attr_done[dev] = 1;
    }
    const bool gated = job.mode == DG_GATED;
    StreamArgs g = {};
    g.n = job.M;
    g.rows = job.N;
    g.kb = (job.K + DS_BK - 1) / DS_BK;
    g.npad = (job.M + 15) / 16 * 16;
    const int tile_rows = gated ? DS_ROWS / 2 : DS_ROWS;
    const int tiles = (job.N + tile_rows - 1) / tile_rows;
    const bool small = g.npad <= kSmallTokens;
    const int ring = small ? kRingSmall : kRingLarge;
    const int stage = DS_ABYTES + g.npad * DS_BK * 2;
    g.stages = ring / stage < DS_MAX_ST ? ring / stage : DS_MAX_ST;
    // depth split: as many CTAs as are resident at once, each with two slices
    const int slots = num_sms() * (small ? 2 : 1);
    g.split = 1;
    while (g.split < 8 && tiles * g.split * 2 <= slots && g.kb >= g.split * 4) g.split *= 2;
    g.cols = 32;
    while ((int)g.cols < g.npad) g.cols *= 2;
    const uint32_t fmt = job.dt == RVQ_BF16 ? 1u : 0u;
    g.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(g.npad >> 3) << 17) |
              ((uint32_t)(DS_ROWS >> 4) << 24);
    g.dt = job.dt;
    g.act = job.act;
    g.rdt = job.rdt;
    g.odt = job.odt;
    g.alpha = job.alpha;
    g.residual = job.residual;
    g.ldr = job.ldr;
    g.ldo = job.ldo;
    g.out = job.out[0];
    for (int i = 0; i < 2; ++i) {
        g.bias[i] = job.bias[i];
        g.pre[i] = job.pre[i];
    }
    g.status = job.status;
    CUtensorMap mw[2], mx;
    RVQ_TRY(encode_operand(&mw[0], job.b[0], job.N, job.K, job.ldb, 0, job.dt, tile_rows));
    if (gated)
        RVQ_TRY(encode_operand(&mw[1], job.b[1], job.N, job.K, job.ldb, 0, job.dt, tile_rows));
    else
        mw[1] = mw[0];
    RVQ_TRY(encode_operand(&mx, job.a[0], job.M, job.K, job.lda, 0, job.dt, g.npad));
    // the ring, or the partial tile that takes its place
    const int part = g.n * DS_PITCH * 4, dyn = g.stages * stage > part ? g.stages * stage : part;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * g.split));
    cfg.blockDim = dim3(DS_THREADS);
    cfg.dynamicSmemBytes = (size_t)dyn;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)g.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (gated)
        RVQ_CUDA(cudaLaunchKernelEx(&cfg, dense_stream_kernel<true>, mw[0], mw[1], mx, g));
    else
        RVQ_CUDA(cudaLaunchKernelEx(&cfg, dense_stream_kernel<false>, mw[0], mw[1], mx, g));
    RVQ_LAUNCHED("dense_stream");
    return RVQ_OK;
}

}  // namespace rvq
