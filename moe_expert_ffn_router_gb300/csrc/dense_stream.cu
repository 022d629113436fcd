// The products of the dense operators for few tokens (decode batches) as a stream
// of the weights: moe_linear, moe_gated_linear and the gradients of their inputs.
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
//    190 KB per CTA, or 96 KB where there are enough CTAs for two per SM; one
//    thread issues the MMAs.
//  * For the gradient of the input the weights are read as they lie ([depth][row]),
//    through MN-major descriptors, and the gate's and the up half's products follow
//    one another in depth.
//  * The partial tiles (fp32) go to shared memory, and each CTA of the cluster
//    adds its share of the rows over the cluster in rank order (distributed
//    shared memory): no workspace, no atomics, results repeat bit for bit.
//  * Launched programmatically: while the kernel before it ends, a CTA brings its
//    first slices of weights into L2 (13.4 -> 12.4 us below).
// Every wait is bounded (1 s).
//
// Measured (GB300, weights rotated through more than L2, launches back to back):
// one token through the gated projection 7168 -> 2048 12.4 us (58.7 MB, 4.7 TB/s;
// 8.7 us at the copy rate), 64 tokens 15.6 us; 2048 -> 7168 7.9 and 10.8 us; 512 -> 256
// 3.4 us.  Once the stream runs it moves 7 TB/s; the rest is the first load (1.7 us,
// part of it hidden) and the tail of MMA, cluster barrier and joining (2.5 us).
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
    int n, rows, kb;      // tokens, rows of one matrix, 64-deep slices of a product
    int slices;           // kb, or 2 kb (a sum of two products)
    int w_t;              // weights stored [depth][row]
    int npad;             // tokens padded to a multiple of 16
    int stages, split;    // ring depth; CTAs of a cluster
    int ahead;            // slices prefetched before the kernel may read
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

__device__ __forceinline__ void tma_prefetch(const CUtensorMap *tm, int col, int row) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(col), "r"(row)
                 : "memory");
}

__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}

__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}

// two consecutive elements at an even place
__device__ __forceinline__ void ld2(const void *p, int dt, int64_t i, float (&v)[2]) {
    if (dt == RVQ_F32) {
        const float2 q = *reinterpret_cast<const float2 *>(reinterpret_cast<const float *>(p) + i);
        v[0] = q.x;
        v[1] = q.y;
    } else {
        unpack16(dt, *reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint16_t *>(p) + i),
                 v[0], v[1]);
    }
}

template <bool GATED>
__global__ void __launch_bounds__(DS_THREADS, 2) dense_stream_kernel(
    const __grid_constant__ CUtensorMap mw0, const __grid_constant__ CUtensorMap mw1,
    const __grid_constant__ CUtensorMap mx0, const __grid_constant__ CUtensorMap mx1,
    const __grid_constant__ StreamArgs g) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int TR = GATED ? DS_ROWS / 2 : DS_ROWS;  // rows of one matrix in a tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int tile = blockIdx.x / g.split;
    const int r0 = tile * TR;
    const int k0 = (int)((int64_t)g.slices * rank / g.split);
    const int k1 = (int)((int64_t)g.slices * (rank + 1) / g.split);
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
    if (warp == 0 && elect_one()) {
        // While the kernel before this one ends, bring the first weights into L2
        // (whatever that kernel writes is read coherently after the wait).
        for (int k = k0; k < k1 && k < k0 + g.ahead; ++k) {
            const int kx = (k < g.kb ? k : k - g.kb) * DS_BK;
            const CUtensorMap *mw = k < g.kb ? &mw0 : &mw1;
            if (g.w_t) {
                tma_prefetch(mw, r0, kx);
                tma_prefetch(mw, r0 + 64, kx);
            } else {
                tma_prefetch(mw, kx, r0);
                if (GATED) tma_prefetch(&mw1, kx, r0);
            }
        }
    }
    dependency_wait();
    dependents_may_start();

    if (warp == 0) {
        for (int k = k0, it = 0; k < k1; ++k, ++it) {
            const int s = it % g.stages;
            if (it >= g.stages && !warp_wait(empty0 + 8 * s, ((it / g.stages) - 1) & 1, abort_flag,
                                             g.status))
                break;
            const uint32_t st = smem_u32(smem + s * stage), bar = full0 + 8 * s;
            const int kx = (k < g.kb ? k : k - g.kb) * DS_BK;
            const CUtensorMap *mw = k < g.kb ? &mw0 : &mw1, *mx = k < g.kb ? &mx0 : &mx1;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar, (uint32_t)stage);
                if (g.w_t) {
                    tma_load(st, mw, r0, kx, bar);
                    tma_load(st + 8192, mw, r0 + 64, kx, bar);
                } else {
                    tma_load(st, mw, kx, r0, bar);
                    if (GATED) tma_load(st + DS_ABYTES / 2, &mw1, kx, r0, bar);
                }
                tma_load(st + DS_ABYTES, mx, kx, 0, bar);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        for (int k = k0, it = 0; k < k1; ++k, ++it) {
            const int s = it % g.stages;
            if (!warp_wait(full0 + 8 * s, (it / g.stages) & 1, abort_flag, g.status)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t st = smem_u32(smem + s * stage);
            const uint64_t a = operand_desc(st, g.w_t), b = operand_desc(st + DS_ABYTES, 0);
            const uint32_t da = g.w_t ? 2048u >> 4 : 2u;
            if (elect_one()) {
#pragma unroll
                for (int q = 0; q < DS_BK / 16; ++q)
                    mma_one(tmem, a + q * da, b + 2 * q, g.idesc, (it > 0 || q > 0) ? 1u : 0u);
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
        // two rows per thread, every peer's values requested before the first is
        // added (a loop of load and add cost a round trip per peer: 9000 cycles
        // for 64 tokens)
        const int duos = TR / 2 / g.split;  // groups of two rows this CTA finishes
        for (int i = threadIdx.x; i < g.n * duos; i += DS_THREADS) {
            const int t = i / duos, qr = (rank * duos + i % duos) * 2;
            const int r = r0 + qr;
            const uint32_t at = smem_u32(part + t * DS_PITCH + qr);
            float2 x[8], y[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                if (p >= g.split) continue;
                const uint32_t a = cluster_addr(at, (uint32_t)p);
                x[p] = ld_cluster2(a);
                if (GATED) y[p] = ld_cluster2(a + TR * 4);
            }
            float v[2] = {}, u[2] = {};
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                if (p >= g.split) continue;
                v[0] += x[p].x;
                v[1] += x[p].y;
                if (GATED) {
                    u[0] += y[p].x;
                    u[1] += y[p].y;
                }
            }
            if (r >= g.rows) continue;
            float b[2];
            if (g.bias[0]) {
                ld2(g.bias[0], g.dt, r, b);
                v[0] += b[0];
                v[1] += b[1];
            }
            if (g.pre[0])
                *reinterpret_cast<float2 *>(g.pre[0] + (int64_t)t * g.rows + r) =
                    make_float2(v[0], v[1]);
            act_group(g.act, v);
            if (GATED) {
                if (g.bias[1]) {
                    ld2(g.bias[1], g.dt, r, b);
                    u[0] += b[0];
                    u[1] += b[1];
                }
                if (g.pre[1])
                    *reinterpret_cast<float2 *>(g.pre[1] + (int64_t)t * g.rows + r) =
                        make_float2(u[0], u[1]);
                v[0] *= u[0];
                v[1] *= u[1];
            } else {
                v[0] *= g.alpha;
                v[1] *= g.alpha;
                if (g.residual) {
                    ld2(g.residual, g.rdt, (int64_t)t * g.ldr + r, b);
                    v[0] += b[0];
                    v[1] += b[1];
                }
            }
            const int64_t o = (int64_t)t * g.ldo + r;
            if (g.odt == RVQ_F32)
                *reinterpret_cast<float2 *>(reinterpret_cast<float *>(g.out) + o) =
                    make_float2(v[0], v[1]);
            else
                *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(g.out) + o) =
                    pack16(g.odt, v[0], v[1]);
        }
    }
    cluster_sync();  // the peers' tiles stay in place until read
    if (warp == 2) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.cols));
    }
}

constexpr int kRingSmall = 96 << 10, kRingLarge = 190 << 10;

}  // namespace

int stream_tiles(const DenseJob &j) {
    const int rows = j.mode == DG_GATED ? DS_ROWS / 2 : DS_ROWS;
    return (j.N + rows - 1) / rows;
}

// Up to how many tokens the stream of weights beats the tiled product (measured,
// us, stream / tiled: gated 7168 -> 2048, 192 tokens 20.5 / 21.8, 256 23.9 / 22.2;
// gated 1736 -> 1000, 128 8.7 / 9.9, 192 10.7 / 10.4, which one limit for every gated
// product gives away; plain 2048 -> 7168, 96 12.8 /
// 13.6, 128 14.3 / 13.6; 1736 -> 4104, 128 11.4 / 12.1; 512 -> 2048, 48 4.9 / 5.0,
// 64 5.4 / 5.0; gradient of the input, 7168 x 2048, 1 9.4 / 15.2, 96 15.9 / 15.9).
// 64 tokens is the end for few rows, which are split eightfold up to there (7168 ->
// 512: 64 9.0 / 9.7, 96 14.7 / 10.1).
bool dense_stream_fits(const DenseJob &j) {
    if (j.a_t || j.mode == DG_PAIR_M) return false;
    const int depth = j.mode == DG_SUM_K ? 2 * j.K : j.K;
    const int most = j.mode == DG_GATED ? kStreamMaxTokens : depth >= 1024 ? 112 : 48;
    return j.M <= (stream_tiles(j) * 8 <= num_sms() / 2 && most > 64 ? 64 : most);
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
    g.slices = job.mode == DG_SUM_K ? 2 * g.kb : g.kb;
    g.w_t = job.b_t;
    g.npad = (job.M + 15) / 16 * 16;
    const int tile_rows = gated ? DS_ROWS / 2 : DS_ROWS;
    const int tiles = stream_tiles(job);
    // Depth split: as many CTAs as are resident at once (two per SM up to 128
    // tokens), each with two slices or more.  Past 16 tokens at most four, since
    // the joined tile grows (64 tokens, 7168 -> 2 x 2048: 15.7 us with 128 CTAs
    // of large rings, 18.5 us with 256 of small ones), unless tiles are few and deep
    // (64 tokens, 7168 -> 2048 13.1 us in eight parts, 14.8 in four; 1736 -> 2 x 1000
    // 9.7 and 7.0).  Clusters of eight take small rings: with one CTA per SM a GPC's
    // SMs do not divide by eight.
    const int sms = num_sms(), slots = g.npad <= 128 ? 2 * sms : sms;
    const bool deep = tiles * 4 <= sms / 2 && g.slices >= 64;
    const int most = g.npad <= 16 || (g.npad <= 64 && deep) ? 8 : 4;
    g.split = 1;
    while (g.split < most && tiles * g.split * 2 <= slots && g.slices >= g.split * 4) g.split *= 2;
    const bool two = g.npad <= 128 && (tiles * g.split > sms || g.split == 8);
    const int ring = two ? kRingSmall : kRingLarge;
    const int stage = DS_ABYTES + g.npad * DS_BK * 2;
    g.stages = ring / stage < DS_MAX_ST ? ring / stage : DS_MAX_ST;
    g.ahead = g.stages;
    g.cols = 32;
    while ((int)g.cols < g.npad) g.cols *= 2;
    const uint32_t fmt = job.dt == RVQ_BF16 ? 1u : 0u;
    g.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)job.b_t << 15) |
              ((uint32_t)(g.npad >> 3) << 17) |
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
    CUtensorMap mw[2], mx[2];
    for (int i = 0; i < 2; ++i) {
        if (i == 1 && (job.b[1] == nullptr || job.mode == DG_PLAIN))
            mw[1] = mw[0];
        else
            RVQ_TRY(encode_operand(&mw[i], job.b[i], job.N, job.K, job.ldb, job.b_t, job.dt,
                                   tile_rows));
        if (i == 1 && job.mode != DG_SUM_K)
            mx[1] = mx[0];
        else
            RVQ_TRY(encode_operand(&mx[i], job.a[i], job.M, job.K, job.lda, 0, job.dt, g.npad));
    }
    // the ring, or the partial tile that takes its place
    const int part = g.n * DS_PITCH * 4, dyn = g.stages * stage > part ? g.stages * stage : part;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * g.split));
    cfg.blockDim = dim3(DS_THREADS);
    cfg.dynamicSmemBytes = (size_t)dyn;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)g.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (gated)
        RVQ_CUDA(cudaLaunchKernelEx(&cfg, dense_stream_kernel<true>, mw[0], mw[1], mx[0], mx[1], g));
    else
        RVQ_CUDA(cudaLaunchKernelEx(&cfg, dense_stream_kernel<false>, mw[0], mw[1], mx[0], mx[1], g));
    RVQ_LAUNCHED("dense_stream");
    return RVQ_OK;
}

}  // namespace rvq
