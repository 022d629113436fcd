// Products of microscaled matrices as a stream of the weights past up to 128 tokens at
// a time: moe_mx_linear and moe_mx_gated_linear for decode batches.
//
// Memory-bound: rows x cols weights of half a byte (and a 64th of a byte of scales) are
// read once and a handful of tokens multiplied with each, so the weights are the M
// operand (128 rows of a matrix a tile, whatever the batch) and the tokens the N
// operand, padded to a multiple of 16.
//  * A CTA multiplies 128 rows of the weights (128 gate rows and the 128 up rows
//    beside them for a gated product, two accumulators) with the tokens over one part
//    of the depth; a cluster of up to 8 CTAs splits the depth.
//  * Codes arrive by TMA, one slice a stage, and their scales as plain bulk copies (a
//    tensor map costs the host half a microsecond a call); the issuing thread copies the
//    scales into tensor memory ahead of the slice's MMAs, in order with them.
//  * The partial tiles (fp32) go to shared memory, and the CTAs of the cluster share
//    the outputs, 32 of a token at a time (a block of a microscaled output), adding the
//    parts in rank order: no workspace, no atomics, results repeat bit for bit.
//  * Launched programmatically: while the kernel before it ends, a CTA brings its first
//    slices of weights into L2.
// Every wait is bounded (1 s).
//
// Measured (GB300, weights rotated through more than L2, launches back to back; 8-bit
// tokens and 4-bit weights, two 4-bit operands): one token through the gated projection
// 7168 -> 2048 7.8 and 6.1 us (15.6 MB: 2.3 us at the copy rate), 64 tokens 13.0 and 11.3;
// 2048 -> 7168 with a residual 5.5 and 5.0, 64 tokens 7.8 and 7.1; 512 -> 256 3.2-4.1.
// About 3 us of it are launch, first load and joining; an MMA takes some 130 cycles however
// few the tokens, which is what 8-bit tokens, of twice as many MMAs, cost more.
#include "mx_tc.cuh"

namespace rvq {
namespace {

constexpr int MS_ROWS = 128;
constexpr int MS_TOKENS = 128;
constexpr int MS_THREADS = 256;
constexpr int MS_MAX_ST = 10;
constexpr int MS_ABYTES = MS_ROWS * 128;

struct StreamArgs {
    int n, rows;          // tokens of all tiles, rows of one matrix
    int slices;
    int npad;             // tokens of a tile, padded to a multiple of 16
    int tiles;            // tiles of rows
    int stages, split;    // ring depth; CTAs of a cluster
    int stage;            // bytes of a stage
    uint32_t expect;      // bytes that TMA counts per stage
    const uint8_t *sw[2], *sx;  // scales of the weights, of the tokens
    int ktiles;           // tiles of scales of a row
    uint32_t cols;        // TMEM columns
    uint32_t idesc;
    int act, rdt, odt;
    float alpha;
    const float *bias[2];
    const void *residual;
    int64_t ldr, ldo;
    void *out;
    uint8_t *codes, *scales;
    int ofmt, otiles;
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

// contiguous bytes (16-byte aligned, a multiple of 16)
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(mbar)
        : "memory");
}

__device__ __forceinline__ void bulk_prefetch(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// A slice's KT tiles of scales (tile k KT .. of the row at `row`).  Where a row has an odd
// number of tiles, the last slice's second one, whose codes are zero padding, takes the
// first's scales: finite, or NaN of a row that is NaN already.
template <int KT>
__device__ __forceinline__ void load_scales(uint32_t dst, const uint8_t *row, int k, int ktiles,
                                            uint32_t mbar) {
    const uint8_t *src = row + (int64_t)k * KT * kMxTileBytes;
    if (KT == 1 || k * KT + 1 < ktiles) {
        bulk_load(dst, src, KT * kMxTileBytes, mbar);
    } else {
        bulk_load(dst, src, kMxTileBytes, mbar);
        bulk_load(dst + kMxTileBytes, src, kMxTileBytes, mbar);
    }
}

__device__ __forceinline__ void tma_prefetch(const CUtensorMap *tm, int col, int row) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(col), "r"(row)
                 : "memory");
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

// Two columns (c, c + 1) of token t per lane, 16 lanes a block of 32: into the
// microscaled output.
template <int FMT>
__device__ __forceinline__ void put_block(const StreamArgs &g, int t, int c, const float (&v)[2]) {
    uint32_t top = max(__float_as_uint(v[0]) & 0x7FFFFFFFu, __float_as_uint(v[1]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < 16; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t byte = mx_byte<FMT>(top);
    const float inv = mx_inverse(byte);
    const float a = byte == 255 ? 0.f : v[0] * inv, b = byte == 255 ? 0.f : v[1] * inv;
    if (t >= g.n) return;
    const int64_t at = (int64_t)t * g.otiles * kMxTile + c;
    if (FMT == MOE_MX_F8) {
        *reinterpret_cast<uint16_t *>(g.codes + at) = (uint16_t)e4m3x4(a, b, 0.f, 0.f);
    } else {
        const float q[8] = {a, b, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        g.codes[at / 2] = (uint8_t)e2m1x8(q);
    }
    if ((threadIdx.x & 15) == 0)
        g.scales[mx_scale_at(t, c / kMxTile, g.otiles) + (c / kMxBlock & 3)] = (uint8_t)byte;
}

// Outputs of units first, first + step, .. of `units`: sums of the cluster's parts in rank
// order, finished and written.
template <bool GATED, int SPLIT>
__device__ __forceinline__ void join(const StreamArgs &g, const float *part, int units, int first,
                                     int step, int r0, int t0) {
    constexpr int MATS = GATED ? 2 : 1, AT_ONCE = 8 / SPLIT / MATS < 1 ? 1 : 8 / SPLIT / MATS;
    constexpr int PITCH = MATS * MS_ROWS + 4;
    for (int base = first & ~1; base < units; base += AT_ONCE * step) {
        float2 x[AT_ONCE][SPLIT], y[AT_ONCE][SPLIT];
        float b[AT_ONCE][2];
        int r[AT_ONCE], tok[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const int u = base + (first & 1) + i * step;
            const bool in = u < units;
            const int t = in ? u >> 2 : 0, qr = (u & 3) * 32 + (int)(threadIdx.x & 15) * 2;
            r[i] = r0 + qr;
            tok[i] = in ? t0 + t : g.n;
            const uint32_t at = smem_u32(part + t * PITCH + qr);
#pragma unroll
            for (int p = 0; p < SPLIT; ++p) {
                const uint32_t a = cluster_addr(at, (uint32_t)p);
                x[i][p] = ld_cluster2(a);
                if (GATED) y[i][p] = ld_cluster2(a + MS_ROWS * 4);
            }
            b[i][0] = b[i][1] = 0.f;
            if (!GATED && g.residual && in && r[i] < g.rows)
                ld2(g.residual, g.rdt, (int64_t)tok[i] * g.ldr + r[i], b[i]);
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            float v[2] = {}, w[2] = {};
#pragma unroll
            for (int p = 0; p < SPLIT; ++p) {
                v[0] += x[i][p].x;
                v[1] += x[i][p].y;
                if (GATED) {
                    w[0] += y[i][p].x;
                    w[1] += y[i][p].y;
                }
            }
            const bool real = tok[i] < g.n && r[i] < g.rows;
            if (g.bias[0] && real) {
                v[0] += g.bias[0][r[i]];
                v[1] += g.bias[0][r[i] + 1];
            }
            act_group(g.act, v);
            if (GATED) {
                if (g.bias[1] && real) {
                    w[0] += g.bias[1][r[i]];
                    w[1] += g.bias[1][r[i] + 1];
                }
                v[0] *= w[0];
                v[1] *= w[1];
            } else {
                v[0] = g.alpha * v[0] + b[i][0];
                v[1] = g.alpha * v[1] + b[i][1];
            }
            if (GATED && g.codes) {
                if (!real) v[0] = v[1] = 0.f;  // padded columns
                if (g.ofmt == MOE_MX_F8)
                    put_block<MOE_MX_F8>(g, tok[i], r[i], v);
                else
                    put_block<MOE_MX_F4>(g, tok[i], r[i], v);
                continue;
            }
            if (!real) continue;
            const int64_t o = (int64_t)tok[i] * g.ldo + r[i];
            if (g.odt == RVQ_F32)
                *reinterpret_cast<float2 *>(reinterpret_cast<float *>(g.out) + o) =
                    make_float2(v[0], v[1]);
            else
                *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(g.out) + o) =
                    pack16(g.odt, v[0], v[1]);
        }
    }
}

template <bool GATED, bool F4>
__global__ void __launch_bounds__(MS_THREADS, 2) mx_stream_kernel(
    const __grid_constant__ CUtensorMap mw0, const __grid_constant__ CUtensorMap mw1,
    const __grid_constant__ CUtensorMap mx, const __grid_constant__ StreamArgs g) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int MATS = GATED ? 2 : 1;
    constexpr int KT = F4 ? 2 : 1;                     // tiles of scales a slice is deep
    constexpr int PITCH = MATS * MS_ROWS + 4;          // floats between tokens of a partial tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int tile = blockIdx.x / g.split;
    const int row_tile = tile % g.tiles, r0 = row_tile * MS_ROWS;
    const int tok_tile = tile / g.tiles, t0 = tok_tile * MS_TOKENS;
    const int k0 = (int)((int64_t)g.slices * rank / g.split);
    const int k1 = (int)((int64_t)g.slices * (rank + 1) / g.split);
    // a stage: codes of the weights, of the tokens, scales of the weights, of the tokens
    const int b_at = MATS * MS_ABYTES, sw_at = b_at + g.npad * 128, sx_at = sw_at + MATS * KT * kMxTileBytes;
    const int64_t srow = (int64_t)g.ktiles * kMxTileBytes;  // scales of 128 rows
    const uint8_t *sw0 = g.sw[0] + row_tile * srow, *sw1 = GATED ? g.sw[1] + row_tile * srow : nullptr;
    const uint8_t *sx = g.sx + tok_tile * srow;
    __shared__ __align__(8) uint64_t bars[2 * MS_MAX_ST + 1];
    __shared__ uint32_t tslot;
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * MS_MAX_ST,
                   accfull = empty0 + 8 * MS_MAX_ST;
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
        // an SM holds at most two such CTAs, 256 columns each, or one
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
        for (int k = k0; k < k1 && k < k0 + g.stages; ++k) {
            tma_prefetch(&mw0, k * 128, r0);
            if (GATED) tma_prefetch(&mw1, k * 128, r0);
        }
        const int first = k0 * KT, last = min(min(k1, k0 + g.stages) * KT, g.ktiles);
        const uint32_t bytes = (uint32_t)(last - first) * kMxTileBytes;
        bulk_prefetch(sw0 + (int64_t)first * kMxTileBytes, bytes);
        if (GATED) bulk_prefetch(sw1 + (int64_t)first * kMxTileBytes, bytes);
    }
    dependency_wait();
    dependents_may_start();

    if (warp == 0) {
        for (int k = k0, it = 0; k < k1; ++k, ++it) {
            const int s = it % g.stages;
            if (it >= g.stages && !warp_wait(empty0 + 8 * s, ((it / g.stages) - 1) & 1, abort_flag,
                                             g.status))
                break;
            const uint32_t st = smem_u32(smem + s * g.stage), bar = full0 + 8 * s;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar, g.expect);
                tma_load(st, &mw0, k * 128, r0, bar);
                load_scales<KT>(st + sw_at, sw0, k, g.ktiles, bar);
                if (GATED) {
                    tma_load(st + MS_ABYTES, &mw1, k * 128, r0, bar);
                    load_scales<KT>(st + sw_at + KT * kMxTileBytes, sw1, k, g.ktiles, bar);
                }
                tma_load(st + b_at, &mx, k * 128, t0, bar);
                load_scales<KT>(st + sx_at, sx, k, g.ktiles, bar);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        const uint32_t tsw = tmem + (uint32_t)(MATS * g.npad), tsx = tsw + MATS * KT * 4;
        for (int k = k0, it = 0; k < k1; ++k, ++it) {
            const int s = it % g.stages;
            if (!warp_wait(full0 + 8 * s, (it / g.stages) & 1, abort_flag, g.status)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t st = smem_u32(smem + s * g.stage);
            const uint64_t b = smem_desc(st + b_at);
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < MATS * KT; ++i)
                    copy_scales<1>(tsw + 4 * i, st + sw_at + i * kMxTileBytes);
#pragma unroll
                for (int i = 0; i < KT; ++i) copy_scales<1>(tsx + 4 * i, st + sx_at + i * kMxTileBytes);
#pragma unroll
                for (int m = 0; m < MATS; ++m) {
                    const uint64_t a = smem_desc(st + m * MS_ABYTES);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int kt = F4 ? q >> 1 : 0;
                        mx_mma<1, F4>(tmem + m * g.npad, a + 2 * q, b + 2 * q,
                                      g.idesc | scale_places(F4 ? 2 * (q & 1) : q),
                                      tsw + (m * KT + kt) * 4, tsx + kt * 4,
                                      (it > 0 || q > 0) ? 1u : 0u);
                    }
                }
                mma_commit(empty0 + 8 * s);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(accfull);
        __syncwarp();
    } else if (!GATED && g.residual) {
        // the residual of this CTA's outputs into L2 meanwhile: a row's 128 columns are
        // four (16-bit: two) lines of 128 bytes
        const int e = g.rdt == RVQ_F32 ? 4 : 2, lines = e;
        const int tokens = min(g.n - t0, g.npad);
        for (int i = (int)threadIdx.x - 64 + rank * (MS_THREADS - 64); i < tokens * lines;
             i += g.split * (MS_THREADS - 64)) {
            const int c = r0 + i % lines * (128 / e);
            if (c < g.rows)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(
                    reinterpret_cast<const char *>(g.residual) +
                    ((int64_t)(t0 + i / lines) * g.ldr + c) * e));
        }
    }
    // the partial tile, [token][row], over the ring (its last slice is consumed)
    warp_wait(accfull, 0, abort_flag, g.status);
    __syncthreads();
    const bool ok = !*abort_flag;  // no wait of this CTA is left that could raise it
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const int nt = min(g.n - t0, g.npad);
    float *part = reinterpret_cast<float *>(smem);
    if (ok) {
        const int q = warp & 3;
#pragma unroll
        for (int m = 0; m < MATS; ++m)
            for (int c = (warp >> 2) * 16; c < g.npad; c += 32) {
                uint32_t r[16];
                tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(m * g.npad + c), r);
                tmem_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (c + e < nt)
                        part[(c + e) * PITCH + m * MS_ROWS + 32 * q + lane] = __uint_as_float(r[e]);
            }
    }
    __syncthreads();
    if (*abort_flag) {
        // copies and MMAs still in flight end well within this time
        const unsigned long long w0 = global_ns();
        while (global_ns() - w0 < 2000000ull) __nanosleep(1000);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();  // every partial tile of the cluster is in place
    if (ok) {
        // blocks of 32 outputs of a token, dealt over the cluster's half warps; two
        // outputs per lane, and as many blocks at once as make eight loads from the
        // peers (a block at a time cost a round trip each: 64 tokens 6 us more than
        // one).  Whole warps go through the loop together (the shuffles of put_block).
        const int units = nt * 4, step = g.split * (MS_THREADS / 16);
        const int first = rank * (MS_THREADS / 16) + (int)(threadIdx.x >> 4);
        if (g.split == 8)
            join<GATED, 8>(g, part, units, first, step, r0, t0);
        else if (g.split == 4)
            join<GATED, 4>(g, part, units, first, step, r0, t0);
        else if (g.split == 2)
            join<GATED, 2>(g, part, units, first, step, r0, t0);
        else
            join<GATED, 1>(g, part, units, first, step, r0, t0);
    }
    cluster_sync();  // the peers' tiles stay in place until read
    if (warp == 2) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(g.cols));
    }
}

// of one CTA where two share an SM, and of one alone
constexpr int kRingSmall = 111 << 10, kRingLarge = 200 << 10;
// the most that two CTAs of an SM have each: half its 228 KB, less 1 KB that every block
// takes and 1 KB for the barriers
constexpr int kHalfSm = 112 << 10;
static_assert(kRingSmall <= kHalfSm, "two rings on an SM");

// Clusters of `split` CTAs that the device holds at once with one CTA per SM (the query
// does not count a second one per SM; it gives 15 clusters of eight, 36 of four).
template <bool GATED, bool F4>
int resident_clusters(int split) {
    static std::atomic<int> cached[64][4];  // per device and split, plus one
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
    std::atomic<int> &known = cached[dev][split == 8 ? 3 : split == 4 ? 2 : split - 1];
    if (known) return known - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms() / split * split));
    cfg.blockDim = dim3(MS_THREADS);
    cfg.dynamicSmemBytes = kRingLarge;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(mx_stream_kernel<GATED, F4>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kRingLarge) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, mx_stream_kernel<GATED, F4>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();  // not the caller's error: the depth stays whole
        n = 0;
    }
    known = n + 1;
    return n;
}

// Tokens of a tile, padded to a multiple of 16; bytes of a stage; of the partial tile that
// takes the ring's place; TMEM columns.
struct Shape {
    int npad, stage, part;
    uint32_t cols;
};
template <bool GATED, bool F4>
Shape shape_of(const MxJob &job) {
    constexpr int MATS = GATED ? 2 : 1, KT = F4 ? 2 : 1;
    Shape s;
    const int tokens = job.n < MS_TOKENS ? job.n : MS_TOKENS;
    s.npad = (tokens + 15) / 16 * 16;
    s.part = tokens * (MATS * MS_ROWS + 4) * 4;
    s.stage = (MATS * MS_ABYTES + s.npad * 128 + (MATS + 1) * KT * kMxTileBytes + 1023) / 1024 * 1024;
    s.cols = 32;
    while ((int)s.cols < MATS * s.npad + (MATS + 1) * KT * 4) s.cols *= 2;
    return s;
}

// Two CTAs per SM where both fit (a ring of two stages or more, the partial tile and 256
// columns of tensor memory each), and the depth split among as many CTAs, up to eight, as
// leaves every cluster resident at once, with two slices or more each.  One token, gated
// 7168 -> 2048, 16 tiles of 4-bit weights: eight CTAs each 7.7 us, four 9.7; with the
// large ring, where a sixteenth cluster of eight waits for the others, 13.7; 2048 ->
// 7168, 56 tiles: four 5.5, eight 9.5, two 6.5.  112 tokens, whose partial tiles do not fit
// an SM twice: planned as if they did 24.7, alone 13.9 (110, two to an SM, 16.9).
template <bool GATED, bool F4>
MxStreamPlan plan_of(const MxJob &job, const Shape &s) {
    MxStreamPlan p;
    p.slices = F4 ? (mx_tiles(job.cols) + 1) / 2 : mx_tiles(job.cols);
    p.tiles = (long long)mx_tiles(job.rows) * ((job.n + MS_TOKENS - 1) / MS_TOKENS);
    p.two = s.cols <= 256 && 2 * s.stage <= kRingSmall && s.part <= kHalfSm;
    p.split = 8;
    while (p.split > 1 && (p.slices < 2 * p.split ||
                           p.tiles > (p.two ? 2 : 1) * resident_clusters<GATED, F4>(p.split)))
        p.split /= 2;
    return p;
}

template <bool GATED, bool F4>
rvq_status launch(const MxJob &job, cudaStream_t stream) {
    constexpr int MATS = GATED ? 2 : 1, KT = F4 ? 2 : 1;
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(mx_stream_kernel<GATED, F4>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kRingLarge));
        attr_done[dev] = 1;
    }
    const Shape s = shape_of<GATED, F4>(job);
    const MxStreamPlan plan = plan_of<GATED, F4>(job, s);
    if (plan.tiles > 0x7fffffff / 8) {
        set_error("microscaled product: %lld tiles", plan.tiles);
        return RVQ_ENOTIMPL;
    }
    StreamArgs g = {};
    g.n = job.n;
    g.rows = job.rows;
    g.slices = plan.slices;
    g.npad = s.npad;
    g.tiles = mx_tiles(job.rows);
    g.cols = s.cols;
    g.stage = s.stage;
    g.split = plan.split;
    const int ring = plan.two ? kRingSmall : kRingLarge;
    g.stages = ring / g.stage < MS_MAX_ST ? ring / g.stage : MS_MAX_ST;
    g.expect = MATS * slice_bytes(F4, job.wfmt, MS_ROWS) + slice_bytes(F4, job.xfmt, g.npad) +
               (MATS + 1) * KT * kMxTileBytes;
    g.idesc = mx_idesc(F4, job.wfmt, job.xfmt, MS_ROWS, g.npad);
    g.act = job.act;
    g.rdt = job.rdt;
    g.odt = job.odt;
    g.alpha = job.alpha;
    g.residual = job.residual;
    g.ldr = job.ldr;
    g.ldo = job.ldo;
    g.out = job.out;
    g.bias[0] = job.bias[0];
    g.bias[1] = job.bias[1];
    g.codes = job.codes;
    g.scales = job.scales;
    g.ofmt = job.ofmt;
    g.otiles = mx_tiles(job.rows);
    g.status = job.status;
    CUtensorMap mw[2], mx;
    for (int i = 0; i < MATS; ++i) {
        RVQ_TRY(encode_codes(&mw[i], job.w[i], job.rows, job.cols, job.wfmt, F4, MS_ROWS));
        g.sw[i] = job.ws[i];
    }
    if (!GATED) mw[1] = mw[0];
    RVQ_TRY(encode_codes(&mx, job.x, job.n, job.cols, job.xfmt, F4, g.npad));
    g.sx = job.xs;
    g.ktiles = mx_tiles(job.cols);
    // the ring, or the partial tile that takes its place
    const int dyn = g.stages * g.stage > s.part ? g.stages * g.stage : s.part;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(plan.tiles * g.split));
    cfg.blockDim = dim3(MS_THREADS);
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
    RVQ_CUDA(cudaLaunchKernelEx(&cfg, mx_stream_kernel<GATED, F4>, mw[0], mw[1], mx, g));
    RVQ_LAUNCHED("mx_stream");
    return RVQ_OK;
}

}  // namespace

MxStreamPlan plan_mx_stream(const MxJob &job) {
    if (job.mats == 2)
        return job.f4() ? plan_of<true, true>(job, shape_of<true, true>(job))
                        : plan_of<true, false>(job, shape_of<true, false>(job));
    return job.f4() ? plan_of<false, true>(job, shape_of<false, true>(job))
                    : plan_of<false, false>(job, shape_of<false, false>(job));
}

rvq_status launch_mx_stream(const MxJob &job, cudaStream_t stream) {
    if (job.mats == 2)
        return job.f4() ? launch<true, true>(job, stream) : launch<true, false>(job, stream);
    return job.f4() ? launch<false, true>(job, stream) : launch<false, false>(job, stream);
}

}  // namespace rvq
