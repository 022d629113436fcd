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
//    of 16-bit elements), six 32 KB stages per CTA (more of a narrower tile); the
//    slices of both CTAs complete on the leader's barrier.
//  * A transposed operand (stored [K][rows]) is loaded as it lies, in boxes of
//    64 rows x 64 deep, and read through MN-major descriptors, so the gradients
//    need no transposed copies.
//  * Accumulators are fp32 in tensor memory, two of up to 256 columns: eight
//    warps per CTA write one tile out while the next one is multiplied.
//  * A gated product loads its gate half from B0 (leader) and its up half from
//    B1 (follower), so both projections of an output lie in one accumulator row
//    and act(g) * u is formed in registers.
//  * Outputs are turned from a row per lane into rows of 64 or 128 contiguous
//    bytes through 4 KB of staging per warp; biases are staged once per tile.
//  * A tile of too few for half the pairs is split among the two or four pairs of a
//    cluster, which multiply a run of its slices each and exchange the sums through
//    distributed shared memory (512 x 2048 x 2048 13.7 -> 11.8 us, 250 x 856 x 1240
//    10.4 -> 8.1), or, where the depth is long, cut by slices into parts, which a
//    second launch adds in order (512 tokens, gated 7168 -> 2048 27.7 us, split 30.5).
//    The products of dx and dw share a launch where their tiles fill the pairs better
//    together.  (Tiles of 256 columns are not split: what the pairs send takes a third
//    of the ring, 256 x 7168 x 2048 14.9 -> 17.5 us.)
// Rows, columns and depth past the ends are zero-filled by TMA and not stored.
// Each output is rounded once, from fp32.  Every wait is bounded (1 s).
//
// Measured (GB300, operands rotated through more than L2): 2048 tokens through
// the gated projection 7168 -> 2048 70.5 us (1.70 PFLOP/s; 80 us in a loop of half
// a second, where the power cap holds a library product of the same size at
// 74-77), 4096^2 x 8192 154 us (1.79).  A slice of a 256-wide tile takes 528 cycles
// against 512 of its MMAs; a narrower one is bound by the operand fill (about 55
// bytes per cycle and SM) and the issue.  Around the slices a tile costs 2200
// cycles to its first operands and, at the end, 4800 for the outputs, when all
// SMs write at once.
#include "dense_epilogue.cuh"
#include "dense_tc.cuh"

#include <cudaTypedefs.h>
#include <math.h>

namespace rvq {
namespace {

constexpr int DG_BM = 128;   // rows of A per CTA
constexpr int DG_BK = 64;    // depth of a slice
constexpr int DG_ABYTES = DG_BM * DG_BK * 2;
constexpr int DG_MAX_ST = 9;  // stages: as many as fit
constexpr int DG_RING = 192 << 10;
constexpr int DG_EPI_WARPS = 8;
constexpr int DG_TURN = 4096;  // staging of an epilogue warp: 32 rows x 32 fp32 columns
constexpr int DG_BIAS = DG_RING + DG_EPI_WARPS * DG_TURN;  // of two tiles, fp32
constexpr int DG_BARS = DG_BIAS + 2 * 256 * 4;
constexpr int DG_SMEM = DG_BARS + 256;
constexpr int kSumsMax = 48 << 10;        // of the ring, for sums of a split tile
constexpr int DG_THREADS = 32 * (4 + DG_EPI_WARPS);
constexpr int DG_ACC = 256;  // TMEM columns per accumulator
constexpr int DG_GROUP = 8;  // M tiles walked together (operand reuse in L2)
static_assert(DG_SMEM <= 232448, "shared memory of a CTA");

struct GemmArgs {
    int mode, M, N, a_t, b_t;
    int kb;              // slices of one product
    int slices;          // slices of a tile
    int tile_n, half;    // columns of an accumulator; rows of B per CTA
    int stages, stage;   // ring depth; bytes of a stage (A, then B)
    int mt, nt;          // output tiles (M tiles of both problems for PAIR_M)
    int parts;           // runs of slices that a tile is cut into (1: whole tiles)
    uint32_t idesc;
    int dt, act, rdt, odt;
    float alpha;
    const void *bias[2], *residual;
    int64_t ldr, ldo;
    void *out[2];
    float *pre[2];
    float *partial;      // sums of the parts, [part][plane][M][N] (see plane_of)
    uint32_t *status;
};

// One product, or two for one launch (the gradients dx and dw, whose tiles alone
// leave CTA pairs idle), with the tensor maps of their operands.
template <int JOBS>
struct GemmParams {
    CUtensorMap a[JOBS][2], b[JOBS][2];
    GemmArgs g[JOBS];
    int bonus;           // see Work
    int split;           // pairs that share a unit's slices (a cluster), or 1
    BiasSums sums;       // added beside the products
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
__device__ __forceinline__ void commit_pair(uint32_t mbar, uint32_t lead) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(mbar),
        "h"((uint16_t)(3u << lead))
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

// The work of a CTA pair, the same sequence in every role: units of one tile and
// one run of its slices, every `pairs`-th unit of the first product, then units of
// the second.  Pairs that got one unit less of the first (those from U0 mod pairs
// on) first take `bonus` units of the second alone, as many as that one lasts, so
// that all pairs end together.
// With SPLIT a cluster of `split` pairs has one unit, and pair `part` of it a run of
// its slices.
template <int JOBS, bool SPLIT>
struct Work {
    int pair, pairs, unit, round;
    int job, m, n, part, k0, k1;

    __device__ __forceinline__ Work(int pair_, int pairs_)
        : pair(pair_), pairs(pairs_), unit(pair_), round(0), job(0) {}
    __device__ __forceinline__ bool next(const GemmParams<JOBS> &p) {
        int u;
        if (SPLIT) {
            if (round++) return false;
            u = pair / p.split;
            part = pair - u * p.split;
            const int units = p.g[0].mt * p.g[0].nt;
            if (JOBS > 1 && u >= units) {
                job = 1;
                u -= units;
            }
            const GemmArgs &g = p.g[JOBS == 1 ? 0 : job];
            tile_at(g, u, m, n);
            k0 = (int)((int64_t)g.slices * part / p.split);
            k1 = (int)((int64_t)g.slices * (part + 1) / p.split);
            return true;
        }
        if (job == 0) {
            const int units = p.g[0].mt * p.g[0].nt * p.g[0].parts;
            u = unit;
            unit += pairs;
            if (u >= units) {
                if (JOBS == 1) return false;
                job = 1;
            }
        }
        if (JOBS > 1 && job == 1) {
            const int units = p.g[JOBS - 1].mt * p.g[JOBS - 1].nt;
            const int first = p.g[0].mt * p.g[0].nt % pairs, early = pairs - first;
            const int e = pair - first;
            if (round < p.bonus && e >= 0) {
                u = round * early + e;
            } else {
                if (round < p.bonus) round = p.bonus;
                u = p.bonus * early + (round - p.bonus) * pairs + (e >= 0 ? e : e + pairs);
            }
            ++round;
            if (u >= units) return false;
        }
        const GemmArgs &g = p.g[JOBS == 1 ? 0 : job];
        const int tiles = g.mt * g.nt;
        part = u / tiles;
        tile_at(g, u - part * tiles, m, n);
        k0 = (int)((int64_t)g.slices * part / g.parts);
        k1 = (int)((int64_t)g.slices * (part + 1) / g.parts);
        return true;
    }
};

// fp32 [M][N] of a part: the gate or the up half, or the first or second problem
__device__ __forceinline__ float *plane_of(const GemmArgs &g, int part, int z) {
    const int planes = g.mode == DG_GATED || g.mode == DG_PAIR_M ? 2 : 1;
    return g.partial + ((int64_t)part * planes + z) * g.M * g.N;
}

// adds 32 staged bias values (byte address `at`; the same for every lane)
__device__ __forceinline__ void add_bias32(uint32_t at, float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float b[4];
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3])
                     : "r"(at + 16 * j)
                     : "memory");
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * j + e] += b[e];
    }
}

// 32 columns of a row per lane, finished and written: v (and w, the up half) are
// the sums of columns c .. c + width - 1 of rows row .. row + 31.
template <bool GATED>
__device__ __forceinline__ void finish(const GemmArgs &g, uint32_t turn, int lane, void *out, int row,
                                       int c, int width, float (&v)[32], float (&w)[32],
                                       const Residual &res, uint32_t bias) {
    if (g.bias[0]) add_bias32(bias, v);
    if (g.pre[0]) {
        turn_in(turn, lane, v);
        turn_rows(turn, lane, g.pre[0], RVQ_F32, g.N, row, g.M, c, width, nullptr, 0);
    }
    if (g.act != MOE_ACT_NONE) act_group(g.act, v);
    if (GATED) {
        if (g.bias[1]) add_bias32(bias + g.half * 4, w);
        if (g.pre[1]) {
            turn_in(turn, lane, w);
            turn_rows(turn, lane, g.pre[1], RVQ_F32, g.N, row, g.M, c, width, nullptr, 0);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= w[e];
    } else if (g.alpha != 1.f) {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= g.alpha;
    }
    if (g.odt != RVQ_F32 && g.residual == nullptr) {
        rows_16_plain(turn, lane, out, g.odt, g.ldo, row, g.M, c, width, v);
        return;
    }
    turn_in(turn, lane, v);
    turn_rows(turn, lane, out, g.odt, g.ldo, row, g.M, c, width, g.residual ? &res : nullptr, g.rdt);
}

// Bytes that a CTA receives from the other pairs of its cluster, at the end of the
// ring: per sender and group of 32 columns that it finishes, 128 rows (twice for a
// gated product).
__host__ __device__ __forceinline__ int sums_bytes(int split, int per, bool gated) {
    const int groups = (per + 31) / 32;
    return (split - 1) * ((groups + split - 1) / split) * (gated ? 2 : 1) * 4 * DG_TURN;
}

template <bool GATED>
__device__ __forceinline__ uint32_t sums_at(const uint8_t *smem, int split, int per, int from,
                                            int to, int c, int q) {
    const int groups = ((per + 31) / 32 + split - 1) / split;
    const int block = (from < to ? from : from - 1) * groups + (c >> 5) / split;
    return smem_u32(smem + DG_RING - sums_bytes(split, per, GATED)) +
           (uint32_t)((block * (GATED ? 2 : 1) * 4 + q) * DG_TURN);
}

// Sums of a split tile on their way between the pairs of a cluster: 32 columns of 32
// rows, 16 bytes per lane and access (contiguous for a warp, both ways).
__device__ __forceinline__ void send32(uint32_t addr, int lane, const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr + j * 512 +
                                                                               lane * 16),
                     "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]), "f"(v[4 * j + 3])
                     : "memory");
}

__device__ __forceinline__ void add_sent32(uint32_t addr, int lane, float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float b[4];
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3])
                     : "r"(addr + j * 512 + lane * 16)
                     : "memory");
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * j + e] += b[e];
    }
}

template <bool GATED, int JOBS, bool SPLIT>
__global__ void __launch_bounds__(DG_THREADS, 1) dense_gemm_kernel(
    const __grid_constant__ GemmParams<JOBS> params) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank() & 1u, lead = cluster_rank() & ~1u;
    Work<JOBS, SPLIT> work(blockIdx.x >> 1, gridDim.x >> 1);
    const int stages = params.g[0].stages, stage = params.g[0].stage;  // of both products
    uint32_t *status = params.g[0].status;
    uint8_t *bars = smem + DG_BARS;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * DG_MAX_ST,
                   accfull0 = empty0 + 8 * DG_MAX_ST, accempty0 = accfull0 + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 8 * (2 * DG_MAX_ST + 4));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
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
        // one CTA per SM (shared memory): the allocation waits for nothing but
        // the end of a kernel before this one
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
    dependency_wait();

    const int q = warp & 3, par = (warp - 4) >> 2;  // of an epilogue warp
    const uint32_t turn = smem_u32(smem + DG_RING) + (uint32_t)(warp - 4) * DG_TURN;
    bool sent = false;
    if (warp == 0) {
        // producer: this CTA's rows of A and of B for every slice
        int s = 0;
        uint32_t lap = 0;  // trips around the ring
        bool ok = true;
        while (ok && work.next(params)) {
            const GemmArgs &g = params.g[JOBS == 1 ? 0 : work.job];
            const CUtensorMap *ma = params.a[JOBS == 1 ? 0 : work.job];
            const CUtensorMap *mb = params.b[JOBS == 1 ? 0 : work.job];
            const uint32_t bytes = DG_ABYTES + g.half * 128;
            const int mt1 = g.mode == DG_PAIR_M ? g.mt / 2 : g.mt;  // M tiles of one problem
            const bool second = work.m >= mt1;
            const int m0 = (second ? work.m - mt1 : work.m) * 2 * DG_BM + (int)rank * DG_BM;
            const int n0 = GATED ? work.n * g.half : work.n * g.tile_n + (int)rank * g.half;
            for (int k = work.k0; k < work.k1; ++k) {
                if (lap > 0 && !warp_wait(empty0 + 8 * s, (lap - 1) & 1, abort_flag, status)) {
                    ok = false;
                    break;
                }
                const bool k2 = k >= g.kb;
                const int kx = (k2 ? k - g.kb : k) * DG_BK;
                const CUtensorMap *ta = ma + ((second || k2) ? 1 : 0);
                const CUtensorMap *tb = mb + ((GATED ? rank == 1 : k2) ? 1 : 0);
                const uint32_t st = smem_u32(smem + s * stage), sb = st + DG_ABYTES;
                const uint32_t bar = cluster_addr(full0 + 8 * s, lead);
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
                        if (g.half > 64) tma_pair(sb + 8192, tb, n0 + 64, kx, bar);
                    } else {
                        tma_pair(sb, tb, kx, n0, bar);
                    }
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ++lap;
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        // issuer: four 16-deep MMAs per slice
        int s = 0, done = 0;
        uint32_t lap = 0;
        bool ok = true;
        for (; ok && work.next(params); ++done) {
            const GemmArgs &g = params.g[JOBS == 1 ? 0 : work.job];
            const uint32_t da = g.a_t ? 2048u >> 4 : 2u, db = g.b_t ? 2048u >> 4 : 2u;
            const int a_t = g.a_t, b_t = g.b_t;
            const uint32_t idesc = g.idesc;
            const int buf = done & 1;
            if (done >= 2 && !warp_wait(accempty0 + 8 * buf, ((done >> 1) - 1) & 1, abort_flag,
                                        status))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + (uint32_t)(buf * DG_ACC);
            for (int k = work.k0; k < work.k1; ++k) {
                if (!warp_wait(full0 + 8 * s, lap & 1, abort_flag, status)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t st = smem_u32(smem + s * stage);
                const uint64_t a = operand_desc(st, a_t),
                               b = operand_desc(st + DG_ABYTES, b_t);
                if (elect_one()) {
#pragma unroll
                    for (int q = 0; q < DG_BK / 16; ++q)
                        mma_pair(acc, a + q * da, b + q * db, idesc,
                                 (k > work.k0 || q > 0) ? 1u : 0u);
                    commit_pair(empty0 + 8 * s, lead);
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ++lap;
                }
            }
            if (elect_one()) commit_pair(accfull0 + 8 * buf, lead);
            __syncwarp();
        }
    } else if (warp == 2 || warp == 3) {
        if (!GATED && params.sums.wanted())
            add_bias_sums(params.sums, (int)blockIdx.x * 2 + warp - 2, (int)gridDim.x * 2, lane);
    } else if (warp >= 4) {
        // epilogue: lanes 32 q .. 32 q + 31 of the accumulator, every other
        // group of 32 columns
        for (int done = 0; work.next(params); ++done) {
            const GemmArgs &g = params.g[JOBS == 1 ? 0 : work.job];
            const int per = GATED ? g.half : g.tile_n;  // outputs of a tile's row
            const int mt1 = g.mode == DG_PAIR_M ? g.mt / 2 : g.mt;
            const bool second = work.m >= mt1;
            const int row =
                (second ? work.m - mt1 : work.m) * 2 * DG_BM + (int)rank * DG_BM + 32 * q;
            const int buf = done & 1;
            if (!GATED && g.residual && g.parts == 1 && row + lane < g.M) {
                // this warp's part of the residual into L2 while the tile is multiplied
                const int e = g.rdt == RVQ_F32 ? 4 : 2;
                for (int c = par * 32; c < per && work.n * per + c < g.N; c += 64)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(
                        reinterpret_cast<const char *>(g.residual) +
                        ((int64_t)(row + lane) * g.ldr + work.n * per + c) * e));
            }
            // the tile's biases: each warp brings the columns it will read itself
            // (before the wait) and stages them after it, when no warp still reads
            // those of the tile before the last
            constexpr int CH = GATED ? 2 : 4;  // its groups of 32 columns, at most
            float bias[GATED ? 2 : 1][CH];
            const bool biased = g.parts == 1 && (g.bias[0] || g.bias[1]);
            if (biased) {
#pragma unroll
                for (int z = 0; z < (GATED ? 2 : 1); ++z)
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const int c = (2 * i + par) * 32 + lane, col = work.n * per + c;
                        bias[z][i] = g.bias[z] && c < per && col < g.N
                                         ? ld_elem(g.bias[z], g.dt, col) : 0.f;
                    }
            }
            if (!warp_wait(accfull0 + 8 * buf, (done >> 1) & 1, abort_flag, status)) break;
            const uint32_t bias_at = smem_u32(smem + DG_BIAS) + (uint32_t)buf * 1024;
            if (biased) {
#pragma unroll
                for (int z = 0; z < (GATED ? 2 : 1); ++z)
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const int c = (2 * i + par) * 32 + lane;
                        if (c < per)
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(
                                             bias_at + (uint32_t)(z * g.half + c) * 4),
                                         "f"(bias[z][i])
                                         : "memory");
                    }
                __syncwarp();
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + (uint32_t)(buf * DG_ACC) + ((uint32_t)(32 * q) << 16);
            void *out = g.out[second ? 1 : 0];
            float v[32], w[32];
            if (SPLIT) {
                // group c / 32 is finished by pair c / 32 mod split: the others send theirs
                for (int c = par * 32; c < per; c += 64) {
                    const int owner = (c >> 5) % params.split;
                    if (owner == work.part) continue;
                    const uint32_t to = cluster_addr(
                        sums_at<GATED>(smem, params.split, per, work.part, owner, c, q),
                        2 * owner + rank);
                    tmem_ld32(acc + c, v);
                    send32(to, lane, v);
                    if (GATED) {
                        tmem_ld32(acc + g.half + c, w);
                        send32(to + 4 * DG_TURN, lane, w);
                    }
                }
                sent = true;
                break;
            }
            for (int c = par * 32; c < per; c += 64) {
                const int col = work.n * per + c;
                const int width = min(min(32, per - c), g.N - col);
                if (row >= g.M || width <= 0) continue;
                Residual res;
                if (!GATED && g.residual && g.parts == 1)
                    res.load(g.residual, g.rdt, g.ldr, lane, row, g.M, col, width);
                tmem_ld32(acc + c, v);
                if (GATED) tmem_ld32(acc + g.half + c, w);
                if (g.parts == 1) {
                    finish<GATED>(g, turn, lane, out, row, col, width, v, w, res,
                                  bias_at + (uint32_t)c * 4);
                } else {
                    turn_in(turn, lane, v);
                    turn_rows(turn, lane, plane_of(g, work.part, second ? 1 : 0), RVQ_F32, g.N, row,
                              g.M, col, width, nullptr, 0);
                    if (GATED) {
                        turn_in(turn, lane, w);
                        turn_rows(turn, lane, plane_of(g, work.part, 1), RVQ_F32, g.N, row, g.M, col,
                                  width, nullptr, 0);
                    }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_cluster(cluster_addr(accempty0 + 8 * buf, lead));
        }
    }
    __syncwarp();
    if (SPLIT) {
        cluster_sync();  // the sums have arrived
        if (warp >= 4 && sent) {
            // this pair's share of the columns, the pairs' sums added in order
            const GemmArgs &g = params.g[JOBS == 1 ? 0 : work.job];
            const int per = GATED ? g.half : g.tile_n;
            const int mt1 = g.mode == DG_PAIR_M ? g.mt / 2 : g.mt;
            const bool second = work.m >= mt1;
            const int row =
                (second ? work.m - mt1 : work.m) * 2 * DG_BM + (int)rank * DG_BM + 32 * q;
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
            float v[32], w[32];
            for (int c = par * 32; c < per; c += 64) {
                const int col = work.n * per + c;
                const int width = min(min(32, per - c), g.N - col);
                if ((c >> 5) % params.split != work.part || row >= g.M || width <= 0) continue;
                Residual res;
                if (!GATED && g.residual)
                    res.load(g.residual, g.rdt, g.ldr, lane, row, g.M, col, width);
                tmem_ld32(acc + c, v);
                if (GATED) tmem_ld32(acc + g.half + c, w);
                for (int from = 0; from < params.split; ++from) {
                    if (from == work.part) continue;
                    const uint32_t at =
                        sums_at<GATED>(smem, params.split, per, from, work.part, c, q);
                    add_sent32(at, lane, v);
                    if (GATED) add_sent32(at + 4 * DG_TURN, lane, w);
                }
                finish<GATED>(g, turn, lane, g.out[second ? 1 : 0], row, col, width, v, w, res,
                              smem_u32(smem + DG_BIAS) + (uint32_t)c * 4);
            }
        }
    }
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

// Adds a tile's parts in slice order and finishes the outputs: eight columns per
// thread.  Memory-bound (the parts are in L2).
template <bool GATED>
__global__ void __launch_bounds__(256) dense_parts_kernel(const __grid_constant__ GemmArgs g) {
    dependency_wait();
    const int n8 = g.N / 8, z = blockIdx.y;  // second problem of PAIR_M
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)g.M * n8) return;
    const int64_t row = i / n8;
    const int c = (int)(i % n8) * 8;
    const int64_t at = row * g.N + c;
    float v[8] = {}, w[8] = {}, t[8];
    for (int p = 0; p < g.parts; ++p) {
        ld8(plane_of(g, p, z), RVQ_F32, at, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += t[e];
        if (GATED) {
            ld8(plane_of(g, p, 1), RVQ_F32, at, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] += t[e];
        }
    }
    if (g.bias[0]) {
        ld8(g.bias[0], g.dt, c, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    if (g.pre[0]) st8(g.pre[0], RVQ_F32, at, v);
    act_group(g.act, v);
    if (GATED) {
        if (g.bias[1]) {
            ld8(g.bias[1], g.dt, c, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] += t[e];
        }
        if (g.pre[1]) st8(g.pre[1], RVQ_F32, at, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= w[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= g.alpha;
        if (g.residual) {
            ld8(g.residual, g.rdt, row * g.ldr + c, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t[e];
        }
    }
    st8(g.out[z], g.odt, row * g.ldo + c, v);
}

// How a product is cut: tile width, and the parts of a tile.
struct GemmPlan {
    int tile_n, mt, nt, slices, parts, split;
    double cycles;
};

// Cycles of a 64-deep slice of a 256 x tile_n tile: the MMAs' 2 per column, or, for
// narrower tiles, the issue and the operand fill (measured 508 at 128 columns, 530
// at 192 and 224).  Of rows on 128-byte lines: others touch five 32-byte sectors for
// every four (663 at 256 columns), which the model leaves out.
double slice_cycles(int tile_n) {
    const double fill = 460.0 + 0.375 * tile_n;
    return 2.0 * tile_n > fill ? 2.0 * tile_n : fill;
}

// A tile's share of a pair's time: its slices, or, of a short depth, its outputs'
// way out, which the next tile's slices would have hidden (18 cycles a column for a
// plain 16-bit output; pre, an activation and a residual take more, left out).
double tile_cycles(int slices, int tile_n) {
    const double in = slices * slice_cycles(tile_n) + 600.0, out = 18.0 * tile_n;
    return in > out ? in : out;
}

// Clusters of `split` pairs that the device holds at once (0: none).
int max_clusters(int split);

// A product cut into tiles of tile_n columns, each split among `split` pairs; cycles:
// those of one tile, without its way out (18 a column).  The pairs of a split tile
// send each other the sums that they do not write out: 1200, and 35 a column.
GemmPlan cut(const DenseJob &j, int tile_n, int split) {
    GemmPlan p = {};
    p.tile_n = tile_n;
    p.parts = 1;
    p.split = split;
    p.mt = (j.M + 2 * DG_BM - 1) / (2 * DG_BM) * (j.mode == DG_PAIR_M ? 2 : 1);
    const int per = j.mode == DG_GATED ? tile_n / 2 : tile_n;
    p.nt = (j.N + per - 1) / per;
    const int kb = (j.K + DG_BK - 1) / DG_BK;
    p.slices = j.mode == DG_SUM_K ? 2 * kb : kb;
    p.cycles = tile_cycles((p.slices + split - 1) / split, tile_n);
    if (split > 1) {
        const int groups = (per + 31) / 32, mine = (groups + split - 1) / split;
        const double sent = tile_n * (1.0 - (double)mine / groups);
        p.cycles = ((p.slices + split - 1) / split) * slice_cycles(tile_n) + 600.0 + 1200.0 +
                   (35.0 - 18.0) * sent;
    }
    return p;
}

// A tile of fewer slices than that gains less than the exchange costs.
constexpr int kSplitSlices = 12;

bool split_fits(const GemmPlan &p, bool gated) {
    return p.slices >= 2 * p.split &&
           sums_bytes(p.split, gated ? p.tile_n / 2 : p.tile_n, gated) <= kSumsMax;
}

// The cheapest of the tile widths: (waves of pairs) x (a tile's time).  Where not
// even half the pairs would have a tile, its slices are split among the pairs of a
// cluster, or cut into (up to `most`) parts, which costs the parts' way through L2
// and a second launch.
constexpr int kMaxParts = 8;
GemmPlan plan_gemm(const DenseJob &j, int pairs, int most = kMaxParts, int max_split = 4) {
    constexpr double kParts = 6000.0;
    GemmPlan best = {}, shared = {};
    best.cycles = shared.cycles = 1e300;
    const double planes = j.mode == DG_GATED || j.mode == DG_PAIR_M ? 2.0 : 1.0;
    for (int tn = 256; tn >= 64; tn -= 32) {
        if (j.b_t && tn != 256 && tn != 128) continue;  // whole 64-row boxes per CTA
        GemmPlan p = cut(j, tn, 1);
        const double tiles = (double)p.mt * p.nt;
        for (int parts = 1; parts <= most; ++parts) {
            if (parts > 1 && (tiles * parts > pairs || p.slices < 8 * parts)) break;
            // the parts' bytes, written and read at about 5 KB per cycle
            const double join = parts > 1 ? kParts + parts * planes * j.M * j.N * 8.0 / 5000.0 : 0.0;
            p.parts = parts;
            p.cycles =
                ceil(tiles * parts / pairs) * tile_cycles((p.slices + parts - 1) / parts, tn) + join;
            if (p.cycles < best.cycles * 0.999) best = p;
        }
        for (int split = 2; split <= max_split && p.slices >= kSplitSlices; split *= 2) {
            const GemmPlan q = cut(j, tn, split);
            if (tiles * split <= pairs && split_fits(q, j.mode == DG_GATED) &&
                q.cycles + 18.0 * tn < shared.cycles + 18.0 * shared.tile_n &&
                tiles <= max_clusters(split))
                shared = q;
        }
    }
    // a tile's way out counts here: a split one's is shared.  Parts are estimated
    // high by about a tenth.
    const double most_cycles = (best.cycles + 18.0 * best.tile_n) * (best.parts > 1 ? 0.9 : 1.0);
    if (shared.cycles + 18.0 * shared.tile_n < most_cycles) return shared;
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

// Partial sums of any cut that plan_gemm may choose for up to these M, N and K, so
// that a workspace serves fewer tokens too (which may be cut where more are not).  A
// tile of 256 x 256 at most holds a pair's part, and there are no more parts than pairs.
size_t dense_gemm_partial_bytes(const DenseJob &job) {
    if (dense_stream_fits(job)) return 0;  // and so does every smaller M
    const int kb = (job.K + DG_BK - 1) / DG_BK, slices = job.mode == DG_SUM_K ? 2 * kb : kb;
    const int parts = slices / 8 < kMaxParts ? slices / 8 : kMaxParts;
    if (parts < 2) return 0;
    const size_t planes = job.mode == DG_GATED || job.mode == DG_PAIR_M ? 2 : 1;
    const size_t all = (size_t)parts * planes * job.M * job.N * 4;
    const size_t most = (size_t)(num_sms() / 2) * 2 * DG_BM * DG_ACC * 4;
    return all < most ? all : most;
}

// Arguments and tensor maps of a product cut by `plan`.
static rvq_status fill_args(const DenseJob &job, const GemmPlan &plan, GemmArgs &g,
                            CUtensorMap (&a)[2], CUtensorMap (&b)[2]) {
    g = {};
    g.mode = job.mode;
    g.M = job.M;
    g.N = job.N;
    g.a_t = job.a_t;
    g.b_t = job.b_t;
    g.kb = (job.K + DG_BK - 1) / DG_BK;
    g.slices = plan.slices;
    g.mt = plan.mt;
    g.nt = plan.nt;
    g.parts = plan.parts;
    g.tile_n = plan.tile_n;
    g.half = g.tile_n / 2;
    if ((long long)g.mt * g.nt > 0x7fffffffll / DG_GROUP) {
        set_error("dense product: %lld output tiles", (long long)g.mt * g.nt);
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
    g.partial = job.partial;
    g.status = job.status;
    for (int i = 0; i < 2; ++i) {
        if (i == 1 && job.a[1] == nullptr)
            a[1] = a[0];
        else
            RVQ_TRY(encode_operand(&a[i], job.a[i], job.M, job.K, job.lda, job.a_t, job.dt, DG_BM));
        if (i == 1 && job.b[1] == nullptr)
            b[1] = b[0];
        else
            RVQ_TRY(encode_operand(&b[i], job.b[i], job.N, job.K, job.ldb, job.b_t, job.dt, g.half));
    }
    return RVQ_OK;
}

template <bool GATED, int JOBS, bool SPLIT>
static rvq_status launch_products(GemmParams<JOBS> &p, cudaStream_t stream) {
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(dense_gemm_kernel<GATED, JOBS, SPLIT>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, DG_SMEM));
        attr_done[dev] = 1;
    }
    // B's rows come in whole swizzle atoms of 8 rows (1 KB), so every stage starts
    // on one
    int half = 0, ring = DG_RING;
    long long units = 0;
    for (int i = 0; i < JOBS; ++i) {
        const int sums = SPLIT ? sums_bytes(p.split, GATED ? p.g[i].half : p.g[i].tile_n, GATED) : 0;
        ring = DG_RING - sums < ring ? DG_RING - sums : ring;
        half = p.g[i].half > half ? p.g[i].half : half;
        units += (long long)p.g[i].mt * p.g[i].nt * p.g[i].parts;
    }
    const int stage = DG_ABYTES + half * 128;
    for (int i = 0; i < JOBS; ++i) {
        p.g[i].stage = stage;
        p.g[i].stages = ring / stage < DG_MAX_ST ? ring / stage : DG_MAX_ST;
    }
    const int pairs_max = num_sms() / 2;
    const int pairs = SPLIT ? (int)units * p.split : units < pairs_max ? (int)units : pairs_max;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(DG_THREADS);
    cfg.dynamicSmemBytes = DG_SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SPLIT ? 2 * p.split : 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    RVQ_CUDA(cudaLaunchKernelEx(&cfg, dense_gemm_kernel<GATED, JOBS, SPLIT>, p));
    RVQ_LAUNCHED("dense_gemm");
    return RVQ_OK;
}

// one product, cut by `plan`
static rvq_status launch_one(const DenseJob &job, const GemmPlan &plan, const BiasSums &sums,
                             cudaStream_t stream) {
    const bool gated = job.mode == DG_GATED;
    GemmParams<1> p = {};
    p.sums = sums;
    RVQ_TRY(fill_args(job, plan, p.g[0], p.a[0], p.b[0]));
    p.split = plan.split;
    if (plan.split > 1)
        return gated ? launch_products<true, 1, true>(p, stream)
                     : launch_products<false, 1, true>(p, stream);
    RVQ_TRY((gated ? launch_products<true, 1, false>(p, stream)
                   : launch_products<false, 1, false>(p, stream)));
    if (plan.parts == 1) return RVQ_OK;
    const int64_t threads = (int64_t)job.M * (job.N / 8);
    const dim3 grid((unsigned)((threads + 255) / 256), job.mode == DG_PAIR_M ? 2u : 1u);
    RVQ_CUDA(gated ? launch_after(dense_parts_kernel<true>, grid, 256, 0, stream, p.g[0])
                   : launch_after(dense_parts_kernel<false>, grid, 256, 0, stream, p.g[0]));
    return RVQ_OK;
}

namespace {
int max_clusters(int split) {
    static std::atomic<int> cached[64][2];  // per device, plus one
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
    std::atomic<int> &known = cached[dev][split == 4];
    if (known) return known - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms() / (2 * split) * 2 * split));
    cfg.blockDim = dim3(DG_THREADS);
    cfg.dynamicSmemBytes = DG_SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(dense_gemm_kernel<false, 1, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, DG_SMEM) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, dense_gemm_kernel<false, 1, true>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();  // not the caller's error: tiles stay whole
        n = 0;
    }
    known = n + 1;
    return n;
}
}  // namespace

rvq_status launch_dense_gemm(const DenseJob &job, cudaStream_t stream) {
    if (dense_stream_fits(job)) return launch_dense_stream(job, stream);
    return launch_one(job, plan_gemm(job, num_sms() / 2), BiasSums{}, stream);
}

// How two products without a common output are cut, for one launch or (together
// false) one each.
struct TwoPlan {
    GemmPlan x, y;
    bool together, split, swap;  // split: every tile among the pairs of a cluster
    int bonus;                   // see Work
};

static TwoPlan plan_two(const DenseJob &x, const DenseJob &y, long long pairs) {
    const GemmPlan ax = plan_gemm(x, (int)pairs), ay = plan_gemm(y, (int)pairs);
    const double apart = ax.cycles + ay.cycles + 6500.0;
    // together with every tile split among a cluster's pairs
    GemmPlan sx = {}, sy = {};
    double split_cycles = 1e300;
    for (int split = 2; split <= 4 && (ax.slices >= kSplitSlices || ay.slices >= kSplitSlices);
         split *= 2)
        for (int c = 0; c < 4; ++c) {
            const GemmPlan p = cut(x, c & 1 ? 128 : 256, split), q = cut(y, c & 2 ? 128 : 256, split);
            const double t = p.cycles > q.cycles ? p.cycles : q.cycles;
            const long long units = (long long)p.mt * p.nt + (long long)q.mt * q.nt;
            if (units * split <= pairs && t < split_cycles && split_fits(p, false) &&
                split_fits(q, false) && units <= max_clusters(split)) {
                sx = p;
                sy = q;
                split_cycles = t;
            }
        }
    const GemmPlan px = plan_gemm(x, (int)pairs, 1, 1), py = plan_gemm(y, (int)pairs, 1, 1);
    const double tx = tile_cycles(px.slices, px.tile_n), ty = tile_cycles(py.slices, py.tile_n);
    const bool swap = tx < ty;  // the longer tiles first
    const GemmPlan &p0 = swap ? py : px, &p1 = swap ? px : py;
    const double t0 = swap ? ty : tx, t1 = swap ? tx : ty;
    // Cycles until the last pair is done, one launch after the other and together
    // (see Work); together only where that ends sooner (whole training steps, apart
    // and together: 4096 tokens of 7168 x 2048, equal waves, 484 and 491 us, so 3 %
    // are taken for operands that are shared less; 1333 x 1000 x 2048, equal waves,
    // 57.5 and 54 us, so 6500 cycles for a launch; 1777 x 4104 x 1736, 121 slices and
    // 93, 114 and 101 us).
    const long long u0 = (long long)p0.mt * p0.nt, u1 = (long long)p1.mt * p1.nt;
    const long long first = u0 % pairs, early = pairs - first;
    const int bonus = first ? (int)(t0 / t1) : 0;
    const long long rest = u1 > bonus * early ? u1 - bonus * early : 0;
    const double late_end = (double)(u0 / pairs + (first ? 1 : 0)) * t0 +
                            (double)(rest / pairs + (rest % pairs > early ? 1 : 0)) * t1;
    const double early_end = (double)(u0 / pairs) * t0 +
                             (double)(bonus + (rest + pairs - 1) / pairs) * t1;
    const double together = late_end > early_end ? late_end : early_end;
    const bool one = together * 1.03 < apart && together <= split_cycles;
    const bool split = split_cycles < apart && !one;
    const bool both = one || split;
    return {one ? px : split ? sx : ax, one ? py : split ? sy : ay, both, split, swap && one, bonus};
}

rvq_status launch_dense_gemm_two(const DenseJob &x, const DenseJob &y, const BiasSums &sums,
                                 cudaStream_t stream) {
    const long long pairs = num_sms() / 2;
    if (dense_stream_fits(x) || dense_stream_fits(y)) {
        // few tokens: each its own way, the bias gradients beside the tiled one
        const DenseJob *jobs[2] = {&x, &y};
        bool added = !sums.wanted();
        for (int i = 1; i >= 0; --i) {
            const DenseJob &j = *jobs[i];
            if (!j.out[0]) continue;
            if (dense_stream_fits(j)) {
                RVQ_TRY(launch_dense_stream(j, stream));
            } else {
                RVQ_TRY(launch_one(j, plan_gemm(j, (int)pairs), added ? BiasSums{} : sums, stream));
                added = true;
            }
        }
        return added ? RVQ_OK : launch_bias_sums(sums, stream);
    }
    const TwoPlan t = plan_two(x, y, pairs);
    if (!t.together || !x.out[0] || !y.out[0]) {
        // a product wanted alone is cut as it would be beside the other: the same sums
        if (x.out[0]) RVQ_TRY(launch_one(x, t.x, y.out[0] ? BiasSums{} : sums, stream));
        if (y.out[0]) return launch_one(y, t.y, sums, stream);
        return !x.out[0] && sums.wanted() ? launch_bias_sums(sums, stream) : RVQ_OK;
    }
    const DenseJob &j0 = t.swap ? y : x, &j1 = t.swap ? x : y;
    GemmParams<2> p = {};
    RVQ_TRY(fill_args(j0, t.swap ? t.y : t.x, p.g[0], p.a[0], p.b[0]));
    RVQ_TRY(fill_args(j1, t.swap ? t.x : t.y, p.g[1], p.a[1], p.b[1]));
    p.sums = sums;
    p.split = t.x.split;
    p.bonus = t.bonus;
    return t.split ? launch_products<false, 2, true>(p, stream)
                   : launch_products<false, 2, false>(p, stream);
}

void dense_plan_of(const DenseJob &x, const DenseJob *y, int32_t (&out)[7]) {
    const int pairs = num_sms() / 2;
    const auto way = [](const DenseJob &j, const GemmPlan &p, int32_t *o) {
        const bool streamed = dense_stream_fits(j);
        o[0] = streamed ? MOE_WAY_STREAM
               : p.split > 1 ? MOE_WAY_SPLIT
               : p.parts > 1 ? MOE_WAY_PARTS : MOE_WAY_TILES;
        o[1] = streamed ? 0 : p.split > 1 ? p.split : p.parts;
        o[2] = streamed ? 0 : p.tile_n;
    };
    for (int32_t &v : out) v = 0;
    if (y == nullptr || dense_stream_fits(x) || dense_stream_fits(*y)) {
        way(x, plan_gemm(x, pairs), out + 1);
        if (y) way(*y, plan_gemm(*y, pairs), out + 4);
        return;
    }
    const TwoPlan t = plan_two(x, *y, pairs);
    out[0] = t.together;
    way(x, t.x, out + 1);
    way(*y, t.y, out + 4);
}

}  // namespace rvq
