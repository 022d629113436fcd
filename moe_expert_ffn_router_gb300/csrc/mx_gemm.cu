// Products of microscaled matrices for many tokens, in one persistent kernel; tensor
// maps and the choice of a kernel for both (mx_stream.cu).
//
// Compute-bound at prefill sizes (two 4-bit operands are multiplied four times as fast
// as 16-bit ones, but no less is to be brought per tile and output), so the design feeds
// block-scaled tcgen05.mma without a pause:
//  * A pair of CTAs (a cluster of two) owns a 256 x 256 tile: CTA r holds rows 128 r .. of
//    the tokens and half of the tile's weight rows (a gated product: the leader 128 gate
//    rows, the follower the 128 up rows), the leader's one thread issues cta_group::2
//    MMAs on both halves.
//  * A slice is one 128-byte swizzled row deep (256 columns of two 4-bit operands, else
//    128), five stages per CTA.  The slice's scales come along as they lie in memory:
//    those of its own 128 rows of tokens, and of all the tile's weight rows, in each CTA.
//    The issuing thread copies them into tensor memory ahead of the MMAs, in order with
//    them.
//  * The accumulator (256 columns) and the scales do not leave room for a second one in
//    tensor memory, so the epilogue's eight warps take a tile into registers (128 values
//    each), let the next tile begin, and finish and write it from there.
// Rows, columns and depth past the ends are zero-filled by TMA (scales and codes) and not
// stored.  Each output is rounded once, from fp32.  Every wait is bounded (1 s).
//
// Measured (GB300; two 4-bit operands, 8-bit tokens and 4-bit weights): 8192^3 143 and
// 261 us (7.7 and 4.2 PFLOP/s), 2048 tokens through the gated projection 7168 -> 2048 23.8
// and 38.7 (128 tiles for 76 pairs: 1.68 waves), 4096 tokens 40.5 and 69.8; 2048 x 2048 ->
// 7168 with an fp32 residual 33.7 and 36.5 (its 117 MB of rows, 17 us at the copy rate, in
// epilogues of three tiles a pair).  A slice takes about 640 cycles of two 4-bit
// operands, whose MMAs take 512: the fill (35 KB a CTA, 55 bytes per cycle and SM).
#include "dense_epilogue.cuh"
#include "mx_tc.cuh"

#include <cudaTypedefs.h>

namespace rvq {
namespace {

constexpr int MG_ROWS = 128;            // rows of an operand per CTA
constexpr int MG_CODES = MG_ROWS * 128; // bytes of an operand's slice
constexpr int MG_STAGES = 5;
constexpr int MG_EPI_WARPS = 8;
constexpr int MG_TURN = 4096;           // staging of an epilogue warp
constexpr int MG_GROUP = 8;             // M tiles walked together (operand reuse in L2)
constexpr int MG_THREADS = 32 * (4 + MG_EPI_WARPS);
constexpr int MG_SCALES = 256;          // first TMEM column behind the accumulator

// Bytes of a stage: codes of the tokens, of the weights, their scales.
template <bool F4>
struct Stage {
    static constexpr int KT = F4 ? 2 : 1;  // tiles of scales a slice is deep
    static constexpr int B = MG_CODES, SA = 2 * MG_CODES, SB = SA + KT * kMxTileBytes;
    static constexpr int BYTES = (SB + 2 * KT * kMxTileBytes + 1023) / 1024 * 1024;
    static constexpr int TURN = MG_STAGES * BYTES, BARS = TURN + MG_EPI_WARPS * MG_TURN;
    static constexpr int SMEM = BARS + 256;
    static_assert(SMEM <= 232448, "shared memory of a CTA");
};

struct MxGemmArgs {
    int M, N, slices, mt, nt;
    uint32_t idesc, expect;  // bytes that TMA counts per stage, of both CTAs
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

struct MxGemmParams {
    CUtensorMap a, sa, b[2], sb[2];
    MxGemmArgs g;
};

// Relaxed: what the barrier guards is tensor memory, whose loads have been waited for
// (a release would wait for the warp's stores to global memory too).
__device__ __forceinline__ void arrive_cluster(uint32_t mbar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mbar)
                 : "memory");
}

// Registers move from the warps that only issue to those of the epilogue: the shares
// add up to what the block was launched with.
constexpr int MG_REGS = 168, MG_REGS_ISSUE = 56, MG_REGS_EPI = 224;
static_assert(MG_THREADS * MG_REGS <= 65536 &&
                  128 * MG_REGS_ISSUE + 32 * MG_EPI_WARPS * MG_REGS_EPI <= MG_THREADS * MG_REGS,
              "registers of a block");
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
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

// arrives on the barrier at this offset in both CTAs once the MMAs issued so far are done
__device__ __forceinline__ void commit_pair(uint32_t mbar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(mbar),
        "h"((uint16_t)3)
        : "memory");
}

// output tile t -> (m tile, n tile): groups of MG_GROUP M tiles, N inside
__device__ __forceinline__ void tile_at(const MxGemmArgs &g, int t, int &m, int &n) {
    const int grp = t / (MG_GROUP * g.nt);
    const int first = grp * MG_GROUP;
    const int rows = min(MG_GROUP, g.mt - first);
    const int r = t - grp * MG_GROUP * g.nt;
    m = first + r % rows;
    n = r / rows;
}

// 32 columns of the accumulator; the values are there after tmem_wait()
__device__ __forceinline__ void tmem_ld32_to(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// adds bias[c .. c + 32), of which `width` (a multiple of 8) exist
__device__ __forceinline__ void add_bias(const float *bias, int c, int width, float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (4 * j >= width) continue;
        const float4 b = __ldg(reinterpret_cast<const float4 *>(bias + c) + j);
        v[4 * j] += b.x;
        v[4 * j + 1] += b.y;
        v[4 * j + 2] += b.z;
        v[4 * j + 3] += b.w;
    }
}

// A lane's 32 values as a block of the microscaled output (column c of row `row`);
// returns the scale's byte.
template <int FMT>
__device__ __forceinline__ uint32_t put_block(const MxGemmArgs &g, int row, int c, bool on,
                                              float (&v)[32]) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    const uint32_t byte = mx_byte<FMT>(top);
    const float inv = mx_inverse(byte);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = byte == 255 ? 0.f : v[e] * inv;
    const int64_t at = (int64_t)row * g.otiles * kMxTile + c;
    if (FMT == MOE_MX_F8) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = e4m3x4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        if (on) {
            uint4 *q = reinterpret_cast<uint4 *>(g.codes + at);
            q[0] = make_uint4(w[0], w[1], w[2], w[3]);
            q[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = v[8 * j + e];
            w[j] = e2m1x8(q);
        }
        if (on) *reinterpret_cast<uint4 *>(g.codes + at / 2) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return byte;
}

template <bool GATED, bool F4>
__global__ void __launch_bounds__(MG_THREADS, 1) mx_gemm_kernel(
    const __grid_constant__ MxGemmParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using S = Stage<F4>;
    const MxGemmArgs &g = p.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = g.mt * g.nt;
    uint8_t *bars = smem + S::BARS;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * MG_STAGES,
                   accfull = empty0 + 8 * MG_STAGES, accempty = accfull + 8;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 8 * (2 * MG_STAGES + 2));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < MG_STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(accfull, 1);
        mbar_init(accempty, 2 * MG_EPI_WARPS);
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

    if (warp < 4) {
        fewer_registers<MG_REGS_ISSUE>();
        if (warp == 0) {
            // producer: this CTA's rows of both operands for every slice, and the scales
            int s = 0;
            uint32_t lap = 0;  // trips around the ring
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs) {
                int m, n;
                tile_at(g, t, m, n);
                const int a0 = m * 2 + (int)rank;                          // groups of 128 rows
                const int b0 = GATED ? n : n * 2 + (int)rank;
                const CUtensorMap *mb = &p.b[GATED ? rank : 0];
                for (int k = 0; k < g.slices; ++k) {
                    if (lap > 0 && !warp_wait(empty0 + 8 * s, (lap - 1) & 1, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = smem_u32(smem + s * S::BYTES);
                    const uint32_t bar = cluster_addr(full0 + 8 * s, 0);
                    const int kx = k * 128, ks = k * S::KT * 128;
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, g.expect);
                        tma_pair(st, &p.a, kx, a0 * MG_ROWS, bar);
                        tma_pair(st + S::B, mb, kx, b0 * MG_ROWS, bar);
                        tma_pair(st + S::SA, &p.sa, ks, a0, bar);
                        if (GATED) {
                            tma_pair(st + S::SB, &p.sb[0], ks, n, bar);
                            tma_pair(st + S::SB + S::KT * kMxTileBytes, &p.sb[1], ks, n, bar);
                        } else {
                            tma_pair(st + S::SB, &p.sb[0], ks, 2 * n, bar);
                        }
                    }
                    __syncwarp();
                    if (++s == MG_STAGES) {
                        s = 0;
                        ++lap;
                    }
                }
            }
        } else if (warp == 1 && rank == 0) {
            // issuer: the slice's scales, then four MMAs
            int s = 0, done = 0;
            uint32_t lap = 0;
            bool ok = true;
            const uint32_t tsa = tmem + MG_SCALES, tsb = tsa + 4 * S::KT;
            for (int t = pair; ok && t < tiles; t += pairs, ++done) {
                if (done >= 1 && !warp_wait(accempty, (done - 1) & 1, abort_flag, g.status)) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int k = 0; k < g.slices; ++k) {
                    if (!warp_wait(full0 + 8 * s, lap & 1, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t st = smem_u32(smem + s * S::BYTES);
                    const uint64_t a = smem_desc(st), b = smem_desc(st + S::B);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < S::KT; ++i) {
                            copy_scales<2>(tsa + 4 * i, st + S::SA + i * kMxTileBytes);
                            copy_scales<2>(tsb + 8 * i, st + S::SB + i * kMxTileBytes);
                            copy_scales<2>(tsb + 8 * i + 4, st + S::SB + (S::KT + i) * kMxTileBytes);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int kt = F4 ? q >> 1 : 0;
                            mx_mma<2, F4>(tmem, a + 2 * q, b + 2 * q,
                                          g.idesc | scale_places(F4 ? 2 * (q & 1) : q), tsa + 4 * kt,
                                          tsb + 8 * kt, (k > 0 || q > 0) ? 1u : 0u);
                        }
                        commit_pair(empty0 + 8 * s);
                    }
                    __syncwarp();
                    if (++s == MG_STAGES) {
                        s = 0;
                        ++lap;
                    }
                }
                if (elect_one()) commit_pair(accfull);
                __syncwarp();
            }
        }
    } else {
        more_registers<MG_REGS_EPI>();
        // epilogue: lanes 32 q .. 32 q + 31 of the accumulator, one half of its columns
        const int q = warp & 3, par = (warp - 4) >> 2;
        const uint32_t turn = smem_u32(smem + S::TURN) + (uint32_t)(warp - 4) * MG_TURN;
        constexpr int PER = GATED ? 128 : 256;  // outputs of a tile's row
        constexpr int STEPS = GATED ? 2 : 4;    // groups of 32 outputs of a warp
        int done = 0;
        for (int t = pair; t < tiles; t += pairs, ++done) {
            int m, n;
            tile_at(g, t, m, n);
            const int row = m * 256 + (int)rank * MG_ROWS + 32 * q;
            const int c0 = n * PER + par * (PER / 2);
            if (!GATED && g.residual && row + lane < g.M) {
                // this warp's part of the residual into L2 while the tile is multiplied
                const int e = g.rdt == RVQ_F32 ? 4 : 2;
                for (int c = c0; c < c0 + PER / 2 && c < g.N; c += 32)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(
                        reinterpret_cast<const char *>(g.residual) +
                        ((int64_t)(row + lane) * g.ldr + c) * e));
            }
            if (!warp_wait(accfull, done & 1, abort_flag, g.status)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(par * (PER / 2));
            uint32_t v[128];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                tmem_ld32_to(GATED ? acc + (i >> 1) * 32 + (i & 1) * 128 : acc + i * 32, v + 32 * i);
            tmem_wait();
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_cluster(cluster_addr(accempty, 0));
            uint32_t bytes = 0;
#pragma unroll 1
            for (int i = 0; i < STEPS; ++i) {
                const int col = c0 + 32 * i, width = min(32, g.N - col);
                float x[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e]);
                Residual res;
                if (!GATED && g.residual && width > 0 && row < g.M)
                    res.load(g.residual, g.rdt, g.ldr, lane, row, g.M, col, width);
                if (width > 0 && row < g.M) {
                    if (g.bias[0]) add_bias(g.bias[0], col, width, x);
                    if (g.act != MOE_ACT_NONE) act_group(g.act, x);
                    if (GATED) {
                        float u[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __uint_as_float(v[32 + e]);
                        if (g.bias[1]) add_bias(g.bias[1], col, width, u);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] *= u[e];
                    } else if (g.alpha != 1.f) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] *= g.alpha;
                    }
                }
                if (GATED && g.codes) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (e >= width) x[e] = 0.f;  // padded columns
                    const bool on = row + lane < g.M;
                    const uint32_t byte =
                        g.ofmt == MOE_MX_F8 ? put_block<MOE_MX_F8>(g, row + lane, col, on, x)
                                            : put_block<MOE_MX_F4>(g, row + lane, col, on, x);
                    bytes |= byte << (8 * i);
                    if (i == STEPS - 1 && on)
                        *reinterpret_cast<uint16_t *>(
                            g.scales + mx_scale_at(row + lane, n, g.otiles) + 2 * par) =
                            (uint16_t)bytes;
                } else if (width > 0 && row < g.M) {
                    if (g.odt != RVQ_F32 && g.residual == nullptr) {
                        rows_16_plain(turn, lane, g.out, g.odt, g.ldo, row, g.M, col, width, x);
                    } else {
                        turn_in(turn, lane, x);
                        turn_rows(turn, lane, g.out, g.odt, g.ldo, row, g.M, col, width,
                                  !GATED && g.residual ? &res : nullptr, g.rdt);
                    }
                }
                // the next group's values into place: one body for all of them
#pragma unroll
                for (int e = 0; e + 128 / STEPS < 128; ++e) v[e] = v[e + 128 / STEPS];
            }
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

template <bool GATED, bool F4>
rvq_status launch_tiles(const MxJob &job, cudaStream_t stream) {
    using S = Stage<F4>;
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        // the epilogue's share of registers comes out of what the block is launched with:
        // with fewer it would wait for them forever
        cudaFuncAttributes attr;
        RVQ_CUDA(cudaFuncGetAttributes(&attr, mx_gemm_kernel<GATED, F4>));
        if (attr.numRegs < MG_REGS) {
            set_error("microscaled product: built with %d registers a thread, %d needed",
                      attr.numRegs, MG_REGS);
            return RVQ_ENOTIMPL;
        }
        RVQ_CUDA(cudaFuncSetAttribute(mx_gemm_kernel<GATED, F4>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM));
        attr_done[dev] = 1;
    }
    MxGemmParams p = {};
    MxGemmArgs &g = p.g;
    g.M = job.n;
    g.N = job.rows;
    g.slices = (mx_tiles(job.cols) + S::KT - 1) / S::KT;
    g.mt = (job.n + 255) / 256;
    g.nt = GATED ? mx_tiles(job.rows) : (job.rows + 255) / 256;
    const long long tiles = (long long)g.mt * g.nt;
    if (tiles > 0x7fffffff / MG_GROUP) {
        set_error("microscaled product: %lld output tiles", tiles);
        return RVQ_ENOTIMPL;
    }
    g.idesc = mx_idesc(F4, job.xfmt, job.wfmt, 256, 256);
    g.expect = 2 * (slice_bytes(F4, job.xfmt, MG_ROWS) + slice_bytes(F4, job.wfmt, MG_ROWS) +
                    3 * S::KT * kMxTileBytes);
    g.act = job.act;
    g.rdt = job.rdt;
    g.odt = job.odt;
    g.alpha = job.alpha;
    g.bias[0] = job.bias[0];
    g.bias[1] = job.bias[1];
    g.residual = job.residual;
    g.ldr = job.ldr;
    g.ldo = job.ldo;
    g.out = job.out;
    g.codes = job.codes;
    g.scales = job.scales;
    g.ofmt = job.ofmt;
    g.otiles = mx_tiles(job.rows);
    g.status = job.status;
    RVQ_TRY(encode_codes(&p.a, job.x, job.n, job.cols, job.xfmt, F4, MG_ROWS));
    RVQ_TRY(encode_scales(&p.sa, job.xs, job.n, job.cols, F4, 1));
    for (int i = 0; i < job.mats; ++i) {
        RVQ_TRY(encode_codes(&p.b[i], job.w[i], job.rows, job.cols, job.wfmt, F4, MG_ROWS));
        RVQ_TRY(encode_scales(&p.sb[i], job.ws[i], job.rows, job.cols, F4, GATED ? 1 : 2));
    }
    const int pairs_max = num_sms() / 2;
    const int pairs = tiles < pairs_max ? (int)tiles : pairs_max;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(MG_THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    RVQ_CUDA(cudaLaunchKernelEx(&cfg, mx_gemm_kernel<GATED, F4>, p));
    RVQ_LAUNCHED("mx_gemm");
    return RVQ_OK;
}

}  // namespace

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

// Past 128 tokens the faster by a model of both (measured, us, stream / tiles; 8-bit
// tokens and 4-bit weights: gated 7168 -> 2048, 256 tokens 15.6 / 22.8, 512 22.9 / 21.7;
// plain 7168 -> 2048, 512 13.4 / 21.6, 1024 18.6 / 21.7; 2048 -> 7168 with a residual, 256
// 13.3 / 16.2, 384 19.4 / 16.3; 1736 -> 4104, 256 9.7 / 11.6, 777 15.8 / 10.7; two 4-bit
// operands: gated 256 12.7 / 15.4, 384 15.8 / 13.8).  A slice takes a CTA of the stream
// 0.42 us (0.66 with two matrices) and a pair of CTAs 0.31 (0.33 of two 4-bit operands,
// bound by their fill); launch and outputs take both 6 us.
bool mx_by_tiles(const MxJob &job) {
    if (job.n <= 128) return false;
    const MxStreamPlan s = plan_mx_stream(job);
    const int pairs = num_sms() / 2;
    const long long slots = (long long)num_sms() * (s.two ? 2 : 1);
    const long long rounds = s.split > 1 ? 1 : (s.tiles + slots - 1) / slots;
    const long long per = (s.slices + s.split - 1) / s.split;
    const double stream = 6.3 + rounds * per * (job.mats == 2 ? 0.66 : 0.42);
    const long long tiles = (long long)((job.n + 255) / 256) *
                            (job.mats == 2 ? mx_tiles(job.rows) : (job.rows + 255) / 256);
    const double tiled =
        6.2 + (double)((tiles + pairs - 1) / pairs) * s.slices * (job.f4() ? 0.33 : 0.31);
    return tiled < stream;
}

rvq_status launch_mx_product(const MxJob &job, cudaStream_t stream) {
    if (!mx_by_tiles(job)) return launch_mx_stream(job, stream);
    if (job.mats == 2)
        return job.f4() ? launch_tiles<true, true>(job, stream)
                        : launch_tiles<true, false>(job, stream);
    return job.f4() ? launch_tiles<false, true>(job, stream)
                    : launch_tiles<false, false>(job, stream);
}

}  // namespace rvq
