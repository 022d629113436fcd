// Tensor-core and cluster helpers shared by the dense products (dense_gemm.cu,
// dense_stream.cu).  Inline PTX; sm_100 family.
#pragma once

#include <cuda.h>

#include "dense.cuh"
#include "tc_util.cuh"

namespace rvq {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}

// One lane of a converged warp.  The instructions that feed the tensor cores
// and TMA take their operands from uniform registers: behind elect.sync, in
// code the whole warp runs, the compiler passes them directly; behind a test of
// the lane number it loops over the lanes that might differ (measured: 126
// cycles per MMA at any width, twice the work of a 128-column MMA).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Bounded wait of a whole warp on a barrier phase; every lane gets the same
// answer, so the warp stays converged when a wait gives up.  False once another
// role has aborted, or after kWaitLimitNs (then the abort flag is raised and the
// timeout recorded).  The clock is looked at every 256th try only: a global timer
// read between two tries cost the tensor pipe more than the wait itself.
__device__ __forceinline__ bool warp_wait(uint32_t mbar, uint32_t parity, volatile int *abort_flag,
                                          uint32_t *status) {
    unsigned long long t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_now(mbar, parity))) return true;
        if ((i & 255u) != 255u) continue;
        const unsigned long long now = global_ns();
        if (t0 == 0) t0 = now;
        const bool late = now - t0 > kWaitLimitNs;
        if (late) {
            *abort_flag = 1;
            set_dev_error(status, RVQ_DEV_ERR_TIMEOUT);
        }
        if (__any_sync(0xffffffffu, late || *abort_flag != 0)) return false;
    }
}

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// address of the same shared variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

// Shared-memory descriptor, 128-byte swizzle.  K-major: 8-row groups 1024 bytes
// apart.  MN-major: 64 rows x 8 deep per 1024 bytes; the next 8 deep follow at
// 1024 bytes (stride offset), the next 64 rows at 8192 (leading offset).
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, int t) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(t ? 8192u >> 4 : 1u) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// 16 columns of this warp's 32 TMEM lanes; the values are there after tmem_wait()
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Tensor map of an operand's slices: K-major boxes of 64 deep x box_rows, or,
// transposed, of 64 rows x 64 deep (dense_gemm.cu).
rvq_status encode_operand(CUtensorMap *map, const void *p, int rows, int K, int64_t ld, int t, int dt,
                          int box_rows);

}  // namespace rvq
