// What the attention kernels need beside q2_0_device.cuh and q2_0_tcgen05.cuh. (A header of their
// own: the mat-vec and GEMM kernels' recorded counters hold for those two as they are.)
#pragma once

#include "q2_0_device.cuh"
#include "q2_0_tcgen05.cuh"

namespace q2 {

// As mbar_wait for waits on a critical path: try_wait suspends the thread in hardware
// until the phase completes or a short time passes, and is simply tried again; the
// timer, whose read takes longer than most such waits, is looked at from the 64th try on.
__device__ __forceinline__ bool mbar_wait_spin(uint64_t *bar, uint32_t parity,
                                               unsigned long long *err, int tag,
                                               uint64_t limit_ns = kWaitLimitNs) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit_ns) {
            record_error(err, Q2_0_DEVERR_TIMEOUT, tag);
            return false;
        }
    return true;
}

// 3-D tiled tensor copy global -> shared; c0 is the innermost coordinate.
__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, int c0, int c1,
                                            int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, kind::f16 (types and majors in the
// instruction descriptor; D f32)
__device__ __forceinline__ void tc_mma_f16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// tmem_ld32 without the wait: the registers are valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Shared-memory matrix descriptor with all fields: byte offsets lbo and sbo,
// layout 0 (no swizzle) or 2 (128-byte swizzle).
//   MN-major, no swizzle: 8 x 8 core matrices (a row of 16 bytes along MN for each
//     k); sbo from one group of 8 along MN to the next, lbo along K.
//   MN-major, 128-byte swizzle: 64 (MN) x 8 (K) atoms of 1024 bytes; sbo from one
//     atom to the next along K, lbo along MN.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo,
                                              uint32_t layout) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | uint64_t(lbo >> 4) << 16 | uint64_t(sbo >> 4) << 32 |
           uint64_t(1) << 46 | uint64_t(layout) << 61;
}

}  // namespace q2
