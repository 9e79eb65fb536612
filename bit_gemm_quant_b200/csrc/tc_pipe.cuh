// The ring of the tensor-core W4A16 kernels: its sizes, its bounded waits and
// the issue of one k-block's MMAs.
#pragma once

#include "tc_ptx.cuh"

namespace w4 {
namespace {

constexpr int kThreads = 320;
constexpr int kKB = 64;                      // k per block (one 128-byte swizzle row of bf16)

enum : int {
    kErrWaitTma = 0x101, kErrWaitFullA = 0x102, kErrWaitEmptyTma = 0x103, kErrWaitEmptyDeq = 0x104,
    kErrWaitDone = 0x105, kErrDrain = 0x106
};

// ---------------------------------------------------------------- PTX ----
// Wait for the phase of `bar` with the given parity.  Gives up (returns false)
// when the CTA's abort flag is raised or after `limit` ns, in which case it
// records `code` and raises the abort flag.
__device__ __noinline__ bool wait_bounded(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err, int code,
                                          uint64_t limit)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > limit) {
            *abort_flag = 1;
            atomicCAS(err, 0, code);
            return false;
        }
    }
}

// Drain wait: ignores the abort flag, bounded in time only.
__device__ __noinline__ bool wait_drain(uint64_t *bar, uint32_t parity, int *err)
{
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer() - t0 > kDefaultWaitNs) {
            atomicCAS(err, 0, kErrDrain);
            return false;
        }
    }
    return true;
}

// Bounded wait until both barriers have completed the phase with the given
// parity; each round tests both at once (their latencies overlap).
__device__ __noinline__ bool wait_pair_bounded(uint64_t *a, uint64_t *b, uint32_t parity, volatile int *abort_flag,
                                               int *err, uint64_t limit)
{
    const uint64_t t0 = globaltimer();
    while (true) {
        const bool ra = mbar_test(a, parity), rb = mbar_test(b, parity);
        if (ra && rb) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > limit) {
            *abort_flag = 1;
            atomicCAS(err, 0, kErrWaitFullA);
            return false;
        }
    }
}

// One k-block (four 128 x BN x 16 MMAs, A from tensor memory at a_tmem, B
// from the SW128 descriptor bdesc, accumulate unless acc0 == 0 for the first)
// and its commit to `empty`, with non-blocking tests of the next k-block's
// barriers issued first; returns whether both were complete.
__device__ __forceinline__ bool mma_kblock_test_next(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                     uint32_t acc0, uint64_t *empty, uint64_t *next_a,
                                                     uint64_t *next_b, uint32_t next_parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred pa, pb, p0, p1;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 pa, [%1], %3;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 pb, [%2], %3;\n\t"
        "setp.ne.b32 p0, %8, 0;\n\t"
        "setp.eq.b32 p1, %8, %8;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%4], [%5], %6, %7, p0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%4], [%9], %10, %7, p1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%4], [%11], %12, %7, p1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%4], [%13], %14, %7, p1;\n\t"
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%15];\n\t"
        "and.pred pa, pa, pb;\n\t"
        "selp.u32 %0, 1, 0, pa;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(next_a)), "r"(smem_u32(next_b)), "r"(next_parity), "r"(d_tmem), "r"(a_tmem), "l"(bdesc),
          "r"(idesc), "r"(acc0), "r"(a_tmem + 8), "l"(bdesc + 2), "r"(a_tmem + 16), "l"(bdesc + 4), "r"(a_tmem + 24),
          "l"(bdesc + 6), "r"(smem_u32(empty))
        : "memory");
    return ok != 0;
}

template <int BN>
struct TcCfg {
    static constexpr int kCols = (BN <= 128) ? 256 : 512;               // tensor-memory allocation
    // pipeline depth: as many 32-column A stages as fit beside the accumulator, at most 6 (even)
    static constexpr int kStages = ((kCols - BN) / 32 >= 6) ? 6 : 4;
    static constexpr int kACol0 = BN;                                   // A stages follow the BN fp32 accumulator columns
    static constexpr int kBBytes = BN * 128;                            // activation box bytes
    static constexpr int kCodeBytes = 128 * 32;                         // codes box: 128 channels x 64 k
    static constexpr int kStageBytes = kBBytes + kCodeBytes;            // a multiple of 1024
    static_assert(kACol0 + kStages * 32 <= kCols, "tensor memory overflow");
    static constexpr int kMinBlocks = (BN == 256) ? 1 : 2;
    // kind::f16, fp32 D, bf16 A and B, both K-major, N = BN, M = 128
    static constexpr uint32_t kIdesc =
        (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
};

}  // namespace
}  // namespace w4
