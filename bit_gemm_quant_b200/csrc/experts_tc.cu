// w4a16_experts_gemm for many rows an expert: the tensor-core kernel by expert.
//
// Mathematics: Y[i] = X[i] . W^[e]^T for the sorted rows i of expert e, w^ =
// bf16_rne((u - zp) * s16), fp32 accumulation.  Rows that come through the
// plan's order are moved into sorted order once, into the caller's workspace: a
// product's CTAs read each row N / 128 times in boxes of BN rows, and TMA's
// four-row gather instead, at about 50 clocks an instruction, held the product
// to 232 TFLOP/s (8192 tokens, 2 of 8 experts of [14336, 4096]).
//
// The pipeline is w4a16_gemm's (gemm_tc.cu): D[128 channels, BN rows] in tensor
// memory, A = the dequantized weights, written into tensor memory by eight warps,
// B = the rows by TMA, one warp for the copies, one thread for the MMAs.  CTA
// (x, y) owns the channels 128 x .. of one expert and up to BN of that expert's
// rows (unit y of the plan); N and the channels are per expert.  A box's rows
// past the unit's are other rows of X: the MMAs leave them out from the next
// multiple of 16 on, and their accumulator columns are never stored; a whole tile
// of rows leaves by TMA, a ragged one by plain stores.
//
// What bounds it.  With few rows an expert, the dequantization: 157 instructions
// per warp and k-block (2.4 a weight), whatever BN is, in whose way the MMA
// issuer has to find its slots (about 125 clocks an MMA of 64 rows, 45 alone).  So
// group size and mode are template parameters here, the loop is unrolled over the
// ring, and a group's scale and zero-point word are loaded a round ahead and
// looked at only where they are used.  8 of 8 experts [14336, 4096] with 8 rows
// each: 101 us (37.6 of HBM), a chain of waits more than any one rate: 97 of 105
// without the MMAs, 90 without the arithmetic, 82 without both; and 896 tiles
// take four rounds of 296 CTAs.  With many rows, copies (576 clocks a k-block of 256
// rows at 64 bytes a clock) and MMAs (512) alike: 8192 tokens, 2 of 8 experts:
// 1645 to 1710 us on several B200s, 1125 to 1170 TFLOP/s, 81 to 84% of the sustained
// cuBLAS rate (1828 with w4a16_gemm's loop by expert).
#include "experts.cuh"
#include "tc_pipe.cuh"

namespace w4 {
namespace {

// wait_pair_bounded for an issuer that mostly waits: its tests suspend the
// thread, and so leave the issue slots to the dequantizing warps.
__device__ __noinline__ bool wait_pair_sleeping(uint64_t *a, uint64_t *b, uint32_t parity, volatile int *abort_flag,
                                                int *err, uint64_t limit)
{
    return wait_bounded(a, parity, abort_flag, err, kErrWaitFullA, limit) &&
           wait_bounded(b, parity, abort_flag, err, kErrWaitTma, limit);
}

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok;
}

// mma_kblock_test_next for a whole warp: every lane runs it with the same
// arguments, `leader`'s lane issues.  In a loop that one thread runs alone the
// compiler has to move every operand of an MMA into uniform registers (four
// moves an MMA, measured); in one that the warp runs together they stay there.
__device__ __forceinline__ bool mma_kblock_warp(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                                uint32_t idesc, uint32_t acc0, uint32_t empty, uint32_t next_a,
                                                uint32_t next_b, uint32_t next_parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred pa, pb, p0, p1, pl;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 pa, [%1], %3;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 pb, [%2], %3;\n\t"
        "setp.ne.b32 p0, %8, 0;\n\t"
        "setp.eq.b32 p1, %8, %8;\n\t"
        "setp.ne.b32 pl, %16, 0;\n\t"
        "@pl tcgen05.mma.cta_group::1.kind::f16 [%4], [%5], %6, %7, p0;\n\t"
        "@pl tcgen05.mma.cta_group::1.kind::f16 [%4], [%9], %10, %7, p1;\n\t"
        "@pl tcgen05.mma.cta_group::1.kind::f16 [%4], [%11], %12, %7, p1;\n\t"
        "@pl tcgen05.mma.cta_group::1.kind::f16 [%4], [%13], %14, %7, p1;\n\t"
        "@pl tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%15];\n\t"
        "and.pred pa, pa, pb;\n\t"
        "selp.u32 %0, 1, 0, pa;\n\t}"
        : "=r"(ok)
        : "r"(next_a), "r"(next_b), "r"(next_parity), "r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc0),
          "r"(a_tmem + 8), "l"(bdesc + 2), "r"(a_tmem + 16), "l"(bdesc + 4), "r"(a_tmem + 24), "l"(bdesc + 6),
          "r"(empty), "r"(leader)
        : "memory");
    return __all_sync(0xffffffffu, ok != 0);
}

// Shared memory: a ring of kStages boxes of X (a k-block each, as deep as the
// ring of A stages in tensor memory) and one of kCodes boxes of codes (four
// k-blocks each: 128 bytes of a row.  TMA spends two clocks on a row of 32 bytes
// as on one of 128; with a box a k-block, as w4a16_gemm has, rows of codes were a
// third to two thirds of the copies' time, and the copies what bounded the tile;
// a third box of codes gains nothing).
template <int BN>
struct ExpTcCfg {
    using C = TcCfg<BN>;
    static constexpr int kCodes = 2;
    static constexpr int kCodeBytes = 128 * 128;
    static constexpr int kCodeOff = C::kStages * C::kBBytes;
    static constexpr int kBarOff = kCodeOff + kCodes * kCodeBytes;
    static constexpr int kBytes = kBarOff + 256 + 1024;                // + alignment slack
    static_assert((3 * C::kStages + 2 * kCodes + 2) * 8 + 8 <= 256 && kBytes <= 227 * 1024, "shared memory");
};

template <int BN, int G, int MODE>
__global__ void __launch_bounds__(kThreads, TcCfg<BN>::kMinBlocks)
experts_tc_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_q,
                  const __grid_constant__ CUtensorMap tmap_y, int y_tma, int N, int K,
                  const unsigned short *__restrict__ scales, const uint32_t *__restrict__ qzeros,
                  __nv_bfloat16 *__restrict__ Y, int *err, uint64_t wait_ns, ExpertPlan plan)
{
    using C = TcCfg<BN>;
    using Cfg = ExpTcCfg<BN>;
    constexpr int kStages = C::kStages, kCodes = Cfg::kCodes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sB = smem;                                               // kStages x BN rows of X
    uint64_t *full_b = (uint64_t *)(smem + Cfg::kBarOff);
    uint64_t *full_a = full_b + kStages;
    uint64_t *empty = full_a + kStages;
    uint64_t *full_c = empty + kStages;
    uint64_t *empty_c = full_c + kCodes;
    uint64_t *done = empty_c + kCodes;
    uint64_t *stall = done + 1;                         // a barrier nothing completes (failure tests)
    uint32_t *tmem_slot = (uint32_t *)(stall + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    const uint64_t limit = wait_limit_of(wait_ns);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * 128, nkb = (K + kKB - 1) / kKB;

    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmap_x) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmap_q) : "memory");
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full_b[s], 1);
            mbar_init(&full_a[s], 4);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kCodes; ++s) {
            mbar_init(&full_c[s], 1);
            mbar_init(&empty_c[s], 8);
        }
        mbar_init(done, 1);
        mbar_init(stall, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(tmem_slot, C::kCols);
    pdl_wait();                                                        // the plan is there
    const ExpertUnit unit = find_unit(plan, blockIdx.y, BN);           // (every warp finds the same)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (not before this CTA has its tensor memory: a kernel started beside this one could take it, and waits
    // for this one's end)
    pdl_launch_dependents();
    const uint32_t tmem = *tmem_slot;
    if (unit.rows == 0) {                                              // fewer units than the grid has room for
        __syncthreads();
        if (warp == 1) tmem_dealloc(tmem, C::kCols);
        return;
    }
    const int m0 = unit.row0, q0 = unit.expert * N + n0;
    const bool tile_store = y_tma && unit.rows == BN;                  // no other expert's rows in the tile

    if (warp == 0) {
        // ------------------------------------------------ TMA producer --
        // One thread feeds both rings, each as its barrier allows: neither waits for the other's.  (It
        // polls.  A sleep of 40 ns between two rounds cost 2 to 4% at 1024 rows an expert; boxes of codes
        // asked for by the last warp that had read the one before, 1 to 2%.)
        if (lane == 0) {
            const int ncb = (nkb + 3) >> 2;
            int ix = 0, ic = 0;                       // boxes of X and of codes issued so far
            uint64_t t0 = 0;
            while (ix < nkb || ic < ncb) {
                bool moved = false;
                if (ic < ncb && mbar_test(&empty_c[ic % kCodes], ((ic / kCodes) & 1) ^ 1)) {
                    uint64_t *bar = &full_c[ic % kCodes];
                    mbar_arrive_expect_tx(bar, Cfg::kCodeBytes);
                    tma_load_2d(smem + Cfg::kCodeOff + (ic % kCodes) * Cfg::kCodeBytes, &tmap_q, bar, ic * 32, q0);
                    ++ic;
                    moved = true;
                }
                if (ix < nkb && mbar_test(&empty[ix % kStages], ((ix / kStages) & 1) ^ 1)) {
                    uint64_t *bar = &full_b[ix % kStages];
                    mbar_arrive_expect_tx(bar, C::kBBytes);
                    tma_load_2d(sB + (ix % kStages) * C::kBBytes, &tmap_x, bar, ix * kKB, m0);
                    ++ix;
                    moved = true;
                }
                if (moved) {
                    t0 = 0;
                } else {
                    if (*abort_flag) break;
                    const uint64_t now = globaltimer();
                    t0 = t0 == 0 ? now : t0;
                    if (now - t0 > limit) {
                        *abort_flag = 1;
                        atomicCAS(err, 0, kErrWaitEmptyTma);
                        break;
                    }
                }
            }
            // drain: every issued copy must have landed before the CTA may exit
            for (int i = max(0, ix - kStages); i < ix; ++i) wait_drain(&full_b[i % kStages], (i / kStages) & 1, err);
            for (int i = max(0, ic - kCodes); i < ic; ++i) wait_drain(&full_c[i % kCodes], (i / kCodes) & 1, err);
        }
    } else if (warp == 1) {
        // ------------------------------------------------- MMA issuer ---
        const uint32_t leader = elect_one();
        const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
        // an MMA as wide as the unit's rows, in steps of 16 (N / 8 stands in the descriptor from bit 17 on):
        // 8 experts [14336, 4096], 64 rows each: 129 -> 113 us, 1024: 785 -> 760.  (X by boxes of the rows
        // that are there, 16 to 64 at a time, was slower: 3 to 40 %.)
        const uint32_t idesc = __shfl_sync(
            0xffffffffu, (C::kIdesc & ~(0x3Fu << 17)) | ((uint32_t)((unit.rows + 15) / 16 * 2) << 17), 0);
        const uint64_t bdesc0 = desc_k_sw128(smem_u32(sB));
        const uint32_t fa0 = smem_u32(full_a), fb0 = smem_u32(full_b), em0 = smem_u32(empty);
        bool ready = false, stop = false;
        uint32_t ph = 0;
        const int nmma = stalls_last_mma(wait_ns) ? nkb - 1 : nkb;     // (failure-path tests only)
        for (int i0 = 0; i0 < nmma && !stop; i0 += kStages, ph ^= 1u) {
#pragma unroll
            for (int st = 0; st < kStages; ++st) {
                const int i = i0 + st;
                if (i >= nmma) break;
                if (!ready)
                    ready = __all_sync(0xffffffffu,
                                       wait_pair_sleeping(&full_a[st], &full_b[st], ph, abort_flag, err, limit));
                if (!ready) {
                    stop = true;
                    break;
                }
                tc_fence_after();
                // the next k-block's stage and phase (the last k-block re-tests its own, complete, barriers)
                const int s1 = (st + 1 == kStages) ? 0 : st + 1;
                const uint32_t ph1 = (st + 1 == kStages) ? (ph ^ 1u) : ph;
                const bool last = i + 1 == nmma;
                ready = mma_kblock_warp(leader, tmem_u, tmem_u + C::kACol0 + st * 32,
                                        bdesc0 + (uint64_t)((st * C::kBBytes) >> 4), idesc, i > 0 ? 1u : 0u,
                                        em0 + 8 * st, fa0 + 8 * (last ? st : s1), fb0 + 8 * (last ? st : s1),
                                        last ? ph : ph1);
            }
        }
        if (nmma < nkb && !stop) stop = !wait_bounded(stall, 0, abort_flag, err, kErrWaitFullA, limit / 4);
        if (stop) __threadfence_block();               // the abort flag is up before `done` completes
        __syncwarp();
        if (leader) mma_commit(done);
        __syncwarp();
        wait_drain(done, 0, err);       // no MMA may still be running when tensor memory is freed
        __syncwarp();
    } else {
        // ------------------------------------- dequantize, then epilogue --
        const int q = warp & 3;                      // tensor-memory lane quarter of this warp
        const int h = (warp - 2) >> 2;               // k-block parity handled by this warp
        const int r = 32 * q + lane;
        const int n = n0 + r;
        const bool okn = n < N;
        const int NG = K / G, ZW = (NG + 7) >> 3;
        const unsigned short *srow = scales + (size_t)(okn ? q0 + r : 0) * NG;
        const uint32_t *zrow = MODE == W4_ASYM ? qzeros + (size_t)(okn ? q0 + r : 0) * ZW : nullptr;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16);
        uint32_t magic;                              // 0x43004300, opaque to the compiler
        asm volatile("mov.b32 %0, 0x43004300;" : "=r"(magic));

        // Visit v of this warp is k-block h + 2 v: groups j0 + v * kStep (and the next, when g = 32).
        // Its scales come kU visits ahead; a zero-point word holds the groups of 8 / kStep visits, and the
        // next word is loaded when one is begun.
        constexpr int kU = kStages / 2, kStep = 128 / G;
        static_assert(kStages % 2 == 0, "the dequantizing warps step two stages at a time");
        const int j0 = G == 128 ? 0 : h * (64 / G);
        auto scale = [&](int j) { return okn && j < NG ? __ldg(srow + j) : (unsigned short)0; };
        auto zword = [&](int w) { return MODE == W4_ASYM && w < ZW ? __ldg(zrow + w) : 0u; };
        unsigned short s0[kU], s1[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            s0[u] = scale(j0 + u * kStep);
            s1[u] = G == 32 ? scale(j0 + u * kStep + 1) : (unsigned short)0;
        }
        uint32_t zcur = zword(0), znext = zword(1);

        bool ok = true;
        uint32_t ph = 0, cph = 0;
        int cs = 0;                                  // ring place and phase of this warp's box of codes
        const uint8_t *codes = smem + Cfg::kCodeOff + r * 128;
        for (int v0 = 0; h + 2 * v0 < nkb && ok; v0 += kU, ph ^= 1u) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int v = v0 + u;
                if (h + 2 * v >= nkb || !ok) break;
                const int s = h + 2 * u;
                const int j = j0 + v * kStep;
                if (MODE == W4_ASYM && v > 0 && (v & (8 / kStep - 1)) == 0) {
                    zcur = znext;
                    znext = zword((j >> 3) + 1);
                }
                const GroupConst c0 = group_const(s0[u], MODE == W4_ASYM ? (zcur >> (4 * (j & 7))) & 15u : 8u);
                const GroupConst c1 =
                    G == 32 ? group_const(s1[u], MODE == W4_ASYM ? (zcur >> (4 * ((j + 1) & 7))) & 15u : 8u) : c0;
                // the codes (a box holds two k-blocks of each warp), and the stage's tensor-memory columns:
                // the MMAs of its previous round are done
                // (the first wait targets a barrier that nothing completes in the failure-path tests)
                uint64_t *fc = (v == 0 && stalls_first_wait(wait_ns)) ? stall : &full_c[cs];
                const uint32_t fph = fc == stall ? 0u : cph;
                if (!__all_sync(0xffffffffu,
                                ((v & 1) || mbar_try_wait(fc, fph) ||
                                 wait_bounded(fc, fph, abort_flag, err, kErrWaitTma, limit)) &&
                                    (mbar_try_wait(&empty[s], ph ^ 1) ||
                                     wait_bounded(&empty[s], ph ^ 1, abort_flag, err, kErrWaitEmptyDeq, limit)))) {
                    ok = false;
                    break;
                }
                // this channel's 64 codes: two 16-byte chunks of row r of the box (128-byte swizzle)
                const uint8_t *row = codes + cs * Cfg::kCodeBytes;
                const int chunk = 2 * h + 4 * (v & 1);
                const uint4 w0 = *(const uint4 *)(row + ((chunk ^ (r & 7)) << 4));
                const uint4 w1 = *(const uint4 *)(row + (((chunk + 1) ^ (r & 7)) << 4));
                s0[u] = scale(j + kU * kStep);
                if (G == 32) s1[u] = scale(j + kU * kStep + 1);
                uint32_t a[32];
                const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w};
                const uint32_t wb[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[4 * w + i] = dequant_pair(wa[w], i, c0, magic);
                        a[16 + 4 * w + i] = dequant_pair(wb[w], i, c1, magic);
                    }
                tmem_st32(lane_addr + C::kACol0 + s * 32, a);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&full_a[s]);
                    if (v & 1) mbar_arrive(&empty_c[cs]);
                }
                if ((v & 1) && ++cs == kCodes) {
                    cs = 0;
                    cph ^= 1u;
                }
            }
        }

        // ---- epilogue: accumulator -> Y ----
        // (`done` also completes when the issuer gave up: the flag, raised before, tells)
        const bool have = __all_sync(0xffffffffu, ok && wait_bounded(done, 0, abort_flag, err, kErrWaitDone, limit) &&
                                                      *abort_flag == 0);
        tc_fence_after();
        // The two warps of a lane quarter take 16 rows of the tile in turn.
        constexpr int CH = 16;
        if (have) {
            // a whole tile goes through the (now idle) stage buffers, stored below by one TMA; every warp
            // store writes 64 contiguous bytes
            __nv_bfloat16 *ysm = (__nv_bfloat16 *)smem;
            for (int c = h * CH; c < unit.rows; c += 2 * CH) {
                float acc[CH];
#pragma unroll
                for (int u = 0; u < CH / 8; ++u) tmem_ld8(lane_addr + c + 8 * u, acc + 8 * u);
                tmem_wait_ld();
                if (tile_store) {
#pragma unroll
                    for (int i = 0; i < CH; ++i) ysm[(c + i) * 128 + r] = __float2bfloat16_rn(acc[i]);
                } else {
                    __nv_bfloat16 *y = Y + (size_t)(m0 + c) * N + n;
#pragma unroll
                    for (int i = 0; i < CH; ++i, y += N)
                        if (okn && c + i < unit.rows) *y = __float2bfloat16_rn(acc[i]);
                }
            }
        }
        if (tile_store) {
            // make the tile visible to the TMA unit, then one thread stores it (channels past N are
            // clipped) and waits until shared memory has been read
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (threadIdx.x == 64 && *abort_flag == 0) {
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                                 &tmap_y),
                             "r"(smem_u32(smem)), "r"(n0), "r"(m0)
                             : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::kCols);
}

// The rows of X in sorted order: dst[i] = X[order[i] / top_k] for i < offsets[E],
// 16 bytes a thread and step.
__global__ void __launch_bounds__(256) sort_rows_kernel(const uint4 *X, ExpertPlan plan, int vecs, uint4 *dst)
{
    pdl_wait();
    pdl_launch_dependents();
    const int rows = min(max(plan.offsets[plan.E], 0), plan.P);
    const int64_t total = (int64_t)rows * vecs;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int row = (int)(i / vecs), v = (int)(i - (int64_t)row * vecs);
        dst[i] = X[(int64_t)expert_x_row(plan, row) * vecs + v];
    }
}

struct TcMaps {
    CUtensorMap x, q, y;
    int y_tma;
};

template <int BN, int G, int MODE>
cudaError_t launch_tc(const TcMaps &m, const ExpertPlan &plan, int N, int K, const void *scales, const uint32_t *qzeros,
                      void *Y, int *err, cudaStream_t stream)
{
    constexpr int smem = ExpTcCfg<BN>::kBytes;
    static_assert(smem * 3 > 227 * 1024, "an SM's tensor memory holds two CTAs at most");
    static std::atomic<bool> attr_done[kMaxDevices];
    auto kern = experts_tc_kernel<BN, G, MODE>;
    const cudaError_t e = set_smem_attr(kern, smem, attr_done);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((N + 127) / 128), (unsigned)max_units(plan.P, plan.E, BN));
    return launch_pdl(kern, grid, dim3(kThreads), smem, stream, m.x, m.q, m.y, m.y_tma, N, K,
                      (const unsigned short *)scales, qzeros, (__nv_bfloat16 *)Y, err, wait_limit_ns(), plan);
}

template <int G, int MODE>
cudaError_t launch_tc_bn(int BN, const TcMaps &m, const ExpertPlan &plan, int N, int K, const void *scales,
                         const uint32_t *qzeros, void *Y, int *err, cudaStream_t stream)
{
    switch (BN) {
    case 128: return launch_tc<128, G, MODE>(m, plan, N, K, scales, qzeros, Y, err, stream);
    default: return launch_tc<256, G, MODE>(m, plan, N, K, scales, qzeros, Y, err, stream);
    }
}

}  // namespace

size_t experts_tc_workspace_bytes(int64_t P, int64_t K) { return (size_t)P * K * 2; }

cudaError_t launch_experts_tc(const void *X, ExpertPlan plan, int64_t N, int64_t K, const uint32_t *qweight,
                              const void *scales, const uint32_t *qzeros, int group, int mode, void *Y, void *ws,
                              cudaStream_t stream)
{
    int *err = device_error_word();
    EncodeTiledFn enc = encode_fn();
    if (!err || !enc) return cudaErrorUnknown;
    if (plan.order) {
        const int64_t want = (plan.P * (K / 8) + 255) / 256;
        const unsigned grid = (unsigned)(want < (int64_t)kNumSMs * 16 ? want : (int64_t)kNumSMs * 16);
        const cudaError_t e = launch_pdl(sort_rows_kernel, dim3(grid), dim3(256), 0, stream, (const uint4 *)X, plan,
                                         (int)(K / 8), (uint4 *)ws);
        if (e != cudaSuccess) return e;
        X = ws;
        plan.order = nullptr;
    }
    // Rows of a tile by the rows an expert has on average: a larger tile shares a dequantized weight
    // among more rows, a smaller one has two CTAs on an SM.  (What an MMA computes past an expert's
    // last row is the same with both: at most 15 rows.)  Measured, us with 128 / 256: 8 experts
    // [14336, 4096] at 32 rows each 103 / 146, 64: 107 / 149, 200: 210 / 204, 256: 253 / 246,
    // 1024: 853 / 738; 64 of [2048, 2048] at 32: 67 / 95, 200: 143 / 152, 256: 176 / 175, 1024:
    // 596 / 556; 128 of [768, 2048] at 200: 129 / 137, 300: 179 / 179.  (Tiles of 64 rows are within
    // 2 % of 128's up to 12 rows an expert, on either side, and slower beyond.)
    const int64_t rows = plan.P / plan.E;
    const int BN = rows <= 224 ? 128 : 256;
    TcMaps m;
    const cuuint32_t estride[2] = {1, 1};
    const cuuint64_t gdim[2] = {(cuuint64_t)K, (cuuint64_t)plan.P};
    const cuuint64_t gstride[1] = {(cuuint64_t)K * 2};
    const cuuint32_t box[2] = {(cuuint32_t)kKB, (cuuint32_t)BN};
    if (enc(&m.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(X), gdim, gstride, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    // the codes of all experts as 32-bit words [E * N][K/8]; one box = 128 channels x four 64-wide k-blocks
    const cuuint64_t qdim[2] = {(cuuint64_t)(K / 8), (cuuint64_t)(plan.E * N)};
    const cuuint64_t qstride[1] = {(cuuint64_t)K / 2};
    const cuuint32_t qbox[2] = {32u, 128u};
    if (enc(&m.q, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint32_t *>(qweight), qdim, qstride, qbox, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    m.y = m.x;
    m.y_tma = ((uintptr_t)Y % 16) == 0 && (N * 2) % 16 == 0;
    if (m.y_tma) {
        const cuuint64_t ydim[2] = {(cuuint64_t)N, (cuuint64_t)plan.P};
        const cuuint64_t ystride[1] = {(cuuint64_t)N * 2};
        const cuuint32_t ybox[2] = {128u, (cuuint32_t)BN};
        if (enc(&m.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, Y, ydim, ystride, ybox, estride,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    switch (group * 2 + mode) {
    case 32 * 2 + W4_SYM: return launch_tc_bn<32, W4_SYM>(BN, m, plan, (int)N, (int)K, scales, qzeros, Y, err, stream);
    case 32 * 2 + W4_ASYM: return launch_tc_bn<32, W4_ASYM>(BN, m, plan, (int)N, (int)K, scales, qzeros, Y, err, stream);
    case 64 * 2 + W4_SYM: return launch_tc_bn<64, W4_SYM>(BN, m, plan, (int)N, (int)K, scales, qzeros, Y, err, stream);
    case 64 * 2 + W4_ASYM: return launch_tc_bn<64, W4_ASYM>(BN, m, plan, (int)N, (int)K, scales, qzeros, Y, err, stream);
    case 128 * 2 + W4_SYM: return launch_tc_bn<128, W4_SYM>(BN, m, plan, (int)N, (int)K, scales, qzeros, Y, err, stream);
    case 128 * 2 + W4_ASYM: return launch_tc_bn<128, W4_ASYM>(BN, m, plan, (int)N, (int)K, scales, qzeros, Y, err, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace w4
