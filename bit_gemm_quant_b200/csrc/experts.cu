// w4a16_experts_gemm for few rows an expert: the weights are streamed once and
// dequantized in registers, tokens sit in the columns of mma.sync.
//
// Mathematics: Y[i] = X[row(i)] . W^[e]^T for the sorted rows i of expert e, with
// w^ = bf16_rne((u - zp) * s16) as everywhere in the library (tc_ptx.cuh has the
// exact three-operation form) and fp32 accumulation.
//
// What bounds it.  A weight is 0.5 + 2/g (+ 0.5/g) bytes, and its
// dequantization 19/8 instructions, 12/8 of them bf16x2 operations, of which an
// SM starts two per clock (measured; fp32 FMAs start four): 256 weights take 6
// clocks at least, 12.0e12 weights/s on 148 SMs, the same as the 12.6e12 that
// HBM delivers.  The kernel runs about 3.5 instructions a weight.  Measured for one
// token and 2 of 8 experts [14336, 4096], asymmetric, g = 128 (61 MB, 9.3 us of
// HBM): 26.2 us, of which the copies alone are 13.1 us (kernel start and plan
// 1.3, first copies 2.5) and the dequantization's instructions 9.6 us; 16 tokens
// and 8 of 64 experts [2048, 2048], symmetric, g = 64: 38.1 us (19.3 of HBM).
//   * warps are persistent.  A work item is (unit, tile): up to 8 rows of one
//     expert (the columns of an MMA) and 32 of its channels, two MMA tiles that
//     share the activations (with one tile an item the 16 tokens above took 50 us,
//     with four 61, with two 41 at that stage).  A team of KS warps shares an item, warp j taking the 256-k stages j,
//     j + KS, ...; teams take items in turn.
//   * the codes come by TMA, one box of 32 rows x 256 k (128-byte swizzle) a
//     stage, two stages ahead on the warp's own ring of mbarriers, 128 KB in
//     flight on an SM.  Boxes of 16 rows with 96 of them in flight on an SM fell
//     to 2.5 TB/s (plain copies, no arithmetic; 6.3 TB/s with 48).  The ring runs
//     on from one item to the next, so only the kernel's start waits for memory.
//   * group constants are made once per (channel, group) and stage, lane l making
//     those of channel l, and shared through the warp's slot; their scales (one
//     load) and zero-points are loaded a stage ahead, and asked into L2 when the
//     ring reaches their item.
//   * activations come through L1 (the warps of an SM mostly read the same rows),
//     a stage's 64 bytes of each half in flight before the stage waits for its
//     codes; all CTAs together ask X into L2 at the start.
// The fragment layout is the GEMV's: lane (g, t) = (lane / 4, lane % 4) holds the
// channels g and g + 8 and the 16-byte chunks t and t + 4 of a box, the k-order
// inside an MMA is free, and token g's fragment is the plain 16 bytes of its row.
//
// A team's partial tiles meet in shared memory (two buffers, one named barrier
// per item), summed in warp order by its first warp: results repeat bit for bit.
// Every wait on a copy is bounded; a warp whose wait runs out records a code,
// lets its copies land, and goes on only to meet its team's barriers, with
// nothing stored from then on.
#include "experts.cuh"
#include "tc_ptx.cuh"

namespace w4 {
namespace {

constexpr int kErrExpertsWait = 0x401, kErrExpertsDrain = 0x402;
constexpr int kNW = 8;                               // warps per CTA
constexpr int kCtas = 2;                             // resident CTAs per SM (128 registers a thread)
constexpr int kSK = 256;                             // k per stage: one 128-byte row of codes
constexpr int kC = 2, kRows = 16 * kC;               // channel tiles of an item, its channels
constexpr int kChunk = 8;                            // rows of a unit: the columns of one MMA
constexpr int kR = 2;                                // stages in flight per warp
constexpr int kStageBytes = kRows * 128;
constexpr int kRedBytes = kC * 32 * 16;              // one warp's partial tile
__device__ const uint4 kZeros[4] = {};               // 32 activations behind the end of a row

template <int G>
struct ExpCfg {
    static constexpr int kGroups = kSK / G;
    static constexpr int kConstOff = kNW * kR * kStageBytes;
    static constexpr int kRedOff = kConstOff + kNW * kRows * kGroups * 8;
    static constexpr int kBarOff = kRedOff + 2 * kNW * kRedBytes;
    static constexpr int kPlanOff = kBarOff + (kNW * kR + 1) * 8 + 8;  // + the stall barrier, the failure flag
    static int bytes(int E) { return kPlanOff + (2 * E + 1) * 4 + 1024; }
};
static_assert(kRows == 32, "a lane for each channel of an item");
static_assert(kCtas * (ExpCfg<32>::kPlanOff + 2049 * 4 + 2048) <= 228 * 1024, "shared memory of the resident CTAs");

__device__ __noinline__ bool wait_copy(uint32_t bar, uint32_t parity, uint64_t limit)
{
    auto test = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        return ok != 0;
    };
    const uint64_t t0 = globaltimer();
    while (!test())
        if (globaltimer() - t0 > limit) return false;
    return true;
}

__device__ __forceinline__ bool try_copy(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A group's constants from their slot: (s_hi, s_lo), -(128 + zp) twice.
__device__ __forceinline__ GroupConst unpack_const(uint2 v)
{
    return {__byte_perm(v.x, 0, 0x1010), __byte_perm(v.x, 0, 0x3232), v.y};
}

// The plan in shared memory: off[0..E], clamped to [0, P], and upto[e], the
// number of units of the experts 0 .. e.
struct SharedPlan {
    const int *off, *upto;
    int E;
};

// Unit number `unit`, found by the whole warp: first the block of 32 experts,
// then the expert.  The unit must exist.
__device__ __forceinline__ ExpertUnit lookup(const SharedPlan &p, int unit, int chunk)
{
    const int lane = threadIdx.x & 31;
    int base = 0;
    if (p.E > 32) base = 32 * (__ffs(__ballot_sync(0xffffffffu, unit < p.upto[min(32 * lane + 31, p.E - 1)])) - 1);
    const int e = base + __ffs(__ballot_sync(0xffffffffu, unit < p.upto[min(base + lane, p.E - 1)])) - 1;
    const int first = (unit - (e > 0 ? p.upto[e - 1] : 0)) * chunk;
    const int lo = p.off[e], n = p.off[e + 1] - lo;
    return {e, lo + first, min(chunk, n - first)};
}

template <int G, int MODE>
__global__ void __launch_bounds__(kNW * 32, kCtas)
experts_kernel(const __grid_constant__ CUtensorMap tmap_q, const __nv_bfloat16 *__restrict__ X, int N, int K,
               const unsigned short *__restrict__ scales, const uint32_t *__restrict__ qzeros,
               __nv_bfloat16 *__restrict__ Y, int KS, int *err, uint64_t wait_ns, ExpertPlan plan)
{
    using Cfg = ExpCfg<G>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int NG = K / G, ZW = (NG + 7) >> 3, NS = (K + kSK - 1) / kSK;
    const int tiles = (N + kRows - 1) / kRows;
    const uint64_t limit = wait_limit_of(wait_ns);

    uint8_t *ring = smem + warp * kR * kStageBytes;
    uint2 *cslot = (uint2 *)(smem + Cfg::kConstOff) + warp * kRows * Cfg::kGroups;
    const uint32_t ring_s = smem_u32(ring);
    const uint32_t bar0 = smem_u32(smem + Cfg::kBarOff) + warp * kR * 8;
    const uint32_t stall_bar = smem_u32(smem + Cfg::kBarOff) + kNW * kR * 8;
    volatile int *failed = (volatile int *)(smem + Cfg::kBarOff + (kNW * kR + 1) * 8);
    int *off = (int *)(smem + Cfg::kPlanOff), *upto = off + plan.E + 1;

    if (lane == 0) {
        for (int s = 0; s < kR; ++s) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar0 + 8 * s));
        if (warp == 0) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(stall_bar));
            *failed = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmap_q) : "memory");
    }
    pdl_wait();
    pdl_launch_dependents();

    // the rows of X into L2, a slice by every CTA, before the codes fill the queues to memory (unless X has
    // more rows than the plan: most of it is somebody else's then)
    if (threadIdx.x == 32 && (!plan.order || plan.R <= plan.P)) {
        const size_t all = (size_t)min(plan.R, plan.P) * K, part = (all + gridDim.x - 1) / gridDim.x;
        const size_t from = part * blockIdx.x;
        if (from < all) prefetch_l2(X + from, min(part, all - from) * 2);
    }
    // the plan: offsets, then the units' running count by the first warp
    for (int e = threadIdx.x; e <= plan.E; e += kNW * 32) off[e] = min(max(plan.offsets[e], 0), plan.P);
    __syncthreads();
    if (warp == 0) {
        int sum = 0;
        for (int e0 = 0; e0 < plan.E; e0 += 32) {
            const int e = e0 + lane;
            int n = e < plan.E ? (max(off[e + 1] - off[e], 0) + kChunk - 1) / kChunk : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, n, d);
                if (lane >= d) n += v;
            }
            if (e < plan.E) upto[e] = sum + n;
            sum += __shfl_sync(0xffffffffu, n, 31);
        }
    }
    __syncthreads();
    const SharedPlan sp = {off, upto, plan.E};
    const int units = upto[plan.E - 1];

    const int team = warp / KS, j = warp - team * KS;  // this warp is number j of its team
    const int teams_cta = kNW / KS, step = gridDim.x * teams_cta;
    const int step_u = step / tiles, step_t = step - step_u * tiles;
    // (neighbouring items go to different CTAs, so that a last, partial round spreads over all SMs)
    const int item0 = team * gridDim.x + blockIdx.x, unit0 = item0 / tiles, tile0 = item0 - unit0 * tiles;
    auto advance = [&](int &unit, int &tile) {         // to the team's next item
        unit += step_u;
        tile += step_t;
        if (tile >= tiles) {
            tile -= tiles;
            ++unit;
        }
    };

    // ---- the ring: the position of the copies runs R stages ahead ----
    int is_unit = j < NS ? unit0 : units, is_tile = tile0, is_stage = j;   // (a warp beyond the stages copies nothing)
    int is_row = 0;                                    // the item's first row of the code map
    int issued = 0;                                    // stages issued so far
    auto enter_item = [&]() {                          // by the whole warp
        if (is_unit < units) is_row = lookup(sp, is_unit, kChunk).expert * N + is_tile * kRows;
    };
    auto prefetch_consts = [&]() {                     // the item's scales and zero-points, HBM -> L2
        if (is_unit < units && j == 0 && lane == 1) {
            const int rows = min(kRows, N - is_tile * kRows);
            prefetch_l2(scales + (size_t)is_row * NG, (size_t)rows * NG * 2);
            if (MODE == W4_ASYM) prefetch_l2(qzeros + (size_t)is_row * ZW, (size_t)rows * ZW * 4);
        }
    };
    auto issue_next = [&]() {                          // by the whole warp
        if (is_unit >= units) return;
        if (lane == 0) {
            const uint32_t s = (uint32_t)issued % kR;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("mbarrier.arrive.expect_tx.relaxed.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar0 + 8 * s),
                         "r"(kStageBytes)
                         : "memory");
            asm volatile(
                "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
                "[%2];" ::"r"(ring_s + s * kStageBytes),
                "l"(&tmap_q), "r"(bar0 + 8 * s), "r"(is_stage * 32), "r"(is_row)
                : "memory");
        }
        ++issued;
        is_stage += KS;
        if (is_stage >= NS) {
            is_stage = j;
            advance(is_unit, is_tile);
            enter_item();
            prefetch_consts();
        }
    };

    // ---- scales and zero-points of one stage: lane l holds those of the item's channel l ----
    // (the kGroups scales of a stage are one load where rows of scales are whole stages, and their
    // zero-points lie in one word)
    constexpr int kGroups = Cfg::kGroups;
    const bool whole = NG % kGroups == 0 && (uintptr_t)scales % (2 * kGroups) == 0;
    uint32_t sv[kGroups / 2], zv = 0;
    auto load_consts = [&](int row0, int rows, int stage) {   // row0: in the arrays; rows: valid ones
#pragma unroll
        for (int u = 0; u < kGroups / 2; ++u) sv[u] = 0;
        if (lane >= rows) return;
        const int j0 = stage * kGroups;
        const unsigned short *p = scales + (size_t)(row0 + lane) * NG + j0;
        if (whole) {
            if constexpr (kGroups == 2) sv[0] = __ldg((const uint32_t *)p);
            if constexpr (kGroups == 4) {
                const uint2 v = __ldg((const uint2 *)p);
                sv[0] = v.x;
                sv[1] = v.y;
            }
            if constexpr (kGroups == 8) {
                const uint4 v = __ldg((const uint4 *)p);
                sv[0] = v.x;
                sv[1] = v.y;
                sv[2] = v.z;
                sv[3] = v.w;
            }
        } else {
#pragma unroll
            for (int u = 0; u < kGroups; ++u)
                if (j0 + u < NG) sv[u / 2] |= (uint32_t)__ldg(p + u) << (16 * (u & 1));
        }
        if (MODE == W4_ASYM) zv = __ldg(qzeros + (size_t)(row0 + lane) * ZW + (j0 >> 3));
    };

    const uint32_t magic = 0x43004300u;               // bf16x2 of (128, 128)
    const int offA = g * 128 + ((t ^ g) << 4);
    const int lane_gl = G == 128 ? 0 : G == 64 ? (t >> 1) : t;
    const uint2 *clane = cslot + g + kRows * lane_gl;
    bool ok = true;
    int used = 0, parity = 0;                          // stages consumed; the reduction buffer
    ExpertUnit u = {0, 0, 0};
    int r0 = 0, row0 = 0, xr = 0;                      // xr: the row of X of this lane's token
    int unit = unit0, tile = tile0;
    if (unit < units) {
        // what the first stage needs, in the order of the latencies behind it
        u = lookup(sp, unit, kChunk);
        r0 = tile * kRows;
        row0 = u.expert * N + r0;
        const int sorted = u.row0 + min(g, u.rows - 1);
        xr = plan.order ? __ldg(plan.order + sorted) : sorted;
        is_row = row0;
        if (j < NS) load_consts(row0, N - r0, j);
        for (int s = 0; s < kR; ++s) issue_next();
    }
    while (unit < units) {
        // the next item (its first constants are loaded during this one's last stage)
        ExpertUnit nu = u;
        int nr0 = 0, nrow0 = 0, nxr = 0;
        advance(unit, tile);
        const bool more = unit < units;
        if (more) {
            nu = lookup(sp, unit, kChunk);
            nr0 = tile * kRows;
            nrow0 = nu.expert * N + nr0;
            const int sorted = nu.row0 + min(g, nu.rows - 1);
            nxr = plan.order ? __ldg(plan.order + sorted) : sorted;
        }
        const __nv_bfloat16 *xrow = X + (size_t)min(max(xr / plan.top_k, 0), plan.R - 1) * K;

        float acc[kC][4];
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;

        for (int st = j; st < NS && ok; st += KS) {
            // the activations of the stage, all in flight before anything waits: this lane's 32 elements of
            // each half.  In a stage whose end lies behind K the codes and constants are 0 there; so are the
            // activations, for an infinity among the row's own times 0 would be NaN.
            uint4 x[8];
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
                const int k = st * kSK + odd * 128 + 32 * t;
                const uint4 *p = k < K ? (const uint4 *)(xrow + k) : kZeros;
#pragma unroll
                for (int w = 0; w < 4; ++w) x[4 * odd + w] = __ldg(p + w);
            }
            __syncwarp();                              // every lane is done with the previous stage's constants
            // (nothing has looked at the loaded words before: the loads had a stage's time)
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                const uint32_t zp = MODE == W4_ASYM ? (zv >> (4 * ((st * kGroups + q) & 7))) & 15u : 8u;
                const GroupConst gc = group_const((unsigned short)(sv[q / 2] >> (16 * (q & 1))), zp);
                cslot[lane + 32 * q] = make_uint2(__byte_perm(gc.shi, gc.slo, 0x5410), gc.z);
            }
            if (st + KS < NS) load_consts(row0, N - r0, st + KS);
            else if (more) load_consts(nrow0, N - nr0, j);
            __syncwarp();
            const uint32_t s = (uint32_t)used % kR, ph = ((uint32_t)used / kR) & 1u;
            const bool stall = used == 0 && stalls_first_wait(wait_ns);   // failure-path tests only
            if (!__all_sync(0xffffffffu, stall ? wait_copy(stall_bar, 0u, limit)
                                               : try_copy(bar0 + 8 * s, ph) || wait_copy(bar0 + 8 * s, ph, limit))) {
                ok = false;
                break;
            }
            const uint8_t *box = ring + s * kStageBytes;
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
                uint4 wa[kC], wb[kC];
                GroupConst ca[kC], cb[kC];
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const uint8_t *cp = box + c * 2048 + (offA ^ (odd * 64));
                    wa[c] = *(const uint4 *)cp;
                    wb[c] = *(const uint4 *)(cp + 8 * 128);
                    const uint2 *cc = clane + kRows * (odd * 128 / G) + 16 * c;
                    ca[c] = unpack_const(cc[0]);
                    cb[c] = unpack_const(cc[8]);
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint4 xw = x[4 * odd + w];
#pragma unroll
                    for (int c = 0; c < kC; ++c) {
                        const uint32_t qa = w == 0 ? wa[c].x : w == 1 ? wa[c].y : w == 2 ? wa[c].z : wa[c].w;
                        const uint32_t qb = w == 0 ? wb[c].x : w == 1 ? wb[c].y : w == 2 ? wb[c].z : wb[c].w;
                        const uint32_t a0 = dequant_pair(qa, 0, ca[c], magic), b0 = dequant_pair(qb, 0, cb[c], magic);
                        const uint32_t a1 = dequant_pair(qa, 1, ca[c], magic), b1 = dequant_pair(qb, 1, cb[c], magic);
                        const uint32_t a2 = dequant_pair(qa, 2, ca[c], magic), b2 = dequant_pair(qb, 2, cb[c], magic);
                        const uint32_t a3 = dequant_pair(qa, 3, ca[c], magic), b3 = dequant_pair(qb, 3, cb[c], magic);
                        mma_bf16(acc[c], a0, b0, a1, b1, xw.x, xw.y);
                        mma_bf16(acc[c], a2, b2, a3, b3, xw.z, xw.w);
                    }
                }
            }
            ++used;
            __syncwarp();                              // the stage is read: refill it
            issue_next();
        }
        if (!ok && lane == 0) {
            *failed = 1;
            atomicCAS(err, 0, kErrExpertsWait);
        }

        // ---- the team's sum, then Y ----
        bool store = j == 0;
        if (KS > 1) {
            float4 *red = (float4 *)(smem + Cfg::kRedOff + parity * kNW * kRedBytes);
            constexpr int kPer = kRedBytes / 16;
            if (j > 0) {
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    red[warp * kPer + c * 32 + lane] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * KS) : "memory");
            parity ^= 1;
            if (store)
                for (int w = 1; w < KS; ++w)
#pragma unroll
                    for (int c = 0; c < kC; ++c) {
                        const float4 v = red[(warp + w) * kPer + c * 32 + lane];
                        acc[c][0] += v.x;
                        acc[c][1] += v.y;
                        acc[c][2] += v.z;
                        acc[c][3] += v.w;
                    }
        }
        if (store && ok && *failed == 0) {
            const int m0 = 2 * t, m1 = m0 + 1;            // rows of accumulators 0/2 and 1/3
            __nv_bfloat16 *y0 = Y + (size_t)(u.row0 + m0) * N, *y1 = y0 + N;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int nA = r0 + 16 * c + g, nB = nA + 8;
                if (m0 < u.rows && nA < N) y0[nA] = __float2bfloat16_rn(acc[c][0]);
                if (m1 < u.rows && nA < N) y1[nA] = __float2bfloat16_rn(acc[c][1]);
                if (m0 < u.rows && nB < N) y0[nB] = __float2bfloat16_rn(acc[c][2]);
                if (m1 < u.rows && nB < N) y1[nB] = __float2bfloat16_rn(acc[c][3]);
            }
        }
        u = nu;
        r0 = nr0;
        row0 = nrow0;
        xr = nxr;
    }
    if (lane == 0)                                     // copies still in flight (a wait ran out): let them land
        for (int i = used; i < issued; ++i)
            if (!wait_copy(bar0 + 8 * (i % kR), ((uint32_t)i / kR) & 1u, kDefaultWaitNs)) atomicCAS(err, 0, kErrExpertsDrain);
}

template <int G, int MODE>
cudaError_t launch_g(const CUtensorMap &map, const void *X, const ExpertPlan &plan, int64_t N, int64_t K,
                     const void *scales, const uint32_t *qzeros, void *Y, int *err, cudaStream_t stream)
{
    using Cfg = ExpCfg<G>;
    static std::atomic<bool> attr_done[kMaxDevices];
    auto kern = experts_kernel<G, MODE>;
    const cudaError_t e = set_smem_attr(kern, Cfg::bytes(1024), attr_done);
    if (e != cudaSuccess) return e;
    // One wave of resident CTAs.  With fewer items than warps, enough warps to an
    // item for most of them to have work; with one to three rounds of items, two,
    // so that the last round is shorter.  Measured, us with KS = 1 / 2 / 4 / 8: 2 of
    // 8 experts [14336, 4096] 31.4 / 28.4 / 26.7 / 27.2; 16 tokens, 8 of 64 [2048,
    // 2048] 42.3 / 38.4 / 39.2 / 43.9; 40 tokens, 8 of 128 [1536, 4096] 103 / 103 /
    // 107 / 117; 2 tokens, 8 of 128 [768, 2048] 16.6 / 10.3 / 9.7 / 9.2.
    const int64_t most = max_units(plan.P, plan.E, kChunk) * ((N + kRows - 1) / kRows);
    const int64_t stages = (K + kSK - 1) / kSK, warps = (int64_t)kNumSMs * kCtas * kNW;
    int KS = most < 3 * warps && stages > 1 ? 2 : 1;
    while (KS < kNW && most * KS * 5 < warps * 4 && KS * 2 <= stages) KS *= 2;
    const int64_t want = (most * KS + kNW - 1) / kNW;
    const unsigned grid = (unsigned)(want < kNumSMs * kCtas ? want : kNumSMs * kCtas);
    return launch_pdl(kern, dim3(grid), dim3(kNW * 32), Cfg::bytes(plan.E), stream, map, (const __nv_bfloat16 *)X,
                      (int)N, (int)K, (const unsigned short *)scales, qzeros, (__nv_bfloat16 *)Y, KS, err,
                      wait_limit_ns(), plan);
}

}  // namespace

cudaError_t launch_experts_stream(const void *X, const ExpertPlan &plan, int64_t N, int64_t K, const uint32_t *qweight,
                                  const void *scales, const uint32_t *qzeros, int group, int mode, void *Y,
                                  cudaStream_t stream)
{
    int *err = device_error_word();
    EncodeTiledFn enc = encode_fn();
    if (!err || !enc) return cudaErrorUnknown;
    // the codes of all experts as 32-bit words [E * N][K / 8]; a box is 32
    // channels x 32 words (256 k), zero behind the ends
    CUtensorMap map;
    const cuuint64_t gdim[2] = {(cuuint64_t)(K / 8), (cuuint64_t)(plan.E * N)};
    const cuuint64_t gstride[1] = {(cuuint64_t)K / 2};
    const cuuint32_t box[2] = {32u, (cuuint32_t)kRows}, estride[2] = {1u, 1u};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint32_t *>(qweight), gdim, gstride, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    switch (group * 2 + mode) {
    case 32 * 2 + W4_SYM: return launch_g<32, W4_SYM>(map, X, plan, N, K, scales, qzeros, Y, err, stream);
    case 32 * 2 + W4_ASYM: return launch_g<32, W4_ASYM>(map, X, plan, N, K, scales, qzeros, Y, err, stream);
    case 64 * 2 + W4_SYM: return launch_g<64, W4_SYM>(map, X, plan, N, K, scales, qzeros, Y, err, stream);
    case 64 * 2 + W4_ASYM: return launch_g<64, W4_ASYM>(map, X, plan, N, K, scales, qzeros, Y, err, stream);
    case 128 * 2 + W4_SYM: return launch_g<128, W4_SYM>(map, X, plan, N, K, scales, qzeros, Y, err, stream);
    case 128 * 2 + W4_ASYM: return launch_g<128, W4_ASYM>(map, X, plan, N, K, scales, qzeros, Y, err, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace w4
