// w4_route: the choice of experts for each token and the plan of their rows;
// w4_combine: the weighted sum over a token's experts.
//
// Mathematics (include/w4.h has the exact semantics), per token:
//     score = softmax(logits) or 1 / (1 + exp(-logit)),  choice = score + bias,
//     the top_k largest choices (within the best groups), weight = score /
//     sum of the chosen scores * scale,
// and then a stable counting sort of the T * top_k pairs by expert.
//
// Which of two near choices is larger decides a whole number, so the order has
// to be that of the exact scores; fp32 scores of different logits often round to
// the same value.  Without a bias both scores rise with the logit, and the
// logits themselves are the exact order, for experts and for groups taken by
// their best expert (SIMPLE): exponentials are taken of the chosen logits alone,
// or of all where the softmax's sum is wanted.  Otherwise scores and choices are
// fp64 throughout.  Weights are fp64 up to their one rounding.
//
// One warp chooses for one token: lane l holds the experts l, l + 32, ..., so
// logits are read in whole lines and equal choices can be told apart by index.
// A choice is compared as an integer in the order of the floating values (masked
// experts 0, below every number); its maximum over the warp takes one 32-bit
// reduction, a ballot and a shuffle, and two reductions more only where several
// lanes share the largest (high) word.
//
// The plan of up to kPlanMany pairs needs no scan across CTAs: the CTA of expert e
// reads all ids, counts those below e (where its rows begin) and lists its own
// pairs in order; more pairs are counted and placed by one cluster.  Up to
// kFusedPairs pairs of kFusedWarps tokens the one CTA that chooses also makes the
// plan, each thread ranking one pair against all others in shared memory: one
// launch in place of two.  (57 tokens that way took 11.9 us, against 4.3 in two.)
// What bounds it: latency.  8192 tokens, 8 of 128 experts (4.7 MB, 0.8 us of HBM)
// take 17.4 us, 8.7 of them the choice; 8 of 256 in 8 groups by sigmoid and bias 34;
// one token so, 8.3 us, half of it the fp64 scores.
#include "common.cuh"

#include <cooperative_groups.h>

#include <type_traits>

namespace cg = cooperative_groups;

namespace w4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRouteWarps = 8, kFusedWarps = 16, kFusedPairs = 256;   // one token a warp

struct RouteArgs {
    const void *logits;
    const float *bias;
    int *ids, *pos, *offsets, *order;
    float *weights;
    int64_t T;
    int E, k, f32, sigmoid, groups, keep, group_top, renorm;
    float scale;
    int size, lanes_log2;                                 // of a group: its experts, and log2 of the lanes that look through it
};

// Floating values as unsigned integers of the same order; 0 stands below all of
// them, for -infinity, and 1 below every number, for NaN.  -0 and +0 are equal.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (!(v > -INFINITY)) return v != v;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint64_t order_key(double v)
{
    if (!(v > -INFINITY)) return v != v;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

// The double behind a key above 1.
__device__ __forceinline__ double key_value(uint64_t k)
{
    return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}

// The lowest index among the lanes with the warp's largest key, -1 if every key
// is 0.  Mostly one lane alone has the largest (high) word.
__device__ __forceinline__ int warp_best(uint32_t key, int idx)
{
    const uint32_t best = __reduce_max_sync(kFull, key);
    const unsigned who = __ballot_sync(kFull, key == best);
    if ((who & (who - 1)) == 0) return __shfl_sync(kFull, key ? idx : -1, __ffs(who) - 1);
    return best ? (int)__reduce_min_sync(kFull, key == best ? (unsigned)idx : kFull) : -1;
}

__device__ __forceinline__ int warp_best(uint64_t key, int idx)
{
    const uint32_t hi = (uint32_t)(key >> 32);
    const uint32_t mh = __reduce_max_sync(kFull, hi);
    const unsigned who = __ballot_sync(kFull, hi == mh);
    if ((who & (who - 1)) == 0) return __shfl_sync(kFull, key ? idx : -1, __ffs(who) - 1);
    const uint32_t ml = __reduce_max_sync(kFull, hi == mh ? (uint32_t)key : 0u);
    const uint64_t best = ((uint64_t)mh << 32) | ml;
    return best ? (int)__reduce_min_sync(kFull, key == best ? (unsigned)idx : kFull) : -1;
}

// What a group with the best keys m1 >= m2 is worth, as a key.
__device__ __forceinline__ uint32_t group_key(uint32_t m1, uint32_t, int) { return m1; }
__device__ __forceinline__ uint64_t group_key(uint64_t m1, uint64_t m2, int top)
{
    return top == 2 && m2 > 1 ? order_key(key_value(m1) + key_value(m2)) : m1;
}

template <bool SIMPLE>
struct KeyOf {
    typedef uint64_t type;
};
template <>
struct KeyOf<true> {
    typedef uint32_t type;
};

// exp(v) for v <= 0, without a branch, so that a lane's experts run side by side
// (the library's exp and division one after the other took 750 clocks an
// expert): v = n ln 2 + r with ln 2 in two parts (Cody and Waite), |r| <= 0.35,
// and the Taylor polynomial of degree 14 (its remainder is below 2^-63 e^r).
// Below -708, where 2^n leaves the normal range, 0.
__device__ __forceinline__ double exp_neg(double v)
{
    constexpr double kLn2 = 0.693147180559945309417232121458176568;
    constexpr double kLn2Hi = 0x1.62e42feep-1;       // its leading 32 bits: n times this is exact
    constexpr double kLn2Lo = 1.9082149292705877e-10;   // the rest
    const double a = v < -708.0 ? -708.0 : v;        // (keeps a NaN)
    const double n = rint(a * (1.0 / kLn2));
    const double r = fma(-n, kLn2Lo, fma(-n, kLn2Hi, a));
    double p = 1.0 / 87178291200.0;                  // 1 / 14!
    p = fma(p, r, 1.0 / 6227020800.0);
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    const double two_n = __hiloint2double((1023 + (int)n) << 20, 0);
    return v < -708.0 ? 0.0 : p * two_n;
}

// 1 / d for 1 <= d <= 2: an approximate fp32 reciprocal (2^-22) and two Newton steps.
__device__ __forceinline__ double reciprocal(double d)
{
    float f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"((float)d));
    double y = (double)f;
    y = fma(y, fma(-d, y, 1.0), y);
    return fma(y, fma(-d, y, 1.0), y);
}

__device__ __forceinline__ double sigmoid64(double x)
{
    const double e = exp_neg(-fabs(x)), inv = reciprocal(1.0 + e);
    return x < 0.0 ? e * inv : inv;
}

__device__ __forceinline__ float logit(const RouteArgs &a, int64_t i)
{
    return a.f32 ? __ldg((const float *)a.logits + i) : __bfloat162float(__ldg((const __nv_bfloat16 *)a.logits + i));
}

// The choice for token t by one warp; S >= E / 32 experts per lane, a power of
// two.  `sh`: E + 64 8-byte words of this warp's shared memory (groups only).
// Returns the id that this lane's place j = lane got, and writes ids and weights.
template <int S, bool SIMPLE>
__device__ __forceinline__ int choose(const RouteArgs &a, int64_t t, uint64_t *sh)
{
    typedef typename KeyOf<SIMPLE>::type Key;
    const int lane = threadIdx.x & 31;
    float x[S];
    Key key[S];
    float top = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        x[s] = lane + 32 * s < a.E ? logit(a, t * a.E + lane + 32 * s) : -INFINITY;
        top = fmaxf(top, x[s]);
    }
    double total = 1.0;                                   // one over the softmax's sum, where it is wanted
    double score[SIMPLE ? 1 : S];
    if (!a.sigmoid && (!SIMPLE || !a.renorm)) {
        top = warp_max(top);
        total = 0.0;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const double v = x[s] != -INFINITY ? exp_neg((double)x[s] - (double)top) : 0.0;
            if (!SIMPLE) score[SIMPLE ? 0 : s] = v;
            total += v;
        }
        total = warp_sum(total);
        total = total > 0.0 ? 1.0 / total : 1.0;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (!SIMPLE) score[SIMPLE ? 0 : s] *= total;
    }
    if (!SIMPLE && a.sigmoid) {                           // (outside the loop below: side by side, no branch between)
#pragma unroll
        for (int s = 0; s < S; ++s) score[SIMPLE ? 0 : s] = sigmoid64((double)x[s]);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int e = lane + 32 * s;
        if (SIMPLE) {
            key[s] = (Key)order_key(x[s]);
        } else {
            const double c = score[SIMPLE ? 0 : s] + (a.bias && e < a.E ? (double)__ldg(a.bias + e) : 0.0);
            key[s] = x[s] != -INFINITY ? (Key)order_key(c) : (Key)0;   // (a NaN spoils its own token only)
        }
        if (a.groups > 1 && e < a.E) ((Key *)sh)[e] = key[s];
    }
    if (a.groups > 1) {
        // a group's two best choices, by `per_group` lanes each
        const int size = a.size, per_group = 1 << a.lanes_log2;
        Key *gkey = (Key *)(sh + a.E);
        const int sub = lane & (per_group - 1), first = lane >> a.lanes_log2;
        __syncwarp();
        for (int g0 = 0; g0 < a.groups; g0 += 32 >> a.lanes_log2) {
            const int g = g0 + first;
            Key m1 = 0, m2 = 0;
            if (g < a.groups)
                for (int i = sub; i < size; i += per_group) {
                    const Key c = ((const Key *)sh)[g * size + i];
                    m2 = max(m2, min(m1, c));
                    m1 = max(m1, c);
                }
            for (int d = 1; d < per_group; d *= 2) {
                const Key n1 = __shfl_xor_sync(kFull, m1, d), n2 = __shfl_xor_sync(kFull, m2, d);
                m2 = max(min(m1, n1), max(m2, n2));
                m1 = max(m1, n1);
            }
            if (sub == 0 && g < a.groups) gkey[g] = group_key(m1, m2, a.group_top);
        }
        __syncwarp();
        const float per = 1.0f / (float)size;             // (e + 1/2) / size is at least 2^-11 from a whole number
        Key k0 = lane < a.groups ? gkey[lane] : 0, k1 = lane + 32 < a.groups ? gkey[lane + 32] : 0;
        uint64_t kept = 0;                                // the groups that stay, one bit each
        for (int i = 0; i < a.keep; ++i) {
            const bool low = k0 >= k1;
            const int g = warp_best(low ? k0 : k1, low ? lane : lane + 32);
            if (g < 0) break;
            kept |= 1ull << g;
            if (g == lane) k0 = 0;
            if (g == lane + 32) k1 = 0;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = lane + 32 * s;
            if (e < a.E && !(kept >> (int)(((float)e + 0.5f) * per) & 1)) key[s] = 0;
        }
        __syncwarp();                                     // the next token of this warp writes sh again
    }
    int id = -1;
    for (int j = 0; j < a.k; ++j) {
        // this lane's best, pairwise (equal keys: the lower slot)
        Key m[S];
        int at[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            m[s] = key[s];
            at[s] = s;
        }
#pragma unroll
        for (int d = 1; d < S; d *= 2)
#pragma unroll
            for (int s = 0; s + d < S; s += 2 * d)
                if (m[s + d] > m[s]) {
                    m[s] = m[s + d];
                    at[s] = at[s + d];
                }
        const int e = warp_best(m[0], lane + 32 * at[0]);
        if (e < 0) break;
        if (lane == j) id = e;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (lane + 32 * s == e) key[s] = 0;
    }
    // the scores of the chosen, by the lane of each
    const float xc = id >= 0 ? logit(a, t * a.E + id) : 0.f;
    // (renormalised without other need of it, a softmax has no common sum: the largest chosen logit is place 0's)
    const float ref = SIMPLE && a.renorm ? __shfl_sync(kFull, xc, 0) : top;
    double w = id < 0 ? 0.0 : a.sigmoid ? sigmoid64((double)xc) : exp_neg((double)xc - (double)ref) * total;
    if (a.renorm) {
        const double sum = warp_sum(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.weights[t * a.k + lane] = (float)(w * (double)a.scale);
        if (a.pos && id < 0) a.pos[t * a.k + lane] = -1;
    }
    return id;
}

template <int S, bool SIMPLE>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a)
{
    extern __shared__ uint64_t route_sh[];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t < a.T) choose<S, SIMPLE>(a, t, route_sh + warp * (a.E + 64));
}

// Choice and plan of at most kFusedPairs pairs by one CTA.
template <int S, bool SIMPLE>
__global__ void __launch_bounds__(kFusedWarps * 32) route_fused_kernel(RouteArgs a)
{
    extern __shared__ uint64_t route_sh[];
    __shared__ __align__(16) int id_sh[kFusedPairs];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int P = (int)a.T * a.k;
    for (int i = threadIdx.x; i < kFusedPairs; i += blockDim.x) id_sh[i] = -1;
    __syncthreads();
    if (warp < a.T) {
        const int id = choose<S, SIMPLE>(a, warp, route_sh + warp * (a.E + 64));
        if (lane < a.k) id_sh[warp * a.k + lane] = id;
    }
    __syncthreads();
    // entry i < P: the row of pair i, that is the pairs of lower experts and the earlier ones of its own;
    // entry P + e: the pairs of lower experts, offsets[e]
    for (int i = threadIdx.x; i < P + a.E + 1; i += blockDim.x) {
        const int id = i < P ? id_sh[i] : i - P;
        int row = 0;
        for (int q = 0; q < P; q += 4) {                  // (padded with -1)
            const int4 v = *(const int4 *)(id_sh + q);
            row += ((unsigned)v.x < (unsigned)id) + ((unsigned)v.y < (unsigned)id) + ((unsigned)v.z < (unsigned)id) +
                   ((unsigned)v.w < (unsigned)id);
            if (i < P)
                row += (v.x == id && q < i) + (v.y == id && q + 1 < i) + (v.z == id && q + 2 < i) + (v.w == id && q + 3 < i);
        }
        // (-1 as unsigned is above every expert: the pairs without one sort behind the last row)
        if (i >= P) a.offsets[i - P] = row;
        else {
            a.order[row] = id >= 0 ? i : -1;
            if (id >= 0) a.pos[i] = row;
        }
    }
}

// The plan of expert e = blockIdx.x: its first row is the number of pairs of
// lower experts, and its pairs follow in order.  Warp w looks through the w-th
// contiguous part of the ids, 32 at a time.
__global__ void __launch_bounds__(1024) plan_kernel(const int *ids, int P, int E, int *offsets, int *order, int *pos)
{
    __shared__ int warp_below[32], warp_own[32];
    pdl_wait();
    pdl_launch_dependents();
    const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int part = ((P + warps - 1) / warps + 31) & ~31;
    const int lo = min(P, warp * part), hi = min(P, lo + part);
    int below = 0, own = 0;
#pragma unroll 8
    for (int p = lo + lane; p < hi; p += 32) {
        const int id = __ldg(ids + p);
        below += (unsigned)id < (unsigned)e;
        own += id == e;
    }
    below = __reduce_add_sync(kFull, below);
    own = __reduce_add_sync(kFull, own);
    if (lane == 0) {
        warp_below[warp] = below;
        warp_own[warp] = own;
    }
    __syncthreads();
    const int b = lane < warps ? warp_below[lane] : 0, o = lane < warps ? warp_own[lane] : 0;
    const int start = __reduce_add_sync(kFull, b);
    const int count = __reduce_add_sync(kFull, o);
    int row = start + __reduce_add_sync(kFull, lane < warp ? o : 0);
    if (own > 0) {
#pragma unroll 4
        for (int p0 = lo; p0 < hi; p0 += 32) {
            const int p = p0 + lane;
            const bool mine = p < hi && __ldg(ids + p) == e;
            const unsigned all = __ballot_sync(kFull, mine);
            if (mine) {
                const int r = row + __popc(all & ((1u << lane) - 1u));
                order[r] = p;
                pos[p] = r;
            }
            row += __popc(all);
        }
    }
    if (threadIdx.x == 0) offsets[e] = start;
    if (e == E - 1) {
        if (threadIdx.x == 0) offsets[E] = start + count;
        for (int p = start + count + threadIdx.x; p < P; p += blockDim.x) order[p] = -1;
    }
}

// The plan of many pairs, by one cluster of kPlanCtas CTAs: CTA c has the c-th
// contiguous part of the ids and warp w the w-th part of that, 32 at a time.
// Every warp counts its pairs of each expert; the counts are summed over the
// warps of a CTA and, through distributed shared memory, over the CTAs, which
// with the sum over the lower experts gives the row of each warp's first pair of
// each expert; then the ids are read again and placed, lanes with the same id
// (found by a ballot for each bit of the id; the match instruction took 2000
// clocks with 32 warps at it) in their order.  `sh`: kPlanWarps + 2 rows of E
// counts.
constexpr int kPlanCtas = 8, kPlanWarps = 32, kPlanMany = 32768;

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanWarps * 32)
plan_many_kernel(const int *ids, int P, int E, int id_bits, int *offsets, int *order, int *pos)
{
    extern __shared__ int sh[];
    __shared__ int warp_total[32];
    const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *mine = sh + warp * E;                            // this warp's counts, then rows
    int *total = sh + kPlanWarps * E, *start = total + E; // this CTA's counts, and the first rows of its pairs
    cg::cluster_group cluster = cg::this_cluster();
    for (int i = threadIdx.x; i < kPlanWarps * E; i += blockDim.x) sh[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    const int part = (P + kPlanCtas * kPlanWarps - 1) / (kPlanCtas * kPlanWarps);
    const int64_t from = (int64_t)(c * kPlanWarps + warp) * part;
    const int lo = (int)(from < P ? from : P), hi = min(P, lo + part);
    __syncthreads();
    constexpr int kBatch = 8;                             // loads in flight
    int id[kBatch];
    auto load = [&](int p0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) id[i] = p0 + 32 * i + lane < hi ? __ldg(ids + p0 + 32 * i + lane) : -1;
    };
    for (int p0 = lo; p0 < hi; p0 += 32 * kBatch) {
        load(p0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (id[i] >= 0) atomicAdd(mine + id[i], 1);   // (counts alone: their order does not matter)
    }
    __syncthreads();
    const int e = threadIdx.x;                            // (E <= 1024 threads)
    if (e < E) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < kPlanWarps; ++w) {
            const int n = sh[w * E + e];
            sh[w * E + e] = sum;
            sum += n;
        }
        total[e] = sum;
    }
    cluster.sync();                                       // every CTA's totals are there
    int all = 0, before = 0;                              // pairs of expert e, and those of the CTAs in front
    if (e < E)
        for (int r = 0; r < kPlanCtas; ++r) {
            const int n = cluster.map_shared_rank(total, r)[e];
            before += r < c ? n : 0;
            all += n;
        }
    int upto = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kFull, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) warp_total[warp] = upto;
    cluster.sync();                                       // (and no CTA reads another's totals any more)
    const int t = warp_total[lane];
    const int first = __reduce_add_sync(kFull, lane < warp ? t : 0) + upto - all;
    const int rows = __reduce_add_sync(kFull, t);
    if (e < E) {
        start[e] = first + before;
        if (c == 0) offsets[e] = first;
    }
    if (c == 0 && e == 0) offsets[E] = rows;
    for (int64_t p = (int64_t)rows + c * blockDim.x + threadIdx.x; p < P; p += kPlanCtas * blockDim.x) order[p] = -1;
    __syncthreads();
    const unsigned lower = (1u << lane) - 1u;
    for (int p0 = lo; p0 < hi; p0 += 32 * kBatch) {
        load(p0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            unsigned same = __ballot_sync(kFull, id[i] >= 0);
            for (int b = 0; b < id_bits; ++b) {
                const bool bit = (id[i] >> b) & 1;
                const unsigned with = __ballot_sync(kFull, bit);
                same &= bit ? with : ~with;
            }
            if (id[i] >= 0) {
                const int p = p0 + 32 * i + lane, row = start[id[i]] + mine[id[i]] + __popc(same & lower);
                order[row] = p;
                pos[p] = row;
            }
            __syncwarp();
            if (id[i] >= 0 && (same & lower) == 0) mine[id[i]] += __popc(same);
            __syncwarp();
        }
    }
}

// One thread sums 8 (VEC) or 1 columns of one token, the rows of up to kAhead
// pairs in flight at once; `parts` CTAs share a token's columns.  The sum runs in
// fp32 in the order of the pairs.  What bounds it: HBM, each row of Y read once
// (8192 tokens, 8 experts, N = 4096, with a shared expert: 672 MB in 110 to 112 us
// on two B200s, 92 to 94% of the copy rate).
constexpr int kAhead = 8;

template <bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(const __nv_bfloat16 *Y, int64_t P, const int *pos,
                                                      const float *weights, int64_t T, int k, int64_t N, unsigned parts,
                                                      const __nv_bfloat16 *add, __nv_bfloat16 *out)
{
    pdl_wait();
    pdl_launch_dependents();
    constexpr int W = VEC ? 8 : 1;
    for (int64_t b = blockIdx.x; b < T * parts; b += gridDim.x) {
        const int64_t t = b / parts;
        const int64_t c = ((b - t * parts) * blockDim.x + threadIdx.x) * W;
        if (c >= N) continue;
        typedef typename std::conditional<VEC, uint4, unsigned short>::type Word;
        auto unpack = [&](const Word &u, float (&f)[W]) {
            if constexpr (VEC) {
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] = bf16lo_to_f32(w[j]);
                    f[2 * j + 1] = bf16hi_to_f32(w[j]);
                }
            } else {
                f[0] = __uint_as_float((uint32_t)u << 16);
            }
        };
        float acc[W];
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = 0.f;
        if (add) unpack(*(const Word *)(add + t * N + c), acc);
        for (int j0 = 0; j0 < k; j0 += kAhead) {
            Word y[kAhead];
            float w[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int64_t row = j0 + j < k ? __ldg(pos + t * k + j0 + j) : -1;
                const bool on = row >= 0 && row < P;
                w[j] = on ? __ldg(weights + t * k + j0 + j) : 0.f;
                y[j] = Word{};
                if (on) y[j] = __ldg((const Word *)(Y + row * N + c));
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                float f[W];
                unpack(y[j], f);
#pragma unroll
                for (int q = 0; q < W; ++q) acc[q] = fmaf(w[j], f[q], acc[q]);
            }
        }
        if constexpr (VEC) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 p2 = __floats2bfloat162_rn(acc[2 * j], acc[2 * j + 1]);
                w[j] = *(const uint32_t *)&p2;
            }
            *(uint4 *)(out + t * N + c) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            out[t * N + c] = __float2bfloat16_rn(acc[0]);
        }
    }
}

template <int S, bool SIMPLE>
cudaError_t launch_choose(const RouteArgs &a, bool fused, cudaStream_t stream)
{
    const int warps = fused ? (int)a.T : kRouteWarps;
    const size_t smem = a.groups > 1 ? (size_t)warps * (a.E + 64) * sizeof(uint64_t) : 0;
    static std::atomic<bool> attr_done[2][kMaxDevices];
    auto kern = fused ? route_fused_kernel<S, SIMPLE> : route_kernel<S, SIMPLE>;
    if (smem > 0) {                                       // (48 KB without the opt-in, static arrays included)
        const cudaError_t e = set_smem_attr(kern, (fused ? kFusedWarps : kRouteWarps) * (32 * S + 64) * 8, attr_done[fused]);
        if (e != cudaSuccess) return e;
    }
    if (fused)                                            // at least 4 warps: the plan has E entries
        return launch_pdl(kern, dim3(1), dim3((warps < 4 ? 4 : warps) * 32), smem * (warps < 4 ? 4 : warps) / warps, stream, a);
    return launch_pdl(kern, dim3((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps)), dim3(kRouteWarps * 32), smem, stream, a);
}

template <bool SIMPLE>
cudaError_t launch_experts(const RouteArgs &a, bool fused, cudaStream_t stream)
{
    const int s = (a.E + 31) / 32;
    return s <= 1   ? launch_choose<1, SIMPLE>(a, fused, stream)
           : s <= 2 ? launch_choose<2, SIMPLE>(a, fused, stream)
           : s <= 4 ? launch_choose<4, SIMPLE>(a, fused, stream)
           : s <= 8 ? launch_choose<8, SIMPLE>(a, fused, stream)
           : s <= 16 ? launch_choose<16, SIMPLE>(a, fused, stream)
                     : launch_choose<32, SIMPLE>(a, fused, stream);
}

}  // namespace

cudaError_t launch_route(const void *logits, int f32, const float *bias, int64_t T, int E, int k, int sigmoid,
                         int groups, int keep, int group_top, int renorm, float scale, int *ids, float *weights,
                         int *offsets, int *order, int *pos, cudaStream_t stream)
{
    int lanes_log2 = 0;
    while ((2 << lanes_log2) * groups <= 32) ++lanes_log2;
    const RouteArgs a = {logits, bias, ids, pos, offsets, order, weights, T, E, k, f32, sigmoid, groups, keep,
                         group_top, renorm, scale, E / groups, lanes_log2};
    const int64_t P = T * k;
    const bool fused = offsets && T <= kFusedWarps && P <= kFusedPairs;
    const bool simple = !bias && (groups == 1 || group_top == 1);
    const cudaError_t e = simple ? launch_experts<true>(a, fused, stream) : launch_experts<false>(a, fused, stream);
    if (e != cudaSuccess || !offsets || fused) return e;
    // Both kernels for the plan behind the choice, us, a CTA for each expert / a cluster:
    //   pairs      4096        16384       32768       65536
    //   32 experts  3.6 / 6.3   4.6 / 6.5   6.7 / 6.8  12.8 / 7.7
    //   128         3.6 / 7.0   6.7 / 7.6   8.6 / 7.9  18.2 / 8.8
    //   256         3.7 / 7.6  10.4 / 7.9   9.9 / 6.3  18.3 / 9.2
    //   1024        5.2 / 9.7  20.6 / 10   27.4 / 11   56.4 / 11
    // The rule goes by the pairs alone: with many experts the cluster would be ahead from fewer pairs on
    // (256: about 12000, 1024: about 6000).
    if (P <= kPlanMany) {
        const int threads = P >= 8192 ? 1024 : 256;
        return launch_pdl(plan_kernel, dim3(E), dim3(threads), 0, stream, (const int *)ids, (int)P, E, offsets, order, pos);
    }
    const int smem = (kPlanWarps + 2) * E * (int)sizeof(int);
    static std::atomic<bool> attr_done[kMaxDevices];
    const cudaError_t e2 = set_smem_attr(plan_many_kernel, (kPlanWarps + 2) * 1024 * (int)sizeof(int), attr_done);
    if (e2 != cudaSuccess) return e2;
    int id_bits = 0;
    while ((1 << id_bits) < E) ++id_bits;
    return launch_pdl(plan_many_kernel, dim3(kPlanCtas), dim3(kPlanWarps * 32), smem, stream, (const int *)ids, (int)P, E,
                      id_bits, offsets, order, pos);
}

cudaError_t launch_combine(const void *Y, int64_t P, const int *pos, const float *weights, int64_t T, int k, int64_t N,
                           const void *add, void *out, cudaStream_t stream)
{
    const uintptr_t all = (uintptr_t)Y | (uintptr_t)add | (uintptr_t)out;
    const bool vec = N % 8 == 0 && all % 16 == 0;
    const int64_t cols = vec ? N / 8 : N;
    const int threads = cols >= 256 ? 256 : (int)((cols + 31) / 32 * 32);
    const int64_t parts = (cols + threads - 1) / threads;
    if (parts > INT32_MAX || T > INT64_MAX / parts) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(T * parts < INT32_MAX ? T * parts : INT32_MAX);
    return launch_pdl(vec ? combine_kernel<true> : combine_kernel<false>, dim3(grid), dim3(threads), 0, stream,
                      (const __nv_bfloat16 *)Y, P, pos, weights, T, k, N, (unsigned)parts, (const __nv_bfloat16 *)add,
                      (__nv_bfloat16 *)out);
}

}  // namespace w4
