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
// experts 0, below every number); its maximum over the warp takes two 32-bit
// reductions (three for fp64): the key, then the lowest index that has it.
//
// The plan needs no scan across CTAs: the CTA of expert e reads all ids, counts
// those below e (where its rows begin) and lists its own pairs in order.  Up to
// kFusedPairs pairs of kFusedWarps tokens the one CTA that chooses also makes the
// plan, each thread ranking one pair against all others in shared memory: one
// launch in place of two.  (57 tokens that way took 11.9 us, against 5.2 in two.)
// What bounds it: latency.  8192 tokens, 8 of 128 experts (4.7 MB, 0.8 us of HBM)
// take 20.7 us; with fp64 scores for the choice, and each thread of the plan
// reading a run of ids of its own, 88.
#include "common.cuh"

#include <type_traits>

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

// The warp's largest key and the lowest index that has it.
__device__ __forceinline__ int warp_best(uint32_t key, int idx, uint32_t &best)
{
    best = __reduce_max_sync(kFull, key);
    return (int)__reduce_min_sync(kFull, key == best ? (unsigned)idx : kFull);
}

__device__ __forceinline__ int warp_best(uint64_t key, int idx, uint64_t &best)
{
    const uint32_t hi = (uint32_t)(key >> 32);
    const uint32_t mh = __reduce_max_sync(kFull, hi);
    const uint32_t ml = __reduce_max_sync(kFull, hi == mh ? (uint32_t)key : 0u);
    best = ((uint64_t)mh << 32) | ml;
    return (int)__reduce_min_sync(kFull, key == best ? (unsigned)idx : kFull);
}

// What a group is worth, and how the larger of two is found: the keys
// themselves (SIMPLE), or fp64 choices that are summed.
template <bool SIMPLE>
struct Choice;
template <>
struct Choice<true> {
    typedef uint32_t Key, Value;
    static __device__ __forceinline__ Value none() { return 0u; }
    static __device__ __forceinline__ Value larger(Value a, Value b) { return max(a, b); }
    static __device__ __forceinline__ Value smaller(Value a, Value b) { return min(a, b); }
    static __device__ __forceinline__ Key group(Value m1, Value, int) { return m1; }
};
template <>
struct Choice<false> {
    typedef uint64_t Key;
    typedef double Value;
    static __device__ __forceinline__ Value none() { return -INFINITY; }
    static __device__ __forceinline__ Value larger(Value a, Value b) { return fmax(a, b); }
    static __device__ __forceinline__ Value smaller(Value a, Value b) { return fmin(a, b); }
    static __device__ __forceinline__ Key group(Value m1, Value m2, int top)
    {
        return order_key(top == 2 && m2 > -INFINITY ? m1 + m2 : m1);
    }
};

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// The choice for token t by one warp; S >= E / 32 experts per lane.  `sh`: E + 64
// 8-byte words of this warp's shared memory (groups only).  Returns the id that
// this lane's place j = lane got, and writes ids and weights.
template <int S, bool SIMPLE>
__device__ __forceinline__ int choose(const RouteArgs &a, int64_t t, uint64_t *sh)
{
    typedef Choice<SIMPLE> Ch;
    typedef typename Ch::Key Key;
    typedef typename Ch::Value Value;
    const int lane = threadIdx.x & 31;
    float x[S];
    Key key[S];
    double score[SIMPLE ? 1 : S];
    float top = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int e = lane + 32 * s;
        x[s] = -INFINITY;
        if (e < a.E)
            x[s] = a.f32 ? __ldg((const float *)a.logits + t * a.E + e)
                         : __bfloat162float(__ldg((const __nv_bfloat16 *)a.logits + t * a.E + e));
        top = fmaxf(top, x[s]);
    }
    double total = 1.0;                                   // the softmax's sum, where it is wanted
    if (!a.sigmoid && (!SIMPLE || !a.renorm)) {
        top = warp_max(top);
        total = 0.0;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const double v = x[s] != -INFINITY ? exp((double)x[s] - (double)top) : 0.0;
            if (!SIMPLE) score[SIMPLE ? 0 : s] = v;
            total += v;
        }
        total = warp_sum(total);
        total = total > 0.0 ? total : 1.0;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int e = lane + 32 * s;
        if (SIMPLE) {
            key[s] = order_key(x[s]);
            if (a.groups > 1 && e < a.E) ((uint32_t *)sh)[e] = (uint32_t)key[s];
        } else {
            double &sc = score[SIMPLE ? 0 : s];
            const bool live = x[s] != -INFINITY;          // (a NaN stays, and spoils its own token only)
            sc = !live ? 0.0 : a.sigmoid ? sigmoid64((double)x[s]) : sc / total;
            const double c = sc + (a.bias && e < a.E ? (double)__ldg(a.bias + e) : 0.0);
            key[s] = live ? (Key)order_key(c) : (Key)0;
            if (a.groups > 1 && e < a.E) ((double *)sh)[e] = live ? c : -INFINITY;
        }
    }
    if (a.groups > 1) {
        // a group's two best choices, by `per_group` lanes each
        const int size = a.E / a.groups;
        int per_group = 1;
        while (per_group * 2 * a.groups <= 32) per_group *= 2;
        Key *gkey = (Key *)(sh + a.E);
        const int sub = lane & (per_group - 1), first = lane / per_group;
        __syncwarp();
        for (int g0 = 0; g0 < a.groups; g0 += 32 / per_group) {
            const int g = g0 + first;
            Value m1 = Ch::none(), m2 = Ch::none();
            if (g < a.groups)
                for (int i = sub; i < size; i += per_group) {
                    const Value c = ((const Value *)sh)[g * size + i];
                    m2 = Ch::larger(m2, Ch::smaller(m1, c));
                    m1 = Ch::larger(m1, c);
                }
            for (int d = 1; d < per_group; d *= 2) {
                const Value n1 = __shfl_xor_sync(kFull, m1, d), n2 = __shfl_xor_sync(kFull, m2, d);
                m2 = Ch::larger(Ch::smaller(m1, n1), Ch::larger(m2, n2));
                m1 = Ch::larger(m1, n1);
            }
            if (sub == 0 && g < a.groups) gkey[g] = Ch::group(m1, m2, a.group_top);
        }
        __syncwarp();
        Key k0 = lane < a.groups ? gkey[lane] : 0, k1 = lane + 32 < a.groups ? gkey[lane + 32] : 0;
        uint64_t kept = 0;                                // the groups that stay, one bit each
        for (int i = 0; i < a.keep; ++i) {
            Key best;
            const bool low = k0 >= k1;
            const int g = warp_best(low ? k0 : k1, low ? lane : lane + 32, best);
            if (best == 0) break;
            kept |= 1ull << g;
            if (g == lane) k0 = 0;
            if (g == lane + 32) k1 = 0;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int e = lane + 32 * s;
            if (e < a.E && !(kept >> (e / size) & 1)) key[s] = 0;
        }
        __syncwarp();                                     // the next token of this warp writes sh again
    }
    int id = -1;
    float chosen = 0.f;                                   // SIMPLE: the chosen logit, else its score
    double w = 0.0;
    for (int j = 0; j < a.k; ++j) {
        Key mine = 0, best;
        int at = 0;
        float xb = 0.f;
        double sb = 0.0;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (key[s] > mine) {
                mine = key[s];
                at = s;
                if (SIMPLE) xb = x[s];
                else sb = score[SIMPLE ? 0 : s];
            }
        const int e = warp_best(mine, lane + 32 * at, best);
        if (best == 0) break;
        if (SIMPLE) xb = __shfl_sync(kFull, xb, e & 31);
        else sb = __shfl_sync(kFull, sb, e & 31);
        if (lane == j) {
            id = e;
            chosen = xb;
            w = sb;
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (lane + 32 * s == e) key[s] = 0;
    }
    if (SIMPLE) {
        // (renormalised, a softmax needs no common sum: the largest chosen logit is place 0's)
        const float ref = a.renorm ? __shfl_sync(kFull, chosen, 0) : top;
        if (id >= 0) w = a.sigmoid ? sigmoid64((double)chosen) : exp((double)chosen - (double)ref) / total;
    }
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

// One thread sums 8 (VEC) or 1 columns of one token, the rows of up to kAhead
// pairs in flight at once; `parts` CTAs share a token's columns.  The sum runs in
// fp32 in the order of the pairs.  What bounds it: HBM, each row of Y read once
// (8192 tokens, 8 experts, N = 4096, with a shared expert: 672 MB, 102 us).
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
    if (smem > 48 * 1024) {
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
    const RouteArgs a = {logits, bias, ids, pos, offsets, order, weights, T, E, k, f32, sigmoid, groups, keep,
                         group_top, renorm, scale};
    const int64_t P = T * k;
    const bool fused = offsets && T <= kFusedWarps && P <= kFusedPairs;
    const bool simple = !bias && (groups == 1 || group_top == 1);
    const cudaError_t e = simple ? launch_experts<true>(a, fused, stream) : launch_experts<false>(a, fused, stream);
    if (e != cudaSuccess || !offsets || fused) return e;
    const int threads = P >= 8192 ? 1024 : 256;
    return launch_pdl(plan_kernel, dim3(E), dim3(threads), 0, stream, (const int *)ids, (int)P, E, offsets, order, pos);
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
