// w4_route: the choice of experts for each token and the plan of their rows;
// w4_combine: the weighted sum over a token's experts.
//
// Mathematics (include/w4.h has the exact semantics), per token:
//     score = softmax(logits) or 1 / (1 + exp(-logit)),  choice = score + bias,
//     the top_k largest choices (within the best groups), weight = score /
//     sum of the chosen scores * scale,
// and then a stable counting sort of the T * top_k pairs by expert.
//
// Scores and choices are fp64.  Which of two near choices is larger decides a
// whole number, so the order has to be that of the exact scores; fp32 scores
// of different logits often round to the same value.  The fp64 units carry it:
// about 40 operations per logit.
//
// One warp chooses for one token: lane l holds the experts l, l + 32, ..., so
// logits are read in whole lines and equal choices can be told apart by index.
// A choice is compared as a 64-bit integer in the order of the doubles (masked
// experts 0, below every number), and its maximum over the warp takes three
// 32-bit reductions: high word, low word, lowest index.
//
// The plan needs no scan across CTAs: the CTA of expert e reads all ids, counts
// those below e (where its rows begin) and lists its own pairs in order.
#include "common.cuh"

namespace w4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRouteWarps = 8;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int *ids, *pos;
    float *weights;
    int64_t T;
    int E, k, f32, sigmoid, groups, keep, group_top, renorm;
    float scale;
};

// Doubles as unsigned integers of the same order; 0 stands below all of them
// (NaN, which no comparison orders, is taken for the masked value too).
__device__ __forceinline__ uint64_t order_key(double v)
{
    if (!(v > -INFINITY)) return 0;
    const int64_t b = __double_as_longlong(v + 0.0);      // (-0 and +0 are equal choices)
    return b < 0 ? ~(uint64_t)b : (uint64_t)b | (1ull << 63);
}

__device__ __forceinline__ double warp_max(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// The warp's largest key and the lowest index that has it (lanes without one
// give key 0).
__device__ __forceinline__ int warp_best(uint64_t key, int idx, uint64_t &best)
{
    const uint32_t hi = (uint32_t)(key >> 32);
    const uint32_t mh = __reduce_max_sync(kFull, hi);
    const uint32_t lo = hi == mh ? (uint32_t)key : 0u;
    const uint32_t ml = __reduce_max_sync(kFull, lo);
    best = ((uint64_t)mh << 32) | ml;
    return (int)__reduce_min_sync(kFull, key == best ? (unsigned)idx : 0xffffffffu);
}

// The choice for token t by one warp; S = ceil(E / 32) experts per lane.
// `sh`: E doubles and 64 more of shared memory of this warp (groups only).
template <int S>
__device__ __forceinline__ void choose(const RouteArgs &a, int64_t t, double *sh)
{
    const int lane = threadIdx.x & 31;
    double score[S];
    uint64_t key[S];
    double top = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int e = lane + 32 * s;
        double x = -INFINITY;
        if (e < a.E)
            x = a.f32 ? (double)__ldg((const float *)a.logits + t * a.E + e)
                      : (double)__bfloat162float(__ldg((const __nv_bfloat16 *)a.logits + t * a.E + e));
        score[s] = x;
        top = fmax(top, x);
    }
    double total = 1.0;
    if (!a.sigmoid) {
        top = warp_max(top);
        total = 0.0;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const double x = score[s];
        const bool live = x != -INFINITY;                 // (a NaN stays, and spoils its token's weights only)
        if (a.sigmoid) score[s] = live ? 1.0 / (1.0 + exp(-x)) : 0.0;
        else {
            score[s] = live ? exp(x - top) : 0.0;
            total += score[s];
        }
        key[s] = live ? 1 : 0;
    }
    if (!a.sigmoid) {
        total = warp_sum(total);
        total = total > 0.0 ? total : 1.0;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int e = lane + 32 * s;
        score[s] /= total;
        const double c = score[s] + (a.bias && e < a.E ? (double)__ldg(a.bias + e) : 0.0);
        if (key[s]) {
            key[s] = order_key(c);
            key[s] = key[s] ? key[s] : 1;                 // unmasked, but not a number: behind all others
        }
        if (a.groups > 1 && e < a.E) sh[e] = key[s] ? c : -INFINITY;
    }
    if (a.groups > 1) {
        const int per = a.E / a.groups;
        uint64_t *gkey = (uint64_t *)(sh + a.E);
        __syncwarp();
        for (int g = lane; g < a.groups; g += 32) {
            double m1 = -INFINITY, m2 = -INFINITY;
            for (int i = 0; i < per; ++i) {
                const double c = sh[g * per + i];
                m2 = fmax(m2, fmin(m1, c));
                m1 = fmax(m1, c);
            }
            gkey[g] = order_key(a.group_top == 2 && m2 > -INFINITY ? m1 + m2 : m1);
        }
        __syncwarp();
        uint64_t k0 = lane < a.groups ? gkey[lane] : 0, k1 = lane + 32 < a.groups ? gkey[lane + 32] : 0;
        uint64_t kept = 0;                                // the groups that stay, one bit each
        for (int i = 0; i < a.keep; ++i) {
            uint64_t best;
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
            if (e < a.E && !(kept >> (e / per) & 1)) key[s] = 0;
        }
        __syncwarp();                                     // the next token of this warp writes sh again
    }
    int id = -1;
    double w = 0.0;
    for (int j = 0; j < a.k; ++j) {
        uint64_t mine = 0, best;
        int at = 0;
        double sc = 0.0;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (key[s] > mine) {
                mine = key[s];
                at = s;
                sc = score[s];
            }
        const int e = warp_best(mine, lane + 32 * at, best);
        if (best == 0) break;
        sc = __shfl_sync(kFull, sc, e & 31);
        if (lane == j) {
            id = e;
            w = sc;
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (lane + 32 * s == e) key[s] = 0;
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
}

template <int S>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a)
{
    extern __shared__ double route_sh[];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t < a.T) choose<S>(a, t, route_sh + warp * (a.E + 64));
}

// The plan of expert e = blockIdx.x: its first row is the number of pairs of
// lower experts, and its pairs follow in order.  Thread i looks through the
// i-th contiguous part of the ids.
__global__ void __launch_bounds__(1024) plan_kernel(const int *ids, int P, int E, int *offsets, int *order, int *pos)
{
    __shared__ int warp_below[32], warp_own[32];
    pdl_wait();
    pdl_launch_dependents();
    const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int part = (P + blockDim.x - 1) / blockDim.x;
    const int lo = min(P, (int)threadIdx.x * part), hi = min(P, lo + part);
    int below = 0, own = 0;
    for (int p = lo; p < hi; ++p) {
        const int id = ids[p];
        below += id >= 0 && id < e;
        own += id == e;
    }
    int before = own;                                     // inclusive scan of `own` over the warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kFull, before, d);
        if (lane >= d) before += v;
    }
    below = __reduce_add_sync(kFull, below);
    if (lane == 31) {
        warp_below[warp] = below;
        warp_own[warp] = before;
    }
    __syncthreads();
    const int b = lane < warps ? warp_below[lane] : 0, o = lane < warps ? warp_own[lane] : 0;
    const int start = __reduce_add_sync(kFull, b);
    const int count = __reduce_add_sync(kFull, o);
    int row = start + __reduce_add_sync(kFull, lane < warp ? o : 0) + before - own;
    for (int p = lo; p < hi; ++p)
        if (ids[p] == e) {
            order[row] = p;
            pos[p] = row++;
        }
    if (threadIdx.x == 0) offsets[e] = start;
    if (e == E - 1) {
        if (threadIdx.x == 0) offsets[E] = start + count;
        for (int p = start + count + threadIdx.x; p < P; p += blockDim.x) order[p] = -1;
    }
}

// One thread sums 8 (vec) or 1 columns of one token.
template <bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(const __nv_bfloat16 *Y, int64_t P, const int *pos,
                                                      const float *weights, int64_t T, int k, int64_t N,
                                                      const __nv_bfloat16 *add, __nv_bfloat16 *out)
{
    pdl_wait();
    pdl_launch_dependents();
    constexpr int W = VEC ? 8 : 1;
    const int64_t per = N / W, total = T * per;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / per, c = (i - t * per) * W;
        float acc[W];
        auto load = [&](const __nv_bfloat16 *p, float (&f)[W]) {
            if (VEC) {
                const uint4 u = *(const uint4 *)p;
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    f[2 * j] = bf16lo_to_f32(w[j]);
                    f[2 * j + 1] = bf16hi_to_f32(w[j]);
                }
            } else {
                f[0] = __bfloat162float(*p);
            }
        };
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = 0.f;
        if (add) load(add + t * N + c, acc);
        for (int j = 0; j < k; ++j) {
            const int64_t row = __ldg(pos + t * k + j);
            if (row < 0 || row >= P) continue;
            const float w = __ldg(weights + t * k + j);
            float f[W];
            load(Y + row * N + c, f);
#pragma unroll
            for (int q = 0; q < W; ++q) acc[q] = fmaf(w, f[q], acc[q]);
        }
        if (VEC) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                const __nv_bfloat162 p2 = __floats2bfloat162_rn(acc[2 * j], acc[2 * j + 1]);
                w[j] = *(const uint32_t *)&p2;
            }
            *(uint4 *)(out + t * N + c) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            out[t * N + c] = __float2bfloat16_rn(acc[0]);
        }
    }
}

template <int S>
cudaError_t launch_choose(const RouteArgs &a, cudaStream_t stream)
{
    const size_t smem = a.groups > 1 ? (size_t)kRouteWarps * (a.E + 64) * sizeof(double) : 0;
    static std::atomic<bool> attr_done[kMaxDevices];
    const cudaError_t e = set_smem_attr(route_kernel<S>, kRouteWarps * (32 * S + 64) * 8, attr_done);
    if (e != cudaSuccess) return e;
    return launch_pdl(route_kernel<S>, dim3((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps)),
                      dim3(kRouteWarps * 32), smem, stream, a);
}

}  // namespace

cudaError_t launch_route(const void *logits, int f32, const float *bias, int64_t T, int E, int k, int sigmoid,
                         int groups, int keep, int group_top, int renorm, float scale, int *ids, float *weights,
                         int *offsets, int *order, int *pos, cudaStream_t stream)
{
    const RouteArgs a = {logits, bias, ids, pos, weights, T, E, k, f32, sigmoid, groups, keep, group_top, renorm, scale};
    const int s = (E + 31) / 32;
    const cudaError_t e = s <= 1   ? launch_choose<1>(a, stream)
                          : s <= 2 ? launch_choose<2>(a, stream)
                          : s <= 4 ? launch_choose<4>(a, stream)
                          : s <= 8 ? launch_choose<8>(a, stream)
                          : s <= 16 ? launch_choose<16>(a, stream)
                                    : launch_choose<32>(a, stream);
    if (e != cudaSuccess || !offsets) return e;
    const int64_t P = T * k;
    const int threads = P >= 1024 ? 1024 : P >= 256 ? 256 : 32;
    return launch_pdl(plan_kernel, dim3(E), dim3(threads), 0, stream, (const int *)ids, (int)P, E, offsets, order, pos);
}

cudaError_t launch_combine(const void *Y, int64_t P, const int *pos, const float *weights, int64_t T, int k, int64_t N,
                           const void *add, void *out, cudaStream_t stream)
{
    const uintptr_t all = (uintptr_t)Y | (uintptr_t)add | (uintptr_t)out;
    const bool vec = N % 8 == 0 && all % 16 == 0;
    const int64_t want = (T * (vec ? N / 8 : N) + 255) / 256;
    const unsigned grid = (unsigned)(want < (int64_t)kNumSMs * 64 ? want : (int64_t)kNumSMs * 64);
    auto *y = (const __nv_bfloat16 *)Y;
    auto *ad = (const __nv_bfloat16 *)add;
    auto *o = (__nv_bfloat16 *)out;
    if (vec) return launch_pdl(combine_kernel<true>, dim3(grid), dim3(256), 0, stream, y, P, pos, weights, T, k, N, ad, o);
    return launch_pdl(combine_kernel<false>, dim3(grid), dim3(256), 0, stream, y, P, pos, weights, T, k, N, ad, o);
}

}  // namespace w4
