// The rows of a product by expert: which expert and which of its rows a CTA
// works on, read from the plan on the device.
#pragma once

#include "common.cuh"

namespace w4 {

// The plan of w4a16_experts_gemm: rows offsets[e] .. offsets[e + 1] - 1 belong
// to expert e; row i reads row order[i] / top_k of X (row i without `order`).
struct ExpertPlan {
    const int *offsets, *order;
    int top_k, E, R, P;
};

// `rows` rows of expert `expert` from sorted row `row0` on.
struct ExpertUnit {
    int expert, row0, rows;
};

namespace {

// Unit number `unit` when each expert's rows are cut into runs of `chunk`;
// rows = 0 when there are fewer units.  Called by whole warps; every warp of a
// CTA finds the same unit.  Offsets outside [0, P] count as the nearest end.
__device__ __forceinline__ ExpertUnit find_unit(const ExpertPlan &p, int unit, int chunk)
{
    const int lane = threadIdx.x & 31;
    ExpertUnit u = {0, 0, 0};
    int next_lo = lane < p.E ? p.offsets[lane] : 0, next_hi = lane < p.E ? p.offsets[lane + 1] : 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int lo = min(max(next_lo, 0), p.P), hi = min(max(next_hi, 0), p.P);
        const int e = e0 + 32 + lane;                 // (asked for a round ahead)
        next_lo = e < p.E ? p.offsets[e] : 0;
        next_hi = e < p.E ? p.offsets[e + 1] : 0;
        const int n = max(hi - lo, 0), units = n / chunk + (n % chunk != 0);
        int upto = units;                             // units of the experts e0 .. e
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        const unsigned after = __ballot_sync(0xffffffffu, unit < upto);
        if (after) {
            const int src = __ffs(after) - 1;
            const int first = (unit - (__shfl_sync(0xffffffffu, upto, src) - __shfl_sync(0xffffffffu, units, src))) * chunk;
            u.expert = e0 + src;
            u.row0 = __shfl_sync(0xffffffffu, lo, src) + first;
            u.rows = min(chunk, __shfl_sync(0xffffffffu, n, src) - first);
            return u;
        }
        unit -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return u;
}

// The row of X behind sorted row i.
__device__ __forceinline__ int expert_x_row(const ExpertPlan &p, int i)
{
    const int row = p.order ? p.order[i] / p.top_k : i;
    return min(max(row, 0), p.R - 1);
}

}  // namespace

// Units of at most `chunk` rows that P rows of E experts can need.
inline int64_t max_units(int64_t P, int64_t E, int64_t chunk)
{
    return P / chunk + (P < E ? P : E);
}

}  // namespace w4
