// w4_rmsnorm: RMS norm of bf16 rows with the residual's addition before it and
// the MXFP8 quantization of the result behind it.
//
// Mathematics, per row (include/w4.h has the exact semantics):
//     h = x + r,   y = h / sqrt(mean h^2 + eps) * gamma,
//     and per 32 elements of y  e = floor(log2 amax|y|) - 8,  code = e4m3(y / 2^e).
// A row is read once and kept in registers between the sum of squares and the
// scaling, so the traffic is the compulsory one: 2 (+ 2 for r) bytes read per
// element, 2 for H and 2 for Y or 1 + 1/32 for the codes and scales written.
// Unfused, the codes would cost another 2 + 2 bytes (Y out and in again).
//
// One row belongs to one CTA, or, when it is short, to one warp of a CTA; a
// thread holds up to VPT vectors of 8 elements, v = thread + i * threads, so
// every access of a warp is 512 contiguous bytes.  The four threads of a
// 32-element block are neighbours: its maximum takes two shuffles, and four
// blocks' scales leave as one 32-bit word.  The sum of squares runs in fp32:
// within a thread, then a butterfly over the warp, then over the CTA's warps
// through shared memory, always in the same order.
//
// What bounds it: HBM.  8192 rows of 8192, residual: MXFP8 out (472 MB) 77 to 81
// us on two B200s, 5.8 to 6.1 TB/s, 89 to 93% of the measured copy rate (with x
// and r loaded one after the other 110); bf16 out (537 MB) 82 us, the copy rate.
// 8192 rows of 5003, residual, bf16 out (328 MB): 62 us, 81%; gamma comes in single
// elements there.  One row of 4096: 1.9 us in a graph, launch and latency.
//
// Rounding: everything between the bf16 inputs and the outputs is fp32.  h is
// rounded to bf16 for H alone; the norm uses the fp32 sum, and the codes are
// rounded from the fp32 y, so no output carries a second rounding.
#include "mx_layout.cuh"

#include <cuda_fp8.h>

namespace w4 {
namespace {

struct NormArgs {
    const __nv_bfloat16 *x, *r, *gamma;
    __nv_bfloat16 *h, *y;
    uint8_t *codes, *scales;
    int64_t M;
    int K, mma, sf_words, in_place;   // sf_words: scales leave in 32-bit words; in_place: an output over an input
    float eps;
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The row's sum over the threads that share it: one warp, or all `warps` warps
// of the CTA.
__device__ __forceinline__ float row_sum(float v, int warps)
{
    __shared__ float part[32];
    v = warp_sum(v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.f);
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16lo_to_f32(w[j]);
        f[2 * j + 1] = bf16hi_to_f32(w[j]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *(const uint32_t *)&p;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of 16-byte vectors.  `warps` warps share a row: 1 (each warp of the CTA
// has a row of its own) or all of the CTA's.  With SHIFT rows are no whole
// vectors: a row begins `o` elements behind a vector's start, its vectors are
// those that hold any of it, elements of other rows count as 0 and are not
// written (bf16 out only).
template <int VPT, bool SHIFT>
__global__ void __launch_bounds__(1024 / (VPT > 2 ? 2 : 1)) rmsnorm_vec_kernel(NormArgs a, int64_t rows, int warps)
{
    pdl_wait();
    pdl_launch_dependents();
    const int threads = warps * 32;
    const int t = warps == 1 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = warps == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= rows) return;                          // (whole warps, and with warps > 1 whole CTAs)
    if (row >= a.M) {                                 // pads the last band of the tensor-core layout
        for (int kb = 4 * t; kb < a.K >> 5; kb += 4 * threads) *(uint32_t *)(a.scales + mma_sf_offset(row, kb, a.K)) = 0u;
        return;
    }
    const int o = SHIFT ? (int)((row * a.K) & 7) : 0;
    const int nv = SHIFT ? (o + a.K + 7) >> 3 : a.K >> 3;   // vectors of a row
    const int64_t v0 = (row * a.K) >> 3;                    // the first
    // The vectors lo .. lo + whole - 1 are loaded as such: those inside the arrays, and, where an output lies over
    // an input, inside the row (another CTA may be writing the other row's part of a shared one).
    const int lo = SHIFT && a.in_place && o > 0;
    const int whole = !SHIFT ? nv : a.in_place ? max(((o + a.K) >> 3) - lo, 0)
                                               : (int)min(((a.M * a.K) >> 3) - v0, (int64_t)nv);
    auto load = [&](const __nv_bfloat16 *p, int v) {
        if ((unsigned)(v - lo) < (unsigned)whole) return ((const uint4 *)p)[v0 + v];
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (SHIFT && v < nv) {                              // this row's elements alone
            const int k = 8 * v - o;
            for (int64_t e = row * a.K + max(k, 0); e < row * a.K + min(k + 8, a.K); ++e)
                w[(e & 7) >> 1] |= (uint32_t)__bfloat16_as_ushort(p[e]) << (16 * (e & 1));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    auto store = [&](__nv_bfloat16 *p, int v, const float (&f)[8]) {
        const int k = 8 * v - o;
        if (!SHIFT || (k >= 0 && k + 8 <= a.K)) ((uint4 *)p)[v0 + v] = pack8(f);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j >= 0 && k + j < a.K) p[row * a.K + k + j] = __float2bfloat16_rn(f[j]);
    };
    float f[VPT][8];
    float ss = 0.f;
    uint4 xv[VPT], rv[VPT];                                 // (all in flight before any is looked at)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        xv[i] = load(a.x, t + i * threads);
        rv[i] = a.r ? load(a.r, t + i * threads) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float g[8];
        unpack8(xv[i], f[i]);
        unpack8(rv[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] += g[j];
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = 8 * (t + i * threads) - o + j;
            if (SHIFT && (k < 0 || k >= a.K)) f[i][j] = 0.f;
            ss = fmaf(f[i][j], f[i][j], ss);
        }
    const float inv = 1.0f / sqrtf(row_sum(ss, warps) / (float)a.K + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = t + i * threads;
        const bool in = v < nv;
        if (a.h && in) store(a.h, v, f[i]);
        float g[8];
        if (SHIFT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = 8 * v - o + j;
                g[j] = k >= 0 && k < a.K ? __bfloat162float(__ldg(a.gamma + k)) : 0.f;
            }
        } else {
            unpack8(in ? __ldg((const uint4 *)a.gamma + v) : make_uint4(0u, 0u, 0u, 0u), g);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * inv * g[j];
        if (a.y && in) store(a.y, v, f[i]);
        if (!SHIFT && a.codes) {
            // amax as bit patterns (integer order = order of magnitudes), over the block's four threads
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[i][j]) & 0x7FFFFFFFu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const int e8 = max((int)(m >> 23) - 8, 0);                       // e + 127
            const float sc = __uint_as_float((uint32_t)(254 - e8) << 23);   // 2^-e
            uint32_t q[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
                    make_float2(f[i][4 * j] * sc, f[i][4 * j + 1] * sc), __NV_SATFINITE, __NV_E4M3);
                const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
                    make_float2(f[i][4 * j + 2] * sc, f[i][4 * j + 3] * sc), __NV_SATFINITE, __NV_E4M3);
                q[j] = (uint32_t)lo | ((uint32_t)hi << 16);
            }
            if (in) ((uint2 *)a.codes)[row * nv + v] = make_uint2(q[0], q[1]);
            const int kb = v >> 2;
            if (a.sf_words) {
                // four blocks' scales (16 lanes) as one word
                uint32_t word = (uint32_t)e8 << (8 * (kb & 3));
                word |= __shfl_xor_sync(0xffffffffu, word, 4);
                word |= __shfl_xor_sync(0xffffffffu, word, 8);
                if (in && (v & 15) == 0)
                    *(uint32_t *)(a.scales + (a.mma ? mma_sf_offset(row, kb, a.K) : row * (a.K >> 5) + kb)) = word;
            } else if (in && (v & 3) == 0) {
                a.scales[row * (a.K >> 5) + kb] = (uint8_t)e8;
            }
        }
    }
}

// Pointers that are not 16-byte aligned: one element per thread and step, bf16
// out only.
__global__ void __launch_bounds__(1024) rmsnorm_any_kernel(NormArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const __nv_bfloat16 *x = a.x + row * a.K, *r = a.r + row * a.K;
    float f[32];                                      // K <= 32 * 1024
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int k = threadIdx.x + i * blockDim.x;
        f[i] = 0.f;
        if (k < a.K) {
            f[i] = __bfloat162float(x[k]);
            if (a.r) f[i] += __bfloat162float(r[k]);
        }
        ss = fmaf(f[i], f[i], ss);
    }
    const float inv = 1.0f / sqrtf(row_sum(ss, blockDim.x >> 5) / (float)a.K + a.eps);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int k = threadIdx.x + i * blockDim.x;
        if (k < a.K) {
            if (a.h) a.h[row * a.K + k] = __float2bfloat16_rn(f[i]);
            a.y[row * a.K + k] = __float2bfloat16_rn(f[i] * inv * __bfloat162float(a.gamma[k]));
        }
    }
}

// Threads for nv vectors a row.  Few rows: a vector a thread, so that a row's
// latency is one load deep.  Many rows: four, so that a resident CTA has more
// bytes on their way (8192 rows of 8192, MXFP8 out, residual: 77 us with four,
// 99 with two); rows of up to 128 vectors then have a warp each.
template <bool SHIFT>
cudaError_t launch_vec(const NormArgs &a, int64_t rows, int nv, cudaStream_t stream)
{
    const bool many = rows > 2 * kNumSMs;
    const int vpt = many ? (nv <= 32 ? 1 : nv <= 64 ? 2 : 4) : nv <= 1024 ? 1 : nv <= 2048 ? 2 : 4;
    int warps = (nv + 32 * vpt - 1) / (32 * vpt);
    const int per_cta = warps == 1 ? 8 : 1;           // rows
    if (nv > 2048) {                                  // 512 threads; a shifted row of 32767 has 4097 vectors
        constexpr int kLong = SHIFT ? 9 : 8;
        warps = (nv + 32 * kLong - 1) / (32 * kLong);
        return launch_pdl(rmsnorm_vec_kernel<kLong, SHIFT>, dim3((unsigned)rows), dim3(warps * 32), 0, stream, a, rows, warps);
    }
    const dim3 grid((unsigned)((rows + per_cta - 1) / per_cta)), block(warps * per_cta * 32);
    if (vpt == 1) return launch_pdl(rmsnorm_vec_kernel<1, SHIFT>, grid, block, 0, stream, a, rows, warps);
    if (vpt == 2) return launch_pdl(rmsnorm_vec_kernel<2, SHIFT>, grid, block, 0, stream, a, rows, warps);
    return launch_pdl(rmsnorm_vec_kernel<4, SHIFT>, grid, block, 0, stream, a, rows, warps);
}

}  // namespace

cudaError_t launch_rmsnorm(const void *X, const void *residual, const void *gamma, int64_t M, int64_t K, float eps,
                           void *H, void *Y, uint8_t *codes, uint8_t *scales, int layout, cudaStream_t stream)
{
    const int mma = codes && layout == W4_MX_SCALES_MMA;
    NormArgs a = {(const __nv_bfloat16 *)X, (const __nv_bfloat16 *)residual, (const __nv_bfloat16 *)gamma,
                  (__nv_bfloat16 *)H, (__nv_bfloat16 *)Y, codes, scales, M, (int)K,
                  mma, K % 128 == 0 && (uintptr_t)scales % 4 == 0, Y == X || (H && (H == X || H == residual)), eps};
    const uintptr_t all = (uintptr_t)X | (uintptr_t)residual | (uintptr_t)gamma | (uintptr_t)H | (uintptr_t)Y;
    if (all % 16 != 0) {
        const int threads = K >= 1024 ? 1024 : (int)((K + 31) / 32 * 32);
        return launch_pdl(rmsnorm_any_kernel, dim3((unsigned)M), dim3(threads), 0, stream, a);
    }
    const int64_t rows = mma ? mx_padded_rows(M) : M;
    return K % 8 != 0 ? launch_vec<true>(a, rows, (int)(K + 14) / 8, stream) : launch_vec<false>(a, rows, (int)(K / 8), stream);
}

}  // namespace w4
