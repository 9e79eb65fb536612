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
    int K, mma;
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
// has a row of its own) or all of the CTA's.
template <int VPT>
__global__ void __launch_bounds__(1024 / (VPT > 2 ? 2 : 1)) rmsnorm_vec_kernel(NormArgs a, int64_t rows, int warps)
{
    pdl_wait();
    pdl_launch_dependents();
    const int threads = warps * 32;
    const int t = warps == 1 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = warps == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= rows) return;                          // (whole warps, and with warps > 1 whole CTAs)
    const int nv = a.K >> 3;                          // vectors of a row
    if (row >= a.M) {                                 // pads the last band of the tensor-core layout
        for (int kb = t; kb < a.K >> 5; kb += threads) a.scales[mma_sf_offset(row, kb, a.K)] = 0;
        return;
    }
    const uint4 *x = (const uint4 *)a.x + row * nv;
    const uint4 *r = (const uint4 *)a.r + row * nv;
    float f[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = t + i * threads;
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (v < nv) u = x[v];
        unpack8(u, f[i]);
    }
    if (a.r) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * threads;
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (v < nv) u = r[v];
            float g[8];
            unpack8(u, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] += g[j];
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(f[i][j], f[i][j], ss);
    const float inv = 1.0f / sqrtf(row_sum(ss, warps) / (float)a.K + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = t + i * threads;
        const bool in = v < nv;
        if (a.h && in) ((uint4 *)a.h)[row * nv + v] = pack8(f[i]);
        float g[8];
        unpack8(in ? __ldg((const uint4 *)a.gamma + v) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * inv * g[j];
        if (a.y && in) ((uint4 *)a.y)[row * nv + v] = pack8(f[i]);
        if (a.codes) {
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
            if (in) {
                ((uint2 *)a.codes)[row * nv + v] = make_uint2(q[0], q[1]);
                if ((v & 3) == 0) {
                    const int kb = v >> 2;
                    const int64_t at = a.mma ? mma_sf_offset(row, kb, a.K) : row * (a.K >> 5) + kb;
                    a.scales[at] = (uint8_t)e8;
                }
            }
        }
    }
}

// Rows that are no whole vectors, or pointers that are not 16-byte aligned:
// one element per thread and step, bf16 out only.
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

}  // namespace

cudaError_t launch_rmsnorm(const void *X, const void *residual, const void *gamma, int64_t M, int64_t K, float eps,
                           void *H, void *Y, uint8_t *codes, uint8_t *scales, int layout, cudaStream_t stream)
{
    NormArgs a = {(const __nv_bfloat16 *)X, (const __nv_bfloat16 *)residual, (const __nv_bfloat16 *)gamma,
                  (__nv_bfloat16 *)H, (__nv_bfloat16 *)Y, codes, scales, M, (int)K,
                  codes && layout == W4_MX_SCALES_MMA, eps};
    const uintptr_t all = (uintptr_t)X | (uintptr_t)residual | (uintptr_t)gamma | (uintptr_t)H | (uintptr_t)Y;
    if (K % 8 != 0 || all % 16 != 0) {
        const int threads = K >= 1024 ? 1024 : (int)((K + 31) / 32 * 32);
        return launch_pdl(rmsnorm_any_kernel, dim3((unsigned)M), dim3(threads), 0, stream, a);
    }
    const int64_t rows = a.mma ? mx_padded_rows(M) : M;
    const int nv = (int)(K / 8);
    if (nv <= 64) {
        const dim3 grid((unsigned)((rows + 7) / 8));
        if (nv <= 32) return launch_pdl(rmsnorm_vec_kernel<1>, grid, dim3(256), 0, stream, a, rows, 1);
        return launch_pdl(rmsnorm_vec_kernel<2>, grid, dim3(256), 0, stream, a, rows, 1);
    }
    const int vpt = nv <= 1024 ? 1 : nv <= 2048 ? 2 : 8;
    const int warps = (nv + 32 * vpt - 1) / (32 * vpt);
    const dim3 grid((unsigned)rows), block(warps * 32);
    if (vpt == 1) return launch_pdl(rmsnorm_vec_kernel<1>, grid, block, 0, stream, a, rows, warps);
    if (vpt == 2) return launch_pdl(rmsnorm_vec_kernel<2>, grid, block, 0, stream, a, rows, warps);
    return launch_pdl(rmsnorm_vec_kernel<8>, grid, block, 0, stream, a, rows, warps);
}

}  // namespace w4
