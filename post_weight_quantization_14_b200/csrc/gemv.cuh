// Products of a few tokens with packed weights (decoding):
//
//   Y[m, n] = xs[m] sum_k X[m, k] W_hat[n, k],   W_hat[n, k] = s[g(k), n] (q[n, k] - z[g(k), n])
//
// with g(k) = k / g, or g_idx[k] for layers quantized in activation order.  X is bf16 (xs = 1)
// or e4m3 with one fp32 scale per row.
//
// One lane per output row n; eight warps share the rows of a CTA and split the columns k in
// equal runs, whose sums are joined through shared memory in a fixed order.  q - z and
// s (q - z) (at most 11 + 8 significant bits) are exact in fp32; sums are fp32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "pack.cuh"

namespace gq {

__device__ __forceinline__ float to_float(const __nv_bfloat16& v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(const float& v) { return v; }
__device__ __forceinline__ float to_float(const __nv_fp8_e4m3& v) { return (float)v; }

struct GemvArgs {
    const void* X;            // [M, K]
    const float* x_scale;     // [M] or null
    const int32_t* qweight;   // [ceil(K bits / 32), N]
    const __half* scales;     // [n_groups, N]
    const int32_t* qzeros;    // [n_groups, ceil(N bits / 32)] or null
    const int32_t* g_idx;     // [K] or null
    void* Y;                  // [M, N]
    int y_bf16;
    int M;
    long long N, K;
    int g, ng;                // group length and count
    int bits;
    unsigned nblocks;         // blocks of rows n
};

constexpr int GV_WARPS = 8, GV_TOK = 4;

template <typename XT>
__global__ void __launch_bounds__(32 * GV_WARPS) gemv_lane_kernel(const GemvArgs p) {
    __shared__ float part[GV_WARPS][GV_TOK][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long n = (long long)(blockIdx.x % p.nblocks) * 32 + lane;
    const int m0 = (int)(blockIdx.x / p.nblocks) * GV_TOK;
    const long long zwords = (p.N * p.bits + 31) / 32;
    const long long run = (p.K + GV_WARPS - 1) / GV_WARPS;
    const long long k0 = warp * run, k1 = min(p.K, k0 + run);
    const XT* X = reinterpret_cast<const XT*>(p.X);
    float acc[GV_TOK] = {};
    if (n < p.N) {
        long long have = -1;
        float s = 0.f, z = (float)(1 << (p.bits - 1));
        for (long long k = k0; k < k1; ++k) {
            long long gi = p.g_idx ? p.g_idx[k] : k / p.g;
            if (gi < 0 || gi >= p.ng) {
                record_status(GPTQ_ERR_INVALID_ARG, k);
                gi = 0;
            }
            if (gi != have) {
                have = gi;
                s = __half2float(p.scales[gi * p.N + n]);
                if (p.qzeros) z = (float)stream_code(p.qzeros + gi * zwords, 1, n, p.bits);
            }
            const float w = s * ((float)stream_code(p.qweight + n, p.N, k, p.bits) - z);
#pragma unroll
            for (int t = 0; t < GV_TOK; ++t)
                if (m0 + t < p.M) acc[t] = fmaf(to_float(X[(long long)(m0 + t) * p.K + k]), w, acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < GV_TOK; ++t) part[warp][t][lane] = acc[t];
    __syncthreads();
    if (warp < GV_TOK && m0 + warp < p.M && n < p.N) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < GV_WARPS; ++w) y += part[w][warp][lane];
        const int m = m0 + warp;
        if (p.x_scale) y *= p.x_scale[m];
        const long long at = (long long)m * p.N + n;
        if (p.y_bf16)
            reinterpret_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(y);
        else
            reinterpret_cast<float*>(p.Y)[at] = y;
    }
}

}  // namespace gq

namespace gqh {

inline cudaError_t gemv_run(gq::GemvArgs p, bool x_e4m3, cudaStream_t st) {
    TimedScope ts__("dequant_gemv", st);
    p.nblocks = (unsigned)((p.N + 31) / 32);
    const long long blocks = (long long)p.nblocks * ((p.M + gq::GV_TOK - 1) / gq::GV_TOK);
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    return x_e4m3 ? launch_plain(gq::gemv_lane_kernel<__nv_fp8_e4m3>, grid, dim3(32 * gq::GV_WARPS), 0, st, p)
                  : launch_plain(gq::gemv_lane_kernel<__nv_bfloat16>, grid, dim3(32 * gq::GV_WARPS), 0, st, p);
}

}  // namespace gqh
