// Rows to e4m3 with one fp32 scale per row, alone or after a residual addition and a
// root-mean-square norm:
//
//   h = X (+ R),   v = h w  (v = h without a norm),   a = max_k |v_k|,
//   r = 1 / sqrt(mean(h^2) + eps)  (r = 1 without a norm),
//   x_scale = r a / 448,   X8 = e4m3(448 v / a),   R' = h rounded to R's type.
//
// r is positive and common to a row, so it scales a but cancels from the codes: one sum and one
// maximum per row suffice, and they are taken together.  |v| is compared by its bit pattern,
// whose order is that of the magnitudes with NaN above infinity, so a NaN reaches x_scale.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace gq {

struct RowsArgs {
    const void* X;       // [M, D]
    const void* R;       // [M, D] or null
    const void* w;       // [D], norm only
    uint8_t* X8;         // [M, D]
    float* x_scale;      // [M]
    void* R2;            // [M, D], with R
    long long D;
    float eps;
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
// 448 v / a for eight values, rounded to nearest even.
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float f, float inv) {
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(v[4 * i] * f * inv, v[4 * i + 1] * f * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(v[4 * i + 2] * f * inv, v[4 * i + 3] * f * inv), __NV_SATFINITE, __NV_E4M3);
        r[i] = lo | (hi << 16);
    }
    return make_uint2(r[0], r[1]);
}

constexpr int RW_THREADS = 256;

// One CTA per row, the row read twice.  A residual sum is read back from R' unless R' would
// lose its low bits, so both passes form h from X and R; R' is written in the second pass, when
// every element's own X and R have been read by the thread that writes it.
template <typename XT, typename WT, bool NORM>
__global__ void __launch_bounds__(RW_THREADS) rows_e4m3_kernel(const RowsArgs p) {
    __shared__ float s_sum[RW_THREADS / 32];
    __shared__ uint32_t s_max[RW_THREADS / 32];
    const long long row = blockIdx.x;
    const XT* X = reinterpret_cast<const XT*>(p.X) + row * p.D;
    const XT* R = p.R ? reinterpret_cast<const XT*>(p.R) + row * p.D : nullptr;
    const WT* W = reinterpret_cast<const WT*>(p.w);
    float sum = 0.f;
    uint32_t top = 0;
    float h[8], w[8];
    auto read = [&](long long c) {
        load8(X + c, h);
        if (R) {
            load8(R + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] += w[i];
        }
    };
    for (long long c = 8ll * threadIdx.x; c < p.D; c += 8 * RW_THREADS) {
        read(c);
        if (NORM) load8(W + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (NORM) sum = fmaf(h[i], h[i], sum);
            top = max(top, __float_as_uint(NORM ? h[i] * w[i] : h[i]) & 0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        top = max(top, __shfl_xor_sync(~0u, top, o));
    }
    if ((threadIdx.x & 31) == 0) {
        s_sum[threadIdx.x >> 5] = sum;
        s_max[threadIdx.x >> 5] = top;
    }
    __syncthreads();
    sum = 0.f;
    top = 0;
#pragma unroll
    for (int i = 0; i < RW_THREADS / 32; ++i) {
        sum += s_sum[i];
        top = max(top, s_max[i]);
    }
    const float a = __uint_as_float(top);
    // a below 2^-100 would overflow 448 / a: the row is lifted by 2^64 first, which is exact
    const float f = a < 0x1p-100f ? 0x1p64f : 1.f;
    const float inv = a > 0.f ? 448.f / (a * f) : (a == 0.f ? 0.f : a);
    if (threadIdx.x == 0) {
        const float r = NORM ? rsqrtf(sum / (float)p.D + p.eps) : 1.f;
        p.x_scale[row] = a == 0.f ? 0.f : r * (a / 448.f);
    }
    for (long long c = 8ll * threadIdx.x; c < p.D; c += 8 * RW_THREADS) {
        read(c);
        if (R) store8(reinterpret_cast<XT*>(p.R2) + row * p.D + c, h);
        if (NORM) {
            load8(W + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] *= w[i];
        }
        *reinterpret_cast<uint2*>(p.X8 + row * p.D + c) = e4m3x8(h, f, inv);
    }
}

}  // namespace gq

namespace gqh {

template <typename XT, typename WT, bool NORM>
cudaError_t rows_e4m3_run(const gq::RowsArgs& p, long long M, const char* name, cudaStream_t st) {
    TimedScope ts__(name, st);
    return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM>, dim3((unsigned)M), dim3(gq::RW_THREADS), 0, st, p);
}

}  // namespace gqh
