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
//
// Bound by memory for many rows: 2048 x 4096 bf16 with residual 13 us (58.7 MB, 4.4 TB/s; of it about
// 2.5 us launch and tail), 8192 rows 39 us (6.0 TB/s), 4096 x 11008 bf16 without norm 28 us (4.8 TB/s),
// 8191 x 16384 fp32 138 us (4.9 TB/s, w re-read from L2 for every row); by latency for few: 2.4 us for one
// row, 2.8 us for 64.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"

namespace gq {

struct RowsArgs {
    const void* X;       // [M, D]
    const void* R;       // [M, D] or null
    const void* w;       // [D], norm only
    uint8_t* X8;         // [M, D]
    float* x_scale;      // [M]
    void* R2;            // [M, D], with R
    long long D, M;
    float eps;
    int warp_rows;       // a warp per row, not a CTA
};

// Eight elements as loaded, so that a thread's loads can all be in flight before the first is used.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p, bool valid) {
        u = make_uint4(0, 0, 0, 0);
        if (valid) u = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ float at(int i) const {
        const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p, bool valid) {
        a = b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (valid) {
            a = *reinterpret_cast<const float4*>(p);
            b = *reinterpret_cast<const float4*>(p + 4);
        }
    }
    __device__ __forceinline__ float at(int i) const {
        const float4 q = i < 4 ? a : b;
        return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
    }
};
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
// What turns a row into codes: 448 v / a = (v f) (hi + lo), with 448 / (a f) = hi + lo to 48 bits.
struct RowScale {
    float f, hi, lo;
};
// 448 v / a for eight values, rounded to nearest even.  The quotient is rounded to fp32 once, from 48
// bits: where it lies on the boundary between two codes, which happens often with bf16 rows, it is exact.
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], const RowScale& s) {
    auto q = [&](int i) {
        const float t = v[i] * s.f;
        return fmaf(t, s.hi, t * s.lo);
    };
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo =
            __nv_cvt_float2_to_fp8x2(make_float2(q(4 * i), q(4 * i + 1)), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi =
            __nv_cvt_float2_to_fp8x2(make_float2(q(4 * i + 2), q(4 * i + 3)), __NV_SATFINITE, __NV_E4M3);
        r[i] = lo | (hi << 16);
    }
    return make_uint2(r[0], r[1]);
}

// Joins the threads' sums and maxima over the warp or the block (up to 1024 threads), the same bits on
// every run.
template <bool NORM>
__device__ __forceinline__ void rows_join(float& sum, uint32_t& top, bool warp_only) {
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        if (NORM) sum += __shfl_xor_sync(~0u, sum, o);
        top = max(top, __shfl_xor_sync(~0u, top, o));
    }
    if (warp_only || warps == 1) return;
    if (lane == 0) {
        s_sum[warp] = sum;
        s_max[warp] = top;
    }
    __syncthreads();
    sum = lane < warps ? s_sum[lane] : 0.f;
    top = lane < warps ? s_max[lane] : 0u;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        if (NORM) sum += __shfl_xor_sync(~0u, sum, o);
        top = max(top, __shfl_xor_sync(~0u, top, o));
    }
}

template <bool NORM>
__device__ __forceinline__ RowScale row_scale(const RowsArgs& p, float sum, uint32_t top, float* x_scale, bool first) {
    const float a = __uint_as_float(top);
    if (first) {
        const float r = NORM ? rsqrtf(sum / (float)p.D + p.eps) : 1.f;
        *x_scale = a == 0.f ? 0.f : r * (a / 448.f);
    }
    // a below 2^-100 would overflow 448 / a: the row is lifted by 2^64 first, which is exact
    RowScale s;
    s.f = a < 0x1p-100f ? 0x1p64f : 1.f;
    s.hi = a > 0.f ? 448.f / (a * s.f) : (a == 0.f ? 0.f : a);
    s.lo = a > 0.f && a <= 0x1p100f ? fmaf(-s.hi, a * s.f, 448.f) * (s.hi * (1.f / 448.f)) : 0.f;
    return s;
}

constexpr int RW_MAX_VECS = 4096;   // vectors of 8 elements in a row of rows_e4m3_kernel, at most
// Threads of a CTA, at most, where a thread holds VEC vectors: 64 or 128 registers each.
__host__ __device__ constexpr int rw_max_threads(int vec) { return vec <= 2 ? 1024 : 512; }

// One CTA (or, for short rows, one warp) per row, the row in registers: VEC vectors of 8 elements a
// thread, so that X, R and w are read once, the loads of up to four vectors are in flight together, and
// R' is written before the maximum is known.
// R' may be X or R: a thread writes only elements that it has read itself.
template <typename XT, typename WT, bool NORM, int VEC>
__global__ void __launch_bounds__(rw_max_threads(VEC)) rows_e4m3_kernel(const RowsArgs p) {
    const bool wr = p.warp_rows != 0;
    const long long row = wr ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.M) return;   // whole warps
    const int t = wr ? threadIdx.x & 31 : threadIdx.x;
    const XT* X = reinterpret_cast<const XT*>(p.X) + row * p.D;
    const XT* R = p.R ? reinterpret_cast<const XT*>(p.R) + row * p.D : nullptr;
    const int D = (int)p.D, step = wr ? 8 * 32 : 8 * (int)blockDim.x, c0 = 8 * t;
    float v[VEC][8];
    float sum = 0.f;
    uint32_t top = 0;
    constexpr int FLIGHT = VEC > 4 ? 4 : VEC;   // vectors of each input in flight
#pragma unroll
    for (int i0 = 0; i0 < VEC; i0 += FLIGHT) {
        Raw8<XT> x[FLIGHT], r[FLIGHT];
        Raw8<WT> w[FLIGHT];
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) x[i].load(X + c0 + (i0 + i) * step, c0 + (i0 + i) * step < D);
        if (R) {
#pragma unroll
            for (int i = 0; i < FLIGHT; ++i) r[i].load(R + c0 + (i0 + i) * step, c0 + (i0 + i) * step < D);
        }
        if (NORM) {
#pragma unroll
            for (int i = 0; i < FLIGHT; ++i)
                w[i].load(reinterpret_cast<const WT*>(p.w) + c0 + (i0 + i) * step, c0 + (i0 + i) * step < D);
        }
#pragma unroll
        for (int i = 0; i < FLIGHT; ++i) {
            float(&h)[8] = v[i0 + i];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = x[i].at(j);
            if (R) {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] += r[i].at(j);
                if (c0 + (i0 + i) * step < D) store8(reinterpret_cast<XT*>(p.R2) + row * p.D + c0 + (i0 + i) * step, h);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (NORM) {
                    sum = fmaf(h[j], h[j], sum);
                    h[j] *= w[i].at(j);
                }
                top = max(top, __float_as_uint(h[j]) & 0x7FFFFFFFu);
            }
        }
    }
    rows_join<NORM>(sum, top, wr);
    const RowScale s = row_scale<NORM>(p, sum, top, p.x_scale + row, t == 0);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int c = c0 + i * step;
        if (c < D) *reinterpret_cast<uint2*>(p.X8 + row * p.D + c) = e4m3x8(v[i], s);
    }
}

// Rows too long for that: read twice, R' written in the second pass, when the thread that writes an
// element has read its X and R.
template <typename XT, typename WT, bool NORM>
__global__ void __launch_bounds__(1024) rows_e4m3_long_kernel(const RowsArgs p) {
    const long long row = blockIdx.x;
    const XT* X = reinterpret_cast<const XT*>(p.X) + row * p.D;
    const XT* R = p.R ? reinterpret_cast<const XT*>(p.R) + row * p.D : nullptr;
    const WT* W = reinterpret_cast<const WT*>(p.w);
    const int D = (int)p.D, step = 8 * (int)blockDim.x;
    float sum = 0.f;
    uint32_t top = 0;
    float h[8], w[8];
    auto load8 = [](const auto* q, float (&to)[8]) {
        Raw8<std::remove_cv_t<std::remove_pointer_t<decltype(q)>>> raw;
        raw.load(q, true);
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i] = raw.at(i);
    };
    auto read = [&](int c) {
        load8(X + c, h);
        if (R) {
            load8(R + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] += w[i];
        }
    };
    for (int c = 8 * (int)threadIdx.x; c < D; c += step) {
        read(c);
        if (NORM) load8(W + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (NORM) sum = fmaf(h[i], h[i], sum);
            top = max(top, __float_as_uint(NORM ? h[i] * w[i] : h[i]) & 0x7FFFFFFFu);
        }
    }
    rows_join<NORM>(sum, top, false);
    const RowScale s = row_scale<NORM>(p, sum, top, p.x_scale + row, threadIdx.x == 0);
    for (int c = 8 * (int)threadIdx.x; c < D; c += step) {
        read(c);
        if (R) store8(reinterpret_cast<XT*>(p.R2) + row * p.D + c, h);
        if (NORM) {
            load8(W + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] *= w[i];
        }
        *reinterpret_cast<uint2*>(p.X8 + row * p.D + c) = e4m3x8(h, s);
    }
}

}  // namespace gq

namespace gqh {

int num_sms();

template <typename XT, typename WT, bool NORM>
cudaError_t rows_e4m3_run(gq::RowsArgs p, long long M, const char* name, cudaStream_t st) {
    TimedScope ts__(name, st);
    dim3 grid((unsigned)M);
    const int vecs = (int)(p.D / 8);
    p.M = M;
    // Ordinary launches: what precedes a public call may be anything, a wait for another stream included.
    if (vecs > gq::RW_MAX_VECS)
        return launch_plain(gq::rows_e4m3_long_kernel<XT, WT, NORM>, grid, dim3(1024), 0, st, p);
    // Few rows: a vector a thread, for latency.  Many rows: four, for bytes in flight and cheap barriers;
    // eight for long rows without R, whose registers they leave enough of (4096 x 11008 bf16: 28 us against
    // 32 us with four; with R they do not: 2048 x 11008 took 37 us against 29 us).
    const bool few = M <= 2 * num_sms();
    int vec = few ? 1 : p.R == nullptr && vecs > 512 ? 8 : 4, threads;
    while (vec * gq::rw_max_threads(vec) < vecs) vec *= 2;
    threads = ((vecs + vec - 1) / vec + 31) / 32 * 32;
    p.warp_rows = !few && threads == 32;   // short rows: eight to a CTA, which starts as fast as one row's
    if (p.warp_rows) {
        while (vec > 1 && vec * 16 >= vecs) vec /= 2;
        threads = 256;
        grid.x = (unsigned)((M + 7) / 8);
    }
    switch (vec) {
        case 1: return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 1>, grid, dim3(threads), 0, st, p);
        case 2: return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 2>, grid, dim3(threads), 0, st, p);
        case 4: return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 4>, grid, dim3(threads), 0, st, p);
        default: return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 8>, grid, dim3(threads), 0, st, p);
    }
}

}  // namespace gqh
