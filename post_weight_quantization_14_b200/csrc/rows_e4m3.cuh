// Rows to e4m3 with one fp32 scale per row, alone or after a residual addition and a
// root-mean-square norm:
//
//   h = X (+ R),   v = h w  (v = h without a norm),   a = max_k |v_k|,
//   r = 1 / sqrt(mean(h^2) + eps)  (r = 1 without a norm; the sum in fp32, see SquareSum for its range),
//   x_scale = r a / 448,   X8 = e4m3(448 v / a),   R' = h rounded to R's type.
//
// r is positive and common to a row, so it scales a but cancels from the codes: one sum and one
// maximum per row suffice, and they are taken together.  |v| is compared by its bit pattern,
// whose order is that of the magnitudes with NaN above infinity, so a NaN reaches x_scale.
//
// Bound by memory for many rows: 2048 x 4096 bf16 with residual 12 us (58.7 MB, 4.9 TB/s; of it about
// 2.5 us launch and tail), 8192 rows 37.6 us (6.2 TB/s), 4096 x 11008 bf16 without norm 24 us (5.6 TB/s),
// 8191 x 16384 fp32 123 us (5.5 TB/s); by latency for few: 2.4 us for one row, 2.7 us for 64.  Long rows
// (512 x 65536 bf16 with residual) take 63 us; without the code for sums that fp32 does not hold, 57 us.
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

// A row's sum of squares where fp32 may not hold it.  Where a thread's running sum ``mid`` leaves
// [2^-100, 2^110] (values from about 2^55 on, or below 2^-50 alone) its values so far go into ``far``
// instead, scaled by a power of two: positive, the sum of (2^-76 h)^2; or negative, the sum of (2^90 h)^2,
// which one large value makes negligible.  Both hold the squares of every fp32 value, for any row length here.
struct SquareSum {
    float mid = 0.f, far = 0.f;
    template <int N>
    __device__ __forceinline__ void add(const float (*h)[8]) {
        const float before = mid;
#pragma unroll
        for (int i = 0; i < N; ++i) {   // N chains side by side
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(h[i][j], h[i][j], s);
            mid += s;
        }
        if (!(mid >= 0x1p-100f && mid <= 0x1p110f)) {   // a NaN as well
            const bool low = mid < 0x1p-100f;
            const float by = low ? 0x1p90f : 0x1p-76f;
            float s = before * by * by;
#pragma unroll
            for (int i = 0; i < 8 * N; ++i) {
                const float t = h[i >> 3][i & 7] * by;
                s = fmaf(t, t, s);
            }
            if (low)
                far = far <= 0.f ? far - s : far;   // a NaN stays
            else
                far = far <= 0.f ? s : far + s;
            mid = 0.f;
        }
    }
    // Adds up the warp's lanes.
    __device__ __forceinline__ void join() {
        float high = far <= 0.f ? 0.f : far, low = fminf(far, 0.f);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            mid += __shfl_xor_sync(~0u, mid, o);
            high += __shfl_xor_sync(~0u, high, o);
            low += __shfl_xor_sync(~0u, low, o);
        }
        far = high != 0.f ? high : low;
    }
    // The same over the block.
    __device__ __forceinline__ void join_block() {
        __shared__ float s_parts[2][32];
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
            s_parts[0][warp] = mid;
            s_parts[1][warp] = far;
        }
        __syncthreads();
        mid = lane < warps ? s_parts[0][lane] : 0.f;
        far = lane < warps ? s_parts[1][lane] : 0.f;
        join();
    }
    // a / (448 sqrt(sum / D + eps)).  The factors of two are shared out so that nothing leaves the range of fp32.
    __device__ __forceinline__ float scale(float a, float D, float eps) const {
        if (!(far <= 0.f))   // mid is nothing to it
            return a * 0x1p-45f / 448.f * rsqrtf(far / D + eps * 0x1p-76f * 0x1p-76f) * 0x1p-31f;
        if (far < 0.f && mid < 0x1p-60f && eps < 0x1p-60f)
            return a * 0x1p45f / 448.f * rsqrtf((mid * 0x1p90f * 0x1p90f - far) / D + eps * 0x1p90f * 0x1p90f) * 0x1p45f;
        return rsqrtf(mid / D + eps) * (a / 448.f);   // far is nothing to mid or eps
    }
};

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
// Whether fp32 did not hold the row's sum: too large, or too small beside eps (a NaN as well).
__device__ __forceinline__ bool sum_lost(float sum, float eps) {
    return !(fmaxf(sum, eps) >= 0x1p-60f && sum <= 0x1p120f);
}

__device__ __forceinline__ RowScale row_scale(uint32_t top) {
    const float a = __uint_as_float(top);
    // a below 2^-100 would overflow 448 / a, one above 2^100 would leave lo subnormal: the row is moved by
    // 2^64 first, which is exact for values that have a code
    RowScale s;
    s.f = a < 0x1p-100f ? 0x1p64f : a > 0x1p100f ? 0x1p-64f : 1.f;
    s.hi = a > 0.f ? 448.f / (a * s.f) : (a == 0.f ? 0.f : a);
    s.lo = a > 0.f && a <= 0x1.fffffep127f ? fmaf(-s.hi, a * s.f, 448.f) * (s.hi * (1.f / 448.f)) : 0.f;
    return s;
}

template <bool NORM>
__device__ __forceinline__ float x_scale(const RowsArgs& p, const SquareSum& sum, uint32_t top) {
    const float a = __uint_as_float(top);
    return a == 0.f ? 0.f : NORM ? sum.scale(a, (float)p.D, p.eps) : a / 448.f;
}

constexpr int RW_MAX_VECS = 4096;   // vectors of 8 elements in a row of rows_e4m3_kernel, at most
// Threads of a CTA, at most, where a thread holds VEC vectors: 64 or 128 registers each.
__host__ __device__ constexpr int rw_max_threads(int vec) { return vec <= 2 ? 1024 : 512; }

// One CTA (or, for short rows, one warp) per row, the row in registers: VEC vectors of 8 elements a
// thread, so that X, R and w are read once, the loads of up to four vectors are in flight together, and
// R' is written before the maximum is known.
// R' may be X or R: a thread writes only elements that it has read itself.
// Rows whose sum fp32 does not hold are read again: from X, or from R', which holds fp32 values exactly.
// bf16 R' does not and may have replaced X, so with KEEP the values stay in registers until a thread's sum
// is known to be in range.  RES: there may be an R.  Eight vectors need the registers of both: 8191 x 16384
// fp32 without R takes 122 us, 151 us with KEEP, 174 us with RES; 1024 x 32768 fp32 with R takes 79 us with
// KEEP, 90 us without.
template <typename XT, typename WT, bool NORM, int VEC, bool KEEP, bool RES>
__global__ void __launch_bounds__(rw_max_threads(VEC), VEC == 1 && sizeof(XT) + sizeof(WT) == 4 ? 2 : 0)
    rows_e4m3_kernel(const RowsArgs p) {
    const bool wr = p.warp_rows != 0;
    const long long row = wr ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.M) return;   // whole warps
    const int t = wr ? threadIdx.x & 31 : threadIdx.x;
    const XT* X = reinterpret_cast<const XT*>(p.X) + row * p.D;
    const XT* R = RES && p.R ? reinterpret_cast<const XT*>(p.R) + row * p.D : nullptr;
    const int D = (int)p.D, step = wr ? 8 * 32 : 8 * (int)blockDim.x, c0 = 8 * t;
    float v[VEC][8];
    SquareSum kept;   // KEEP
    float sum = 0.f;
    uint32_t top = 0;
    // With a norm apart from the sums above, so that w may come last (4096 x 8192 bf16, fp32 w: 25 us against
    // 30 us); without one at once, for its registers (4096 x 11008 bf16: 24 us against 35 us).
    auto weigh = [&](float(&h)[8], const Raw8<WT>& w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (NORM && !KEEP) sum = fmaf(h[j], h[j], sum);
            if (NORM) h[j] *= w.at(j);
            top = max(top, __float_as_uint(h[j]) & 0x7FFFFFFFu);
        }
    };
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
            if (!NORM) weigh(h, w[i]);
        }
        if (KEEP) kept.add<FLIGHT>(v + i0);
        if (NORM) {
#pragma unroll
            for (int i = 0; i < FLIGHT; ++i) weigh(v[i0 + i], w[i]);
        }
    }
    if (KEEP) sum = kept.far == 0.f ? kept.mid : __int_as_float(0x7F800000);   // infinity: not held
    rows_join<NORM>(sum, top, wr);
    const RowScale s = row_scale(top);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int c = c0 + i * step;
        if (c < D) *reinterpret_cast<uint2*>(p.X8 + row * p.D + c) = e4m3x8(v[i], s);
    }
    // x_scale last: a sum that takes longer then holds up no registers
    SquareSum all{sum, 0.f};
    if (NORM && (KEEP ? !(sum <= 0x1p120f) : sum_lost(sum, p.eps))) {   // the same for the whole row
        if (!KEEP) {
            const XT* H = R ? reinterpret_cast<const XT*>(p.R2) + row * p.D : X;
            for (int c = c0; c < D; c += step) {
                Raw8<XT> x;
                x.load(H + c, true);
                float h[1][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) h[0][j] = x.at(j);
                kept.add<1>(h);
            }
        }
        kept.join();
        if (!wr) kept.join_block();
        all = kept;
    }
    if (t == 0) p.x_scale[row] = x_scale<NORM>(p, all, top);
}

// Rows too long for that: read twice, R' written in the second pass, when the thread that writes an
// element has read its X and R.
template <typename XT, typename WT, bool NORM>
__global__ void __launch_bounds__(1024, 2) rows_e4m3_long_kernel(const RowsArgs p) {
    const long long row = blockIdx.x;
    const XT* X = reinterpret_cast<const XT*>(p.X) + row * p.D;
    const XT* R = p.R ? reinterpret_cast<const XT*>(p.R) + row * p.D : nullptr;
    const WT* W = reinterpret_cast<const WT*>(p.w);
    const int D = (int)p.D, step = 8 * (int)blockDim.x;
    float sum = 0.f;
    uint32_t top = 0;
    float h[1][8], w[8];
    auto load8 = [](const auto* q, float (&to)[8]) {
        Raw8<std::remove_cv_t<std::remove_pointer_t<decltype(q)>>> raw;
        raw.load(q, true);
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i] = raw.at(i);
    };
    auto read = [&](int c) {
        load8(X + c, h[0]);
        if (R) {
            load8(R + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[0][i] += w[i];
        }
    };
    for (int c = 8 * (int)threadIdx.x; c < D; c += step) {
        read(c);
        if (NORM) load8(W + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (NORM) sum = fmaf(h[0][i], h[0][i], sum);
            top = max(top, __float_as_uint(NORM ? h[0][i] * w[i] : h[0][i]) & 0x7FFFFFFFu);
        }
    }
    rows_join<NORM>(sum, top, false);
    const bool lost = NORM && sum_lost(sum, p.eps);   // summed again in the second pass
    SquareSum all{lost ? 0.f : sum, 0.f};
    const RowScale s = row_scale(top);
    for (int c = 8 * (int)threadIdx.x; c < D; c += step) {
        read(c);
        if (lost) all.add<1>(h);
        if (R) store8(reinterpret_cast<XT*>(p.R2) + row * p.D + c, h[0]);
        if (NORM) {
            load8(W + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[0][i] *= w[i];
        }
        *reinterpret_cast<uint2*>(p.X8 + row * p.D + c) = e4m3x8(h[0], s);
    }
    if (lost) {
        all.join();
        all.join_block();
    }
    if (threadIdx.x == 0) p.x_scale[row] = x_scale<NORM>(p, all, top);
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
    // eight for long rows without R, whose registers they leave enough of (4096 x 11008 bf16: 24 us, with four
    // 28 us; 8191 x 16384 fp32 norm: 122 and 163 us).  With R they do not (2048 x 11008: 39 us, with four 30 us).
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
    constexpr bool KEEP = NORM && sizeof(XT) == 2;
    dim3 block(threads);
    switch (vec) {
        case 1: return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 1, KEEP, NORM>, grid, block, 0, st, p);
        case 2: return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 2, KEEP, NORM>, grid, block, 0, st, p);
        case 4: return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 4, KEEP, NORM>, grid, block, 0, st, p);
        default:
            if (NORM && p.R) return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 8, NORM, NORM>, grid, block, 0, st, p);
            return launch_plain(gq::rows_e4m3_kernel<XT, WT, NORM, 8, false, false>, grid, block, 0, st, p);
    }
}

}  // namespace gqh
