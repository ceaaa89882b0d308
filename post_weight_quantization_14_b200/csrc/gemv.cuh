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
    unsigned split;           // CTAs of a cluster, which split K
    int vec;                  // N % 4 == 0: 16-byte loads of packed words
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


// ---------------------------------------------------------------------------- tensor instruction
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, __nv_bfloat16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, __nv_fp8_e4m3) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t bits_of(const T& v) {
    static_assert(sizeof(T) == 4, "a pair of 16-bit values");
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }
__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }

// The eight columns k .. k + 7 of one token as the pairs (i, i + 4), i = 0 .. 3.
__device__ __forceinline__ void x_pairs(const __nv_bfloat16* x, uint32_t (&b)[4]) {
    const uint4 u = *reinterpret_cast<const uint4*>(x);
    b[0] = __byte_perm(u.x, u.z, 0x5410);
    b[1] = __byte_perm(u.x, u.z, 0x7632);
    b[2] = __byte_perm(u.y, u.w, 0x5410);
    b[3] = __byte_perm(u.y, u.w, 0x7632);
}
__device__ __forceinline__ void x_pairs(const __nv_fp8_e4m3* x, uint32_t (&b)[4]) {   // e4m3 is exact in fp16
    const uint2 u = *reinterpret_cast<const uint2*>(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = __byte_perm(u.x, u.y, i | ((i + 4) << 4));   // bytes i and i + 4
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
        b[i] = bits_of(h);
    }
}

// The four columns k .. k + 3 of one token as the pairs (0, 2) and (1, 3).
__device__ __forceinline__ void x_quad(const __nv_bfloat16* x, uint32_t& b0, uint32_t& b1) {
    const uint2 u = *reinterpret_cast<const uint2*>(x);
    b0 = __byte_perm(u.x, u.y, 0x5410);
    b1 = __byte_perm(u.x, u.y, 0x7632);
}
__device__ __forceinline__ void x_quad(const __nv_fp8_e4m3* x, uint32_t& b0, uint32_t& b1) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(x);
    b0 = bits_of(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(__byte_perm(u, 0, 0x4420) & 0xFFFFu), __NV_E4M3));
    b1 = bits_of(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(__byte_perm(u, 0, 0x4431) & 0xFFFFu), __NV_E4M3));
}

// q - z of one row's columns in pairs.  For up to 4 bits ``w`` holds the codes as nibbles and pair i is
// those at bits 4 i and 16 + 4 i; for 8 bits pair i is byte i of w and byte i of w2.  zz holds the zero
// point as zero_pair makes it.
template <int BITS, int NP>
__device__ __forceinline__ void w_pairs(uint32_t w, uint32_t w2, uint32_t zz, uint32_t (&v)[NP], __nv_bfloat16) {
    if constexpr (BITS <= 4) {   // 0x4300 | q is the bf16 of 128 + q
#pragma unroll
        for (int i = 0; i < NP; ++i)
            v[i] = bits_of(__hsub2(as_bf162(((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u), as_bf162(zz)));
    } else {                     // both nibbles this way, then 16 high + (low - z): 8 significant bits
        const __nv_bfloat162 c128 = as_bf162(0x43004300u), c16 = as_bf162(0x41804180u);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint32_t two = __byte_perm(w, w2, i | ((i + 4) << 8));   // bytes i in the two halves
            const __nv_bfloat162 lo = __hsub2(as_bf162((two & 0x000F000Fu) | 0x43004300u), c128);
            const __nv_bfloat162 hi = __hsub2(as_bf162(((two >> 4) & 0x000F000Fu) | 0x43004300u), c128);
            v[i] = bits_of(__hfma2(hi, c16, __hsub2(lo, as_bf162(zz))));
        }
    }
}
template <int BITS, int NP>
__device__ __forceinline__ void w_pairs(uint32_t w, uint32_t w2, uint32_t zz, uint32_t (&v)[NP], __nv_fp8_e4m3) {
    if constexpr (BITS <= 4) {   // 0x6400 | q is the fp16 of 1024 + q, 0x6400 | 16 q of 1024 + 16 q
        const __half2 c16 = as_half2(0x2C002C00u);   // 1 / 16
        const __half2 za = as_half2(zz);             // 1024 + z
        const __half2 zb = __hsub2(as_half2(0x63806380u), za);   // 960 - (1024 + z) = -(64 + z)
#pragma unroll
        for (int i = 0; i < NP; i += 2) {
            const uint32_t x = w >> (4 * i);
            v[i] = bits_of(__hsub2(as_half2((x & 0x000F000Fu) | 0x64006400u), za));
            v[i + 1] = bits_of(__hfma2(as_half2((x & 0x00F000F0u) | 0x64006400u), c16, zb));
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint32_t two = __byte_perm(w, w2, i | ((i + 4) << 8));
            v[i] = bits_of(__hsub2(as_half2((two & 0x00FF00FFu) | 0x64006400u), as_half2(zz)));
        }
    }
}
// A thread's eight codes of a step of 32 columns (8 tig .. 8 tig + 7) as nibbles, from the one or two
// words that hold them; 8-bit codes stay as they are.
template <int BITS>
__device__ __forceinline__ uint32_t chunk_nibbles(uint32_t w, uint32_t w2, int tig) {
    if constexpr (BITS == 2) return codes_to_nibbles<2>((w >> (16 * (tig & 1))) & 0xFFFFu);
    if constexpr (BITS == 3) return codes_to_nibbles<3>(__funnelshift_r(w, w2, (24 * tig) & 31) & 0xFFFFFFu);
    return w;
}
// Four codes that start at bit ``sh`` of w, arranged for the pairs (0, 2) and (1, 3).
template <int BITS>
__device__ __forceinline__ void quad_nibbles(uint32_t w, uint32_t w2, int sh, uint32_t& a, uint32_t& b) {
    if constexpr (BITS == 8) {   // bytes 0, 1 against bytes 2, 3
        a = w;
        b = w >> 16;
    } else {
        const uint32_t v = __funnelshift_r(w, w2, sh) & ((1u << (4 * BITS)) - 1u);
        const uint32_t h = BITS == 4 ? v : codes_to_nibbles<BITS>(v);
        a = (h & 0xFFu) | ((h & 0xFF00u) << 8);
        b = 0;
    }
}
template <int BITS>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z, __nv_bfloat16) {
    const float f = (BITS <= 4 ? 128.f : 0.f) + (float)z;
    return bits_of(__floats2bfloat162_rn(f, f));
}
template <int BITS>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z, __nv_fp8_e4m3) {
    return ((0x6400u | z) << 16) | 0x6400u | z;
}

constexpr int GM_WARPS = 8;        // warps of a CTA, all on the same rows n
constexpr int GM_UNIT = 128;       // columns of a unit: four steps of 32

template <int BITS, typename XT, int MT, int NT, bool G16>
__global__ void __launch_bounds__(32 * GM_WARPS, 2) gemv_mma_kernel(const GemvArgs p) {
    constexpr int ROWS = 32 * NT, TOK = 8 * MT, TILES = 2 * NT;
    constexpr int WPC = G16 ? (BITS == 3 ? 4 : 2) : BITS == 8 || BITS == 3 ? 2 : 1;   // words that hold a thread's eight codes
    __shared__ float red[GM_WARPS][TOK][ROWS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const unsigned cta = blockIdx.x / p.split, rank = blockIdx.x % p.split;
    const long long n0 = (long long)(cta % p.nblocks) * ROWS + 4 * gid;   // n0 + 32 i + 0 .. 3, i < NT
    const int m0 = (int)(cta / p.nblocks) * TOK;
    const int K = (int)p.K;
    const long long zwords = (p.N * BITS + 31) / 32;
    const XT* X = reinterpret_cast<const XT*>(p.X);

    const int units = (K + GM_UNIT - 1) / GM_UNIT;
    const int slot = (int)rank * GM_WARPS + warp, slots = (int)p.split * GM_WARPS;
    const int u0 = (int)((long long)units * slot / slots), u1 = (int)((long long)units * (slot + 1) / slots);

    float total[TILES][MT][4] = {}, part[TILES][MT][4] = {};
    float sc[4 * NT];
    uint32_t zz[4 * NT];
    // Row ``r`` of the packed words, the thread's 4 NT rows n.
    auto load_row = [&](long long r, bool valid, uint32_t (&w)[4 * NT]) {
        const int32_t* src = p.qweight + r * p.N;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const long long n = n0 + 32 * i;
            if (p.vec) {
                const uint4 u = valid && n < p.N ? __ldg(reinterpret_cast<const uint4*>(src + n)) : make_uint4(0, 0, 0, 0);
                w[4 * i] = u.x;
                w[4 * i + 1] = u.y;
                w[4 * i + 2] = u.z;
                w[4 * i + 3] = u.w;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) w[4 * i + c] = valid && n + c < p.N ? (uint32_t)__ldg(src + n + c) : 0u;
            }
        }
    };
    auto load_group = [&](long long gi) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const long long n = n0 + 32 * i;
            if (p.vec) {
                const uint2 u = n < p.N ? __ldg(reinterpret_cast<const uint2*>(p.scales + gi * p.N + n)) : make_uint2(0, 0);
                const float2 a = __half22float2(as_half2(u.x)), b = __half22float2(as_half2(u.y));
                sc[4 * i] = a.x;
                sc[4 * i + 1] = a.y;
                sc[4 * i + 2] = b.x;
                sc[4 * i + 3] = b.y;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    sc[4 * i + c] = n + c < p.N ? __half2float(p.scales[gi * p.N + n + c]) : 0.f;
            }
            uint32_t z4 = 0;   // four zero points; n is a multiple of 4, so only 3-bit ones straddle words
            if (p.qzeros != nullptr && n < p.N) {
                const uint32_t* zp = reinterpret_cast<const uint32_t*>(p.qzeros) + gi * zwords;
                const long long bit = n * BITS, k = bit >> 5;
                z4 = __ldg(zp + k) >> (bit & 31);
                if (BITS == 3 && (bit & 31) > 20 && k + 1 < zwords) z4 |= __ldg(zp + k + 1) << (32 - (bit & 31));
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t z = p.qzeros != nullptr ? (z4 >> (BITS * c)) & ((1u << BITS) - 1u) : 1u << (BITS - 1);
                zz[4 * i + c] = zero_pair<BITS>(z, XT());
            }
        }
    };
    auto flush = [&] {   // the group's sums, scaled
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
            const int lo = j, hi = NT == 2 ? 4 + j : j + 2;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                total[j][mt][0] = fmaf(sc[lo], part[j][mt][0], total[j][mt][0]);
                total[j][mt][1] = fmaf(sc[lo], part[j][mt][1], total[j][mt][1]);
                total[j][mt][2] = fmaf(sc[hi], part[j][mt][2], total[j][mt][2]);
                total[j][mt][3] = fmaf(sc[hi], part[j][mt][3], total[j][mt][3]);
#pragma unroll
                for (int c = 0; c < 4; ++c) part[j][mt][c] = 0.f;
            }
        }
    };

    for (int u = u0; u < u1; ++u) {
        uint32_t raw[4][WPC][4 * NT];
#pragma unroll
        for (int st = 0; st < 4; ++st) {   // all of the unit's words first: their latencies overlap
            const int k = u * GM_UNIT + 32 * st;
            if constexpr (G16) {           // four codes of each half of the step
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int kh = k + 16 * h + 4 * tig, sh = kh * BITS & 31;
                    const long long r = (long long)kh * BITS / 32;
                    load_row(r, kh < K, raw[st][h]);
                    if constexpr (BITS == 3) load_row(r + 1, kh < K && sh > 20, raw[st][2 + h]);
                }
            } else {
                const int kc = k + 8 * tig;
                const long long r = (long long)kc * BITS / 32;
                load_row(r, kc < K, raw[st][0]);
                if constexpr (BITS == 8) load_row(r + 1, kc < K, raw[st][1]);
                // codes of 24 bits that start past bit 8 of a word end in the next
                if constexpr (BITS == 3) load_row(r + 1, kc < K && tig != 0 && tig != 3, raw[st][1]);
            }
        }
#pragma unroll
        for (int st = 0; st < 4; ++st) {
            const int k = u * GM_UNIT + 32 * st;
            if (k >= K) break;
            if (!G16 && (k % p.g == 0 || (st == 0 && u == u0))) load_group(k / p.g);
            uint32_t xb[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int m = m0 + 8 * mt + gid;
                xb[mt][0] = xb[mt][1] = xb[mt][2] = xb[mt][3] = 0u;
                if constexpr (G16) {
                    // columns k + 4 tig + 0 .. 3 and k + 16 + 4 tig + 0 .. 3
                    if (m < p.M && k + 4 * tig < K) x_quad(X + (long long)m * K + k + 4 * tig, xb[mt][0], xb[mt][1]);
                    if (m < p.M && k + 16 + 4 * tig < K)
                        x_quad(X + (long long)m * K + k + 16 + 4 * tig, xb[mt][2], xb[mt][3]);
                } else {
                    if (m < p.M && k + 8 * tig < K) x_pairs(X + (long long)m * K + k + 8 * tig, xb[mt]);
                }
            }
#pragma unroll
            for (int h = 0; h < (G16 ? 2 : 1); ++h) {
                if constexpr (G16) {
                    if (k + 16 * h >= K) break;
                    load_group((k + 16 * h) / p.g);
                }
#pragma unroll
                for (int j = 0; j < TILES; ++j) {
                    const int lo = j, hi = NT == 2 ? 4 + j : j + 2;
                    constexpr int NP = G16 ? 2 : 4;
                    uint32_t a[NP], b[NP];   // rows gid and gid + 8 of the tile
                    if constexpr (G16) {
                        const int sh = (k + 16 * h + 4 * tig) * BITS & 31;
                        uint32_t c, d;
                        quad_nibbles<BITS>(raw[st][h][lo], raw[st][WPC - 2 + h][lo], sh, c, d);
                        w_pairs<BITS, NP>(c, d, zz[lo], a, XT());
                        quad_nibbles<BITS>(raw[st][h][hi], raw[st][WPC - 2 + h][hi], sh, c, d);
                        w_pairs<BITS, NP>(c, d, zz[hi], b, XT());
                    } else {
                        const uint32_t l2 = raw[st][WPC - 1][lo], h2 = raw[st][WPC - 1][hi];
                        w_pairs<BITS, NP>(chunk_nibbles<BITS>(raw[st][0][lo], l2, tig), l2, zz[lo], a, XT());
                        w_pairs<BITS, NP>(chunk_nibbles<BITS>(raw[st][0][hi], h2, tig), h2, zz[hi], b, XT());
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_16816(part[j][mt], a[0], b[0], a[1], b[1], xb[mt][2 * h], xb[mt][2 * h + 1], XT());
                        if constexpr (!G16)
                            mma_16816(part[j][mt], a[2], b[2], a[3], b[3], xb[mt][2], xb[mt][3], XT());
                    }
                }
                if (G16) flush();
            }
            if (!G16 && ((k + 32) % p.g == 0 || k + 32 >= K || (st == 3 && u == u1 - 1))) flush();
        }
    }

    // join the warps' sums, then those of the cluster's CTAs, in a fixed order
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
        const int lo = 4 * gid + j, hi = NT == 2 ? 32 + 4 * gid + j : 4 * gid + j + 2;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int t = 8 * mt + 2 * tig;
            red[warp][t][lo] = total[j][mt][0];
            red[warp][t + 1][lo] = total[j][mt][1];
            red[warp][t][hi] = total[j][mt][2];
            red[warp][t + 1][hi] = total[j][mt][3];
        }
    }
    __syncthreads();
    const long long nc = (long long)(cta % p.nblocks) * ROWS;
    auto finish = [&](int e, float y) {
        const int m = m0 + e / ROWS;
        const long long n = nc + e % ROWS;
        if (m < p.M && n < p.N) store_y(p.Y, p.y_bf16, (long long)m * p.N + n, p.x_scale ? y * p.x_scale[m] : y);
    };
    for (int e = threadIdx.x; e < TOK * ROWS; e += 32 * GM_WARPS) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < GM_WARPS; ++w) y += (&red[w][0][0])[e];
        if (p.split == 1)
            finish(e, y);
        else
            (&red[0][0][0])[e] = y;   // read above by this thread alone
    }
    if (p.split > 1) {
        __syncwarp();
        cluster_sync_all();
        for (int e = (int)rank * (32 * GM_WARPS) + threadIdx.x; e < TOK * ROWS; e += (int)p.split * (32 * GM_WARPS)) {
            float y = 0.f;
            for (unsigned r = 0; r < p.split; ++r) y += ld_cluster_f32(smem_u32(&red[0][0][0] + e), r);
            finish(e, y);
        }
        __syncwarp();
        cluster_sync_all();   // no CTA leaves while its sums are being read
    }
}

}  // namespace gq

namespace gqh {

int num_sms();

template <int BITS, typename XT, int MT, int NT, bool G16>
cudaError_t gemv_mma_launch(gq::GemvArgs p, cudaStream_t st) {
    constexpr int ROWS = 32 * NT, TOK = 8 * MT;
    p.nblocks = (unsigned)((p.N + ROWS - 1) / ROWS);
    p.vec = p.N % 4 == 0;
    const long long blocks = (long long)p.nblocks * ((p.M + TOK - 1) / TOK);
    // K is split until two CTAs per SM have work, with a unit at least for each warp
    p.split = 1;
    while (p.split < 8 && blocks * p.split < 2 * num_sms() && p.K > (long long)gq::GM_UNIT * gq::GM_WARPS * p.split)
        p.split *= 2;
    if (blocks * p.split > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * p.split));
    cfg.blockDim = dim3(32 * gq::GM_WARPS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gq::gemv_mma_kernel<BITS, XT, MT, NT, G16>, p);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

template <int BITS, typename XT>
cudaError_t gemv_mma_run(const gq::GemvArgs& p, cudaStream_t st) {
    if (p.g == 16) return gemv_mma_launch<BITS, XT, 2, 1, true>(p, st);
    if (p.M <= 8) return gemv_mma_launch<BITS, XT, 1, 2, false>(p, st);
    if (p.M <= 16) return gemv_mma_launch<BITS, XT, 2, 1, false>(p, st);
    return gemv_mma_launch<BITS, XT, 4, 1, false>(p, st);
}

template <typename XT>
cudaError_t gemv_run_x(gq::GemvArgs p, cudaStream_t st) {
    TimedScope ts__("dequant_gemv", st);
    if (!p.g_idx) {
        switch (p.bits) {
            case 2: return gemv_mma_run<2, XT>(p, st);
            case 3: return gemv_mma_run<3, XT>(p, st);
            case 4: return gemv_mma_run<4, XT>(p, st);
            default: return gemv_mma_run<8, XT>(p, st);
        }
    }
    p.nblocks = (unsigned)((p.N + 31) / 32);
    const long long blocks = (long long)p.nblocks * ((p.M + gq::GV_TOK - 1) / gq::GV_TOK);
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    return launch_plain(gq::gemv_lane_kernel<XT>, dim3((unsigned)blocks), dim3(32 * gq::GV_WARPS), 0, st, p);
}

inline cudaError_t gemv_run(const gq::GemvArgs& p, bool x_e4m3, cudaStream_t st) {
    return x_e4m3 ? gemv_run_x<__nv_fp8_e4m3>(p, st) : gemv_run_x<__nv_bfloat16>(p, st);
}

}  // namespace gqh
