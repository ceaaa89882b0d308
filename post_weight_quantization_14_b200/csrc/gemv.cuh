// Products of a few tokens with packed weights (decoding):
//
//   Y[m, n] = xs[m] sum_k X[m, k] W_hat[n, k],   W_hat[n, k] = s[g(k), n] (q[n, k] - z[g(k), n])
//
// with g(k) = k / g, or g_idx[k] for layers quantized in activation order.  X is bf16 (xs = 1)
// or e4m3 with one fp32 scale per row.
//
// Two kernels:
//
// gemv_mma_kernel (groups of consecutive columns).  The work is one pass over the packed words, so
// the design is about issue slots next to the loads: with fp32 FMAs every weight costs an unpack, a
// subtraction and M multiplies, with the warp-level tensor instruction (16 x 8 x 16, fp32 sums) the same
// for any M up to 8.  (tcgen05 would need the unpacked weights in shared or tensor
// memory first; here they stay in the registers that unpacked them.)  K order inside one instruction
// is free as long as both operands agree, which makes the packed layout fit without any shuffle: a
// thread's word of 8 codes (row n, columns k .. k + 7) is four pairs (i, i + 4) that mask out of the
// word side by side, and its 16 bytes of X (token, k .. k + 7) are the matching pairs.  Codes become
// numbers by the published exponent-bias method: placed in the low fraction bits of a bf16 or fp16 power of
// two they are that power plus the code, and one subtraction takes it and z away.  q - z is exact
// in bf16 and fp16, P = X (q - z)^T is summed over a group (128 columns at most, as the tensor instruction
// may cut its sums off) and enters y as s P in fp32.
// A CTA owns 128 rows n and a run of columns.  One warp fills a ring of stages of 256 columns with TMA
// (or bulk copies of rows), which keeps some 100 KB in flight on an SM and costs the others no issue
// slots; four warps take 32 rows each of a stage's first 128 columns, four of the others.  The halves'
// sums, and those of the CTAs of a cluster that split K, are joined in a fixed order through shared
// memory.
//
// Measured, all inputs from memory: 4-bit groups of 128, one token through 4096 x 4096 8.6 us (8.9 MB,
// 1.0 TB/s: of that about 4.6 us are launch, first loads and the join), through 11008 x 4096 15.6 us; eight
// e4m3 tokens through 50001 x 8192 (odd row count: bulk copies of rows) 102 us (214 MB, 2.1 TB/s); 16
// tokens through 11008 x 4096, 3 bits, groups of 64, 32 us.  The copies alone would take a third of
// that.  By the counters of the 50001 x 8192 product 65 % of the issue slots are used, 5.1 instructions a
// weight, of which unpacking, subtracting and multiplying are about 2; the rest (rows that start between
// 16-byte boundaries, X widened by each of the warps, polling, a flush per group) is not separated.
//
// gemv_act_kernel (g_idx: any column in any group): see there.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "dqgemm_e4m3.cuh"
#include "pack.cuh"

namespace gq {

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
    int g_all;                // one group per row (g = K)
    int bits;
    unsigned nblocks;         // blocks of rows n
    unsigned split;           // CTAs of a cluster, which split K
    int vec;                  // N % 4 == 0: 16-byte loads of packed words
    int tma;                  // words and X by TMA
    int gshift;               // log2 g, or 31 for one group per row
};

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
// (a & mask) | c as one instruction: with both constants as immediates the compiler takes two.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(c));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t bits_of(const T& v) {
    static_assert(sizeof(T) == 4, "a pair of 16-bit values");
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }
__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }

// A thread's eight columns of a step of one token, as loaded: k .. k + 7, or (two runs of four, groups
// of 16) lo .. lo + 3 and hi .. hi + 3.
template <typename XT>
struct XRaw;
template <>
struct XRaw<__nv_bfloat16> {
    uint4 u;
};
template <>
struct XRaw<__nv_fp8_e4m3> {
    uint2 u;
};
__device__ __forceinline__ XRaw<__nv_bfloat16> load_x8(const __nv_bfloat16* x) {
    return {*reinterpret_cast<const uint4*>(x)};
}
__device__ __forceinline__ XRaw<__nv_fp8_e4m3> load_x8(const __nv_fp8_e4m3* x) {
    return {*reinterpret_cast<const uint2*>(x)};
}
__device__ __forceinline__ XRaw<__nv_bfloat16> load_x44(const __nv_bfloat16* lo, const __nv_bfloat16* hi) {
    const uint2 a = *reinterpret_cast<const uint2*>(lo), b = *reinterpret_cast<const uint2*>(hi);
    return {make_uint4(a.x, a.y, b.x, b.y)};
}
__device__ __forceinline__ XRaw<__nv_fp8_e4m3> load_x44(const __nv_fp8_e4m3* lo, const __nv_fp8_e4m3* hi) {
    return {make_uint2(*reinterpret_cast<const uint32_t*>(lo), *reinterpret_cast<const uint32_t*>(hi))};
}
__device__ __forceinline__ void x_floats(const XRaw<__nv_bfloat16>& r, float (&x)[8]) {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void x_floats(const XRaw<__nv_fp8_e4m3>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = (i < 2 ? r.u.x : r.u.y) >> (16 * (i & 1));
        const float2 f = __half22float2(
            __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3)));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
// The columns in pairs: (i, i + 4), i = 0 .. 3; or (0, 2), (1, 3) of the first four and of the second.
template <bool G16>
__device__ __forceinline__ void x_pairs(const XRaw<__nv_bfloat16>& r, uint32_t (&b)[4]) {
    const uint32_t y = G16 ? r.u.y : r.u.z, z = G16 ? r.u.z : r.u.y;
    b[0] = __byte_perm(r.u.x, y, 0x5410);
    b[1] = __byte_perm(r.u.x, y, 0x7632);
    b[2] = __byte_perm(z, r.u.w, 0x5410);
    b[3] = __byte_perm(z, r.u.w, 0x7632);
}
template <bool G16>
__device__ __forceinline__ void x_pairs(const XRaw<__nv_fp8_e4m3>& r, uint32_t (&b)[4]) {   // exact in fp16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = G16 ? __byte_perm(i < 2 ? r.u.x : r.u.y, 0, (i & 1) ? 0x4431 : 0x4420)
                                 : __byte_perm(r.u.x, r.u.y, i | ((i + 4) << 4));
        b[i] = bits_of(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3));
    }
}

// q - z of one row's columns in pairs.  For up to 4 bits ``w`` holds the codes as nibbles and pair i is
// those at bits 4 i and 16 + 4 i; for 8 bits pair i is byte i of w and byte i of w2.  zz holds the zero
// point as zero_pair makes it.
template <int BITS, int NP>
__device__ __forceinline__ void w_pairs(uint32_t w, uint32_t w2, uint32_t zz, uint32_t (&v)[NP], __nv_bfloat16) {
    if constexpr (BITS <= 4) {   // 0x4300 | q is the bf16 of 128 + q
#pragma unroll
        for (int i = 0; i < NP; ++i)
            v[i] = bits_of(__hsub2(as_bf162(and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u)), as_bf162(zz)));
    } else {                     // both nibbles this way, then 16 high + (low - z): 8 significant bits
        const __nv_bfloat162 c128 = as_bf162(0x43004300u), c16 = as_bf162(0x41804180u);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint32_t two = __byte_perm(w, w2, i | ((i + 4) << 8));   // bytes i in the two halves
            const __nv_bfloat162 lo = __hsub2(as_bf162(and_or(two, 0x000F000Fu, 0x43004300u)), c128);
            const __nv_bfloat162 hi = __hsub2(as_bf162(and_or(two >> 4, 0x000F000Fu, 0x43004300u)), c128);
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
            v[i] = bits_of(__hsub2(as_half2(and_or(x, 0x000F000Fu, 0x64006400u)), za));
            v[i + 1] = bits_of(__hfma2(as_half2(and_or(x, 0x00F000F0u, 0x64006400u)), c16, zb));
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint32_t two = __byte_perm(w, w2, i | ((i + 4) << 8));
            v[i] = bits_of(__hsub2(as_half2(and_or(two, 0x00FF00FFu, 0x64006400u)), as_half2(zz)));
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
    if constexpr (BITS <= 4) return z * 0x00010001u | 0x43004300u;   // 128 + z, twice
    return bits_of(__floats2bfloat162_rn((float)z, (float)z));
}
template <int BITS>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z, __nv_fp8_e4m3) {
    return z * 0x00010001u | 0x64006400u;   // 1024 + z, twice
}

constexpr int GM_WARPS = 8;        // four of 32 rows n each, times two runs of columns
constexpr int GM_THREADS = 32 * GM_WARPS + 32;   // and one that fills the ring
constexpr int GM_ROWS = 128;       // rows n of a CTA
constexpr int GM_K = 256;          // columns of a stage, 128 for each half of the warps
// bytes of a row of words: 16-byte reads without bank conflicts, room to skew
constexpr int GM_WSTRIDE = 4 * GM_ROWS + 32;

template <int BITS, typename XT, int MT, int GROUPS>
struct GmCfg {
    // CTAs of an SM, as registers go: 3 against 2 for up to eight tokens took the 50001 x 8192 product
    // above from 123 to 101 us.  Two token tiles with groups of 32 or 64 do not fit the 96 registers of two
    // CTAs: 16 tokens through 11008 x 4096, groups of 64, take 32 us with one and 36 us with two (3 bits),
    // 28 and 31 us (4 bits); only 2 bits with e4m3 tokens go the other way (32 and 28 us).
    static constexpr int CTAS = MT == 4 || GROUPS == 8 || (MT == 2 && GROUPS == 4) ? 1 : MT == 1 && GROUPS == 1 && BITS <= 4 ? 3 : 2;
    static constexpr int TOK = 8 * MT;
    static constexpr int WROWS = GM_K * BITS / 32;
    static constexpr int W_BOX = WROWS * 128;   // 32 rows n by TMA
    static constexpr int W_BYTES = WROWS * GM_WSTRIDE;
    // the reads of eight (16-byte) or sixteen (8-byte) lanes fall into different banks
    static constexpr int XSTRIDE = GM_K * (int)sizeof(XT) + (sizeof(XT) == 2 ? 64 : 32);
    static constexpr int STAGE = (W_BYTES + TOK * XSTRIDE + 1023) / 1024 * 1024;   // TMA's swizzle
    static constexpr int FIT = 220 / CTAS * 1024 / STAGE;
    static constexpr int STAGES = FIT > 4 ? 4 : FIT < 2 ? 2 : FIT;
    static constexpr int SUMS = 2 * TOK * GM_ROWS * 4;
    static constexpr int SMEM = 1024 + (STAGES * STAGE > SUMS ? STAGES * STAGE : SUMS);
    static_assert(W_BYTES % 128 == 0, "TMA's destination");
};

// GROUPS: those of 128 columns, at most: 1 (groups of 128, or one per row), 4 (64 and 32) or 8 (16).
template <int BITS, typename XT, int MT, int GROUPS>
__global__ void __launch_bounds__(GM_THREADS, GmCfg<BITS, XT, MT, GROUPS>::CTAS)
    gemv_mma_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const GemvArgs p) {
    using Cfg = GmCfg<BITS, XT, MT, GROUPS>;
    constexpr int TOK = Cfg::TOK, STAGES = Cfg::STAGES;
    constexpr bool G16 = GROUPS == 8;
    extern __shared__ uint8_t gm_raw[];
    uint8_t* gm_smem = gm_raw + (-smem_u32(gm_raw) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
    const int nw = warp & 3, kg = warp >> 2 & 1;
    const unsigned cta = blockIdx.x / p.split, rank = blockIdx.x % p.split;
    const long long nc = (long long)(cta % p.nblocks) * GM_ROWS;   // the CTA's first row
    const int m0 = (int)(cta / p.nblocks) * TOK;
    const int K = (int)p.K;
    const XT* X = reinterpret_cast<const XT*>(p.X);
    const int nst = (K + GM_K - 1) / GM_K;
    const int st0 = (int)((long long)nst * rank / p.split), st1 = (int)((long long)nst * (rank + 1) / p.split);

    __shared__ uint64_t full[STAGES], empty[STAGES];   // a lane of the copying warp each; a warp of the others each
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], p.tma ? 1 : 32);
            mbar_init(&empty[i], GM_WARPS);
        }
        fence_mbar_init();
    }
    __syncthreads();

    // Without TMA (N no multiple of 4, or e4m3 rows that are no multiple of 16 bytes) rows that start
    // between two 16-byte boundaries are copied from the boundary on, and the reader skips the 'skew'.
    const int nmod = (int)p.N & 3;
    if (warp == GM_WARPS) {
        // ---- copies into the ring
        if (p.tma && lane == 0) {
            prefetch_tmap(&mW);
            prefetch_tmap(&mX);
        }
        const long long wtotal = ((long long)K * BITS + 31) / 32 * p.N, xtotal = (long long)p.M * K;
        const int wrows = (int)(((long long)K * BITS + 31) / 32), cols = (int)min((long long)GM_ROWS, p.N - nc);
        bool ok = true;
        int st = st0;
        for (; st < st1 && ok; ++st) {
            const int slot = (st - st0) % STAGES;
            ok = __all_sync(~0u, mbar_wait(&empty[slot], (((st - st0) / STAGES) & 1) ^ 1, st));
            if (!ok) break;
            uint8_t* base = gm_smem + slot * Cfg::STAGE;
            if (p.tma) {   // four boxes of 32 rows n and one of X; what lies outside the arrays comes as zeros
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[slot], Cfg::W_BOX * 4 + TOK * GM_K * (int)sizeof(XT));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tma_load_2d(base + i * Cfg::W_BOX, &mW, &full[slot], (int)nc + 32 * i, st * Cfg::WROWS);
                    tma_load_2d(base + Cfg::W_BYTES, &mX, &full[slot], st * GM_K, m0);
                }
                continue;
            }
            // Otherwise a lane copies whole rows in pieces of 16 bytes, as far as the array goes, and the up
            // to three words behind the last piece singly.
            constexpr int WR = (Cfg::WROWS + 31) / 32, XE = 16 / (int)sizeof(XT), XR = (TOK + 31) / 32;
            long long wat[WR], xat[XR];
            int wn[WR], xn[XR];
            uint32_t bytes = 0;
#pragma unroll
            for (int i = 0; i < WR; ++i) {
                const int r = lane + 32 * i, row = st * Cfg::WROWS + r;
                wn[i] = 0;
                if (r < Cfg::WROWS && row < wrows) {
                    const int skew = r * nmod & 3, need = cols + skew;
                    wat[i] = (long long)row * p.N + nc - skew;
                    wn[i] = (int)min((long long)((need + 3) & ~3), (wtotal - wat[i]) & ~3ll);
                    for (int j = wn[i]; j < need; ++j)
                        reinterpret_cast<int32_t*>(base + r * GM_WSTRIDE)[j] = p.qweight[wat[i] + j];
                    bytes += 4 * wn[i];
                }
            }
#pragma unroll
            for (int i = 0; i < XR; ++i) {
                const int r = lane + 32 * i;
                xn[i] = 0;
                if (r < TOK && m0 + r < p.M) {
                    xat[i] = (long long)(m0 + r) * K + st * GM_K;
                    const int skew = (int)(xat[i] % XE), need = min(GM_K, K - st * GM_K) + skew;
                    xat[i] -= skew;
                    xn[i] = (int)min((long long)((need + XE - 1) & ~(XE - 1)), (xtotal - xat[i]) & ~(long long)(XE - 1));
                    if (xn[i] < need)   // eight elements of e4m3
                        *reinterpret_cast<uint2*>(base + Cfg::W_BYTES + r * Cfg::XSTRIDE + xn[i] * (int)sizeof(XT)) =
                            *reinterpret_cast<const uint2*>(X + xat[i] + xn[i]);
                    bytes += xn[i] * (int)sizeof(XT);
                }
            }
            mbar_arrive_expect_tx(&full[slot], bytes);
#pragma unroll
            for (int i = 0; i < WR; ++i)
                if (wn[i] > 0) bulk_g2s(base + (lane + 32 * i) * GM_WSTRIDE, p.qweight + wat[i], 4 * wn[i], &full[slot]);
#pragma unroll
            for (int i = 0; i < XR; ++i)
                if (xn[i] > 0)
                    bulk_g2s(base + Cfg::W_BYTES + (lane + 32 * i) * Cfg::XSTRIDE, X + xat[i], xn[i] * (int)sizeof(XT),
                             &full[slot]);
        }
        // after a wait that ran out, the copies still in flight land before the CTA leaves
        for (int i = max(st0, st - STAGES); !ok && i < st; ++i)
            (void)mbar_wait(&full[(i - st0) % STAGES], ((i - st0) / STAGES) & 1, -1);
    }

    // ---- scales and zero points of this thread's rows n0 .. n0 + 3, one stage ahead, as loaded
    const long long n0 = nc + 32 * nw + 4 * gid;
    const long long zwords = (p.N * BITS + 31) / 32;
    const int gmask = (int)((1u << p.gshift) - 1u);   // one group per row: no column but the first begins one
    uint2 s_raw[GROUPS], s_next[GROUPS] = {};
    constexpr int ZW = BITS == 3 ? 2 : 1;   // words that hold four zero points
    uint32_t z_raw[GROUPS][ZW], z_next[GROUPS][ZW] = {};
    auto load_group = [&](int gi, uint2& sr, uint32_t (&zr)[ZW]) {
        const __half* sp = p.scales + (long long)gi * p.N + n0;
        sr = make_uint2(0, 0);
        if (p.vec) {
            if (n0 < p.N) sr = __ldg(reinterpret_cast<const uint2*>(sp));
        } else {
            uint32_t h[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) h[c] = n0 + c < p.N ? __half_as_ushort(sp[c]) : 0u;
            sr = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        }
        // as loaded: the first use of a load waits for it.  n0 is a multiple of 4, so only 3-bit zero
        // points straddle words.
        if (p.qzeros != nullptr && n0 < p.N) {
            const uint32_t* zp = reinterpret_cast<const uint32_t*>(p.qzeros) + gi * zwords + (n0 * BITS >> 5);
            zr[0] = __ldg(zp);
            if constexpr (ZW == 2) zr[ZW - 1] = __ldg(zp + ((n0 * BITS >> 5) + 1 < zwords ? 1 : 0));
        }
    };
    // groups that begin in the 128 columns from k on (or the one that k lies in, at the run's start)
    auto load_groups = [&](int k, bool start) {
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int kk = k + (G16 ? 16 : 32) * i;
            if (kk < K && (G16 || (GROUPS == 1 && p.gshift == 7) || (kk & gmask) == 0 || (i == 0 && start)))
                load_group(kk >> p.gshift, s_next[i], z_next[i]);
        }
    };

    float total[2][MT][4] = {}, part[2][MT][4] = {};   // tile j: rows n0 + j (first 8 of the tile) and n0 + j + 2
    float sc[4] = {};
    uint32_t zz[4] = {};
    const uint32_t zshift = (uint32_t)(n0 * BITS) & 31u;
    auto use_group = [&](const uint2& sr, const uint32_t (&zw)[ZW]) {
        const uint32_t zr = ZW == 2 ? __funnelshift_r(zw[0], zw[ZW - 1], zshift) : zw[0] >> zshift;
        const float2 a = __half22float2(as_half2(sr.x)), b = __half22float2(as_half2(sr.y));
        sc[0] = a.x;
        sc[1] = a.y;
        sc[2] = b.x;
        sc[3] = b.y;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t z = p.qzeros != nullptr ? (zr >> (BITS * c)) & ((1u << BITS) - 1u) : 1u << (BITS - 1);
            zz[c] = zero_pair<BITS>(z, XT());
        }
    };
    auto flush = [&] {   // the group's sums, scaled
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    total[j][mt][c] = fmaf(sc[c < 2 ? j : j + 2], part[j][mt][c], total[j][mt][c]);
                    part[j][mt][c] = 0.f;
                }
    };

    const int last = warp < GM_WARPS ? st1 : st0;   // the copying warp has no share in the sums
    if (st0 < last) load_groups(st0 * GM_K + 128 * kg, true);
    for (int st = st0; st < last; ++st) {
        const int slot = (st - st0) % STAGES;
        if (!__all_sync(~0u, mbar_wait(&full[slot], ((st - st0) / STAGES) & 1, st))) break;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            s_raw[i] = s_next[i];
#pragma unroll
            for (int j = 0; j < ZW; ++j) z_raw[i][j] = z_next[i][j];
        }
        if (st + 1 < last) load_groups(st * GM_K + 128 * kg + GM_K, false);

        const uint8_t* base = gm_smem + slot * Cfg::STAGE;
        const uint8_t* wbase = p.tma ? base + nw * Cfg::W_BOX + kg * (Cfg::W_BOX / 2)
                                     : base + kg * (Cfg::WROWS / 2 * GM_WSTRIDE) + (32 * nw + 4 * gid) * 4;
        const int xstride = p.tma ? GM_K * (int)sizeof(XT) : Cfg::XSTRIDE;
        const uint8_t* xbase = base + Cfg::W_BYTES + gid * xstride + 128 * kg * (int)sizeof(XT);
        // four neighbouring rows n of a row of words; TMA's boxes have 128-byte rows, 16-byte pieces swizzled
        auto row = [&](int r) {
            if (p.tma)
                return *reinterpret_cast<const uint4*>(wbase + r * 128 + ((gid ^ (r + Cfg::WROWS / 2 * kg & 7)) << 4));
            const uint32_t* u = reinterpret_cast<const uint32_t*>(wbase + r * GM_WSTRIDE) + (r * nmod & 3);
            return make_uint4(u[0], u[1], u[2], u[3]);
        };
        const int k0 = st * GM_K + 128 * kg;
#pragma unroll
        for (int s4 = 0; s4 < 4; ++s4) {
            const int k = k0 + 32 * s4;
            if (k >= K) break;
            if constexpr (GROUPS == 1) {
                if (s4 == 0 && (p.gshift == 7 || st == st0)) use_group(s_raw[0], z_raw[0]);
            } else if constexpr (GROUPS == 4) {
                if ((k & gmask) == 0) use_group(s_raw[s4], z_raw[s4]);
            }
            uint32_t xb[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const XT* x = reinterpret_cast<const XT*>(xbase + 8 * mt * xstride) + 32 * s4 +
                              (sizeof(XT) == 1 && !p.tma ? (m0 + gid + 8 * mt) * K & 8 : 0);
                if constexpr (G16)
                    x_pairs<true>(load_x44(x + 4 * tig, x + 16 + 4 * tig), xb[mt]);
                else
                    x_pairs<false>(load_x8(x + 8 * tig), xb[mt]);
                if (k + 32 > K) {   // past the last column the ring holds what was there before
                    const bool lo = k + (G16 ? 4 : 8) * tig < K, hi = G16 ? k + 16 + 4 * tig < K : lo;
                    xb[mt][0] = lo ? xb[mt][0] : 0u;
                    xb[mt][1] = lo ? xb[mt][1] : 0u;
                    xb[mt][2] = hi ? xb[mt][2] : 0u;
                    xb[mt][3] = hi ? xb[mt][3] : 0u;
                }
            }
            if constexpr (!G16) {
                uint4 w = row(s4 * BITS + (BITS == 8 ? 2 * tig : BITS == 4 ? tig : BITS == 2 ? tig >> 1 : 3 * tig >> 2));
                uint4 w2 = w;
                if constexpr (BITS == 8) w2 = row(s4 * BITS + 2 * tig + 1);
                // 24 bits from bit 24 or 16 of a word on end in the next
                if constexpr (BITS == 3) w2 = row(s4 * BITS + min((3 * tig >> 2) + 1, 2));
                const uint32_t a0[4] = {w.x, w.y, w.z, w.w}, a1[4] = {w2.x, w2.y, w2.z, w2.w};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t a[4], b[4];   // rows gid and gid + 8 of the tile
                    w_pairs<BITS, 4>(chunk_nibbles<BITS>(a0[j], a1[j], tig), a1[j], zz[j], a, XT());
                    w_pairs<BITS, 4>(chunk_nibbles<BITS>(a0[j + 2], a1[j + 2], tig), a1[j + 2], zz[j + 2], b, XT());
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_16816(part[j][mt], a[0], b[0], a[1], b[1], xb[mt][0], xb[mt][1], XT());
                        mma_16816(part[j][mt], a[2], b[2], a[3], b[3], xb[mt][2], xb[mt][3], XT());
                    }
                }
                // one group per row as well: the tensor instruction may cut its sums off, always in the same
                // direction, so they are added up in fp32 every 128 columns
                if (GROUPS == 1 ? s4 == 3 || k + 32 >= K : ((k + 32) & gmask) == 0 || k + 32 >= K) flush();
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (k + 16 * h >= K) break;
                    use_group(s_raw[2 * s4 + h], z_raw[2 * s4 + h]);
                    const int bit = (32 * s4 + 16 * h + 4 * tig) * BITS;   // of the four codes, in this run of words
                    const uint4 w = row(bit >> 5);
                    uint4 w2 = w;
                    if constexpr (BITS == 3) w2 = row(min((bit >> 5) + 1, 4 * BITS - 1));
                    const uint32_t a0[4] = {w.x, w.y, w.z, w.w}, a1[4] = {w2.x, w2.y, w2.z, w2.w};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t c, d, a[2], b[2];
                        quad_nibbles<BITS>(a0[j], a1[j], bit & 31, c, d);
                        w_pairs<BITS, 2>(c, d, zz[j], a, XT());
                        quad_nibbles<BITS>(a0[j + 2], a1[j + 2], bit & 31, c, d);
                        w_pairs<BITS, 2>(c, d, zz[j + 2], b, XT());
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            mma_16816(part[j][mt], a[0], b[0], a[1], b[1], xb[mt][2 * h], xb[mt][2 * h + 1], XT());
                    }
                    flush();
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
    }

    // ---- join the two runs of columns, then the CTAs of the cluster, in a fixed order
    __syncthreads();
    float* sums = reinterpret_cast<float*>(gm_smem);   // [2][TOK][GM_ROWS]
    if (warp < GM_WARPS) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    sums[(kg * TOK + 8 * mt + 2 * tig + (c & 1)) * GM_ROWS + 32 * nw + 4 * gid + j + (c & 2)] =
                        total[j][mt][c];
    }
    __syncthreads();
    auto finish = [&](int e, float y) {
        const int m = m0 + e / GM_ROWS;
        const long long n = nc + e % GM_ROWS;
        if (m < p.M && n < p.N) store_y(p.Y, p.y_bf16, (long long)m * p.N + n, p.x_scale ? y * p.x_scale[m] : y);
    };
    constexpr int E = TOK * GM_ROWS;
    if (p.split == 1) {
        for (int e = tid; e < E; e += GM_THREADS) finish(e, sums[e] + sums[E + e]);
    } else {
        __syncwarp();
        cluster_sync_all();
        for (int e = (int)rank * GM_THREADS + tid; e < E; e += (int)p.split * GM_THREADS)
            finish(e, cluster_sum<2>(smem_u32(sums + e), 4 * E, (int)p.split));
        __syncwarp();
        cluster_sync_all();   // no CTA leaves while its sums are being read
    }
}

// Activation order: any column in any group.  The work is a lookup of a scale and a zero point for every
// weight, so the CTA keeps those of all groups for its 32 rows n in shared memory, as (scale, 1024 + zero
// point) in fp16: one 16-byte read gives a column's entries for the 4 neighbouring rows of a thread, and
// the packed words are read along n.  A warp takes 32 columns at a time, in the fragment order of
// gemv_mma_kernel; the 8 warps of a CTA and the CTAs of a cluster split K.  s (q - z) (at most 11 + 8
// significant bits) is formed in fp32 without rounding and cut into bf16 parts that hold it exactly (two
// for codes of up to 4 bits, three for 8 bits), so the products are exact and the sums fp32, and a
// weight's decoding and cutting, some 14 instructions, serve up to 32 tokens.
// Bound by instruction issue: 4096 x 11008, 4-bit groups of 128, all inputs from memory, 2 or 8 tokens
// 47 us, 16 tokens 51 us, 64 tokens in two tiles 106 us.  fp32 multiply-adds in place of the tensor
// instruction took three times as long for 8 tokens.  Where the table does not fit (above 1280 groups), TABLE
// is false and every weight's entry is read from global memory (4 tokens through 4096 x 32768, groups of
// 16: 410 us).
constexpr int GA_THREADS = 256, GA_ROWS = 32;
constexpr int GA_TABLE = 160 * 1024;   // bytes of the table, at most

// The table's entries for the rows from nc on.
template <int BITS>
__device__ __forceinline__ void act_table(const GemvArgs& p, __half2* table, long long nc) {
    const long long zwords = (p.N * BITS + 31) / 32;
    for (int e = threadIdx.x; e < p.ng * GA_ROWS; e += GA_THREADS) {
        const int gi = e / GA_ROWS;
        const long long n = nc + e % GA_ROWS;
        __half s = __float2half(0.f);
        uint32_t z = 1u << (BITS - 1);
        if (n < p.N) {
            s = p.scales[(long long)gi * p.N + n];
            if (p.qzeros != nullptr) z = stream_code(p.qzeros + gi * zwords, 1, n, BITS);
        }
        table[e] = __halves2half2(s, __ushort_as_half((unsigned short)(0x6400u | z)));   // 1024 + z
    }
}
// The one or two words of the columns k .. k + 7 of four neighbouring rows.
template <int BITS>
__device__ __forceinline__ void act_words(const GemvArgs& p, int k, long long n0, uint32_t (&w)[2][4]) {
    const long long r = (long long)k * BITS / 32;
    // 24 bits from bit 16 or 24 of a word on end in the next
    const int words = BITS == 8 || (BITS == 3 && ((k * 3) & 31) > 8) ? 2 : 1;
#pragma unroll
    for (int i = 0; i < (BITS == 8 || BITS == 3 ? 2 : 1); ++i) {
        const int32_t* src = p.qweight + (r + (i < words ? i : 0)) * p.N + n0;
        if (p.vec) {
            const uint4 u = n0 < p.N ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = n0 + j < p.N ? (uint32_t)__ldg(src + j) : 0u;
        }
    }
}
// Entries of a group for the rows n0 .. n0 + 3, as the table holds them.
template <int BITS>
__device__ __forceinline__ uint4 act_entries(const GemvArgs& p, int gi, long long n0) {
    const long long zwords = (p.N * BITS + 31) / 32;
    uint32_t e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t s = 0, z = 1u << (BITS - 1);
        if (n0 + j < p.N) {
            s = __half_as_ushort(p.scales[(long long)gi * p.N + n0 + j]);
            if (p.qzeros != nullptr) z = stream_code(p.qzeros + gi * zwords, 1, n0 + j, BITS);
        }
        e[j] = s | (0x6400u | z) << 16;   // 1024 + z
    }
    return make_uint4(e[0], e[1], e[2], e[3]);
}
// Joins the warps' sums [8][TOK][GA_ROWS], then the CTAs' of the cluster, in a fixed order, and stores.
template <int TOK>
__device__ __forceinline__ void act_join(const GemvArgs& p, float* sums, long long nc, int m0, unsigned rank) {
    constexpr int ROWS = GA_ROWS, E = TOK * ROWS;
    const int tid = threadIdx.x;
    __syncthreads();
    auto finish = [&](int e, float y) {
        const int m = m0 + e / ROWS;
        const long long n = nc + e % ROWS;
        if (m < p.M && n < p.N) store_y(p.Y, p.y_bf16, (long long)m * p.N + n, p.x_scale ? y * p.x_scale[m] : y);
    };
    for (int e = tid; e < E; e += GA_THREADS) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < GA_THREADS / 32; ++w) y += sums[w * E + e];
        if (p.split == 1)
            finish(e, y);
        else
            sums[e] = y;   // read above by this thread alone
    }
    if (p.split > 1) {
        __syncwarp();
        cluster_sync_all();
        for (int e = (int)rank * GA_THREADS + tid; e < E; e += (int)p.split * GA_THREADS)
            finish(e, cluster_sum<1>(smem_u32(sums + e), 0, (int)p.split));
        __syncwarp();
        cluster_sync_all();   // no CTA leaves while its sums are being read
    }
}

// Pairs (i, i + 4) of a thread's columns as bf16, which holds e4m3 exactly.
template <typename XT>
__device__ __forceinline__ void x_pairs_bf16(const XRaw<XT>& r, uint32_t (&b)[4]) {
    if constexpr (sizeof(XT) == 2) {
        x_pairs<false>(r, b);
    } else {
        float x[8];
        x_floats(r, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = bits_of(__floats2bfloat162_rn(x[i], x[i + 4]));
    }
}

template <int BITS, typename XT, int MT, bool TABLE>
__global__ void __launch_bounds__(GA_THREADS, MT == 1 ? 3 : 2) gemv_act_kernel(const GemvArgs p) {
    constexpr int ROWS = GA_ROWS, TOK = 8 * MT, PARTS = BITS == 8 ? 3 : 2, E = TOK * ROWS;
    extern __shared__ __align__(16) uint8_t ga_smem[];
    __half2* table = reinterpret_cast<__half2*>(ga_smem);   // [ng][ROWS]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
    const unsigned cta = blockIdx.x / p.split, rank = blockIdx.x % p.split;
    const long long nc = (long long)(cta % p.nblocks) * ROWS, n0 = nc + 4 * gid;
    const int m0 = (int)(cta / p.nblocks) * TOK;
    const int K = (int)p.K, steps = (K + 31) / 32;
    const XT* X = reinterpret_cast<const XT*>(p.X);
    if (TABLE) act_table<BITS>(p, table, nc);
    __syncthreads();

    const int s0 = (int)((long long)steps * rank / p.split), s1 = (int)((long long)steps * (rank + 1) / p.split);
    struct Chunk {
        uint32_t w[2][4];
        int g[8];
        XRaw<XT> x[MT];
    };
    auto load = [&](int st, Chunk& q) {   // columns k .. k + 7; none behind the last
        const int k = 32 * st + 8 * tig;
        q = Chunk{};
        if (k >= K) return;
        act_words<BITS>(p, k, n0, q.w);
#pragma unroll
        for (int j = 0; j < 8; ++j) q.g[j] = __ldg(p.g_idx + k + j);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            if (m0 + 8 * mt + gid < p.M) q.x[mt] = load_x8(X + (long long)(m0 + 8 * mt + gid) * K + k);
    };
    // Tile j: rows n0 + j and n0 + j + 2.  The tensor instruction may cut its sums off, always in the same
    // direction, so those of 32 columns are added up in fp32.  Four token tiles leave no registers for that
    // (64 tokens through 4096 x 11008: 117 us) and add those of 64 columns to sums in shared memory (106 us).
    constexpr bool PARKED = MT == 4;
    float sum[2][MT][4] = {}, part[2][MT][4] = {};
    float4* parked = reinterpret_cast<float4*>(ga_smem + (TABLE ? p.ng * ROWS * 4 : 0)) + warp * (2 * MT * 32) + lane;
    bool odd = false;
    auto add_part = [&] {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (PARKED) {
                    float4& s = parked[(j * MT + mt) * 32];
                    const float4 v = s;
                    s = make_float4(v.x + part[j][mt][0], v.y + part[j][mt][1], v.z + part[j][mt][2], v.w + part[j][mt][3]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (!PARKED) sum[j][mt][c] += part[j][mt][c];
                    part[j][mt][c] = 0.f;
                }
            }
    };
    if (PARKED)
        for (int i = 0; i < 2 * MT; ++i) parked[i * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
    Chunk now = {}, next = {};
    int st = s0 + warp;
    if (st < s1) load(st, now);
    for (; st < s1; st += GA_THREADS / 32) {
        if (st + GA_THREADS / 32 < s1) load(st + GA_THREADS / 32, next);
        const bool in = 32 * st + 8 * tig < K;
        uint32_t nib[4];
        if constexpr (BITS <= 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) nib[j] = chunk_nibbles<BITS>(now.w[0][j], now.w[1][j], tig);
        }
        uint32_t xb[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) x_pairs_bf16<XT>(now.x[mt], xb[mt]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // pairs (i, i + 4) of columns, i = 2 h and 2 h + 1
            uint32_t a[PARTS][4][2];
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
                const int i = 2 * h + i2;
                uint4 e[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    int gi = now.g[i + 4 * t];
                    if ((unsigned)gi >= (unsigned)p.ng) {
                        if (gid == 0) record_status(GPTQ_ERR_INVALID_ARG, 32ll * st + 8 * tig + i + 4 * t);
                        gi = 0;
                    }
                    e[t] = TABLE ? *reinterpret_cast<const uint4*>(table + gi * ROWS + 4 * gid)
                                 : act_entries<BITS>(p, gi, n0);
                }
                const uint32_t e0[4] = {e[0].x, e[0].y, e[0].z, e[0].w}, e1[4] = {e[1].x, e[1].y, e[1].z, e[1].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t q0 = BITS <= 4 ? nib[j] >> (4 * i) & 15u : now.w[0][j] >> (8 * i) & 255u;
                    const uint32_t q1 = BITS <= 4 ? nib[j] >> (4 * i + 16) & 15u : now.w[1][j] >> (8 * i) & 255u;
                    const float2 z0 = __half22float2(as_half2(e0[j])), z1 = __half22float2(as_half2(e1[j]));
                    float w0 = z0.x * (__uint_as_float(0x44800000u | (q0 << 13)) - z0.y);
                    float w1 = z1.x * (__uint_as_float(0x44800000u | (q1 << 13)) - z1.y);
#pragma unroll
                    for (int c = 0; c < PARTS; ++c) {
                        const uint32_t u = bits_of(__floats2bfloat162_rn(w0, w1));
                        a[c][j][i2] = in ? u : 0u;
                        w0 -= __uint_as_float(u << 16);
                        w1 -= __uint_as_float(u & 0xFFFF0000u);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < PARTS; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        mma_16816(part[j][mt], a[c][j][0], a[c][j + 2][0], a[c][j][1], a[c][j + 2][1], xb[mt][2 * h],
                                  xb[mt][2 * h + 1], __nv_bfloat16());
        }
        if (!PARKED || odd) add_part();
        odd = !odd;
        now = next;
    }
    if (PARKED) {
        add_part();
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const float4 v = parked[i * 32];
            sum[i / MT][i % MT][0] = v.x;
            sum[i / MT][i % MT][1] = v.y;
            sum[i / MT][i % MT][2] = v.z;
            sum[i / MT][i % MT][3] = v.w;
        }
    }

    __syncthreads();
    float* sums = reinterpret_cast<float*>(ga_smem);   // [8 warps][TOK][ROWS]
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sums[warp * E + (8 * mt + 2 * tig + (c & 1)) * ROWS + 4 * gid + j + (c & 2)] = sum[j][mt][c];
    act_join<TOK>(p, sums, nc, m0, rank);
}

}  // namespace gq

namespace gqh {

int num_sms();

template <int BITS, typename XT, int MT, int GROUPS>
cudaError_t gemv_mma_launch(gq::GemvArgs p, cudaStream_t st) {
    using Cfg = gq::GmCfg<BITS, XT, MT, GROUPS>;
    constexpr auto kern = gq::gemv_mma_kernel<BITS, XT, MT, GROUPS>;
    GQ_TRY((smem_attr_once<kern, Cfg::SMEM>()));
    p.nblocks = (unsigned)((p.N + gq::GM_ROWS - 1) / gq::GM_ROWS);
    p.vec = p.N % 4 == 0;
    p.gshift = p.g_all ? 31 : p.g == 128 ? 7 : p.g == 64 ? 6 : p.g == 32 ? 5 : 4;
    const long long blocks = (long long)p.nblocks * ((p.M + Cfg::TOK - 1) / Cfg::TOK);
    // K is split over a cluster where that shortens the run.  An SM's time for its share of the CTAs, in
    // tenths of a stage that a CTA does alone: k CTAs side by side take 3 + 7 k for a stage of each (1.7
    // and 2.4 times a single one's, measured), and a wave takes 25 for its start and end.
    const long long nst = (p.K + gq::GM_K - 1) / gq::GM_K;
    long long best = 0;
    for (unsigned s = 1; s <= 8 && s <= nst; s *= 2) {
        const long long ctas = (blocks * s + num_sms() - 1) / num_sms(), waves = (ctas + Cfg::CTAS - 1) / Cfg::CTAS;
        const long long cost = (nst + s - 1) / s * (3 * waves + 7 * ctas) + 25 * waves;
        if (s == 1 || cost < best) {
            best = cost;
            p.split = s;
        }
    }
    if (blocks * p.split > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * p.split));
    cfg.blockDim = dim3(gq::GM_THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 1 : 0;
    CUtensorMap mw = {}, mx = {};
    p.tma = p.vec && (sizeof(XT) == 2 || p.K % 16 == 0);
    if (p.tma && (!tmap_2d(&mw, p.qweight, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, (uint64_t)((p.K * BITS + 31) / 32),
                           (uint64_t)p.N, Cfg::WROWS, 32, true) ||
                  !tmap_2d(&mx, p.X, sizeof(XT) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                           (int)sizeof(XT), (uint64_t)p.M, (uint64_t)p.K, Cfg::TOK, gq::GM_K, false)))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mw, mx, p);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

// The token tile follows M, as every tile of 8 tokens costs its MMAs whether it is filled or not (16
// tokens in a tile of 16 against one of 32: 34 us against 42 us, 3 bits, groups of 64, 11008 x 4096).
template <int BITS, typename XT>
cudaError_t gemv_mma_run(const gq::GemvArgs& p, cudaStream_t st) {
    if (p.g_all || p.g == 128) {
        if (p.M <= 8) return gemv_mma_launch<BITS, XT, 1, 1>(p, st);
        if (p.M <= 16) return gemv_mma_launch<BITS, XT, 2, 1>(p, st);
        return gemv_mma_launch<BITS, XT, 4, 1>(p, st);
    }
    if (p.g == 16) return gemv_mma_launch<BITS, XT, 2, 8>(p, st);
    if (p.M <= 8) return gemv_mma_launch<BITS, XT, 1, 4>(p, st);
    if (p.M <= 16) return gemv_mma_launch<BITS, XT, 2, 4>(p, st);
    return gemv_mma_launch<BITS, XT, 4, 4>(p, st);
}

template <int BITS, typename XT, int MT, bool TABLE>
cudaError_t gemv_act_launch(gq::GemvArgs p, cudaStream_t st) {
    constexpr int TOK = 8 * MT, ROWS = gq::GA_ROWS;
    constexpr auto kern = gq::gemv_act_kernel<BITS, XT, MT, TABLE>;
    constexpr int SUMS = gq::GA_THREADS / 32 * TOK * ROWS * 4;   // of the warps, in the table's place when it is done with
    constexpr int PARKED = MT == 4 ? SUMS : 0;
    GQ_TRY((smem_attr_once<kern, gq::GA_TABLE + PARKED>()));
    p.nblocks = (unsigned)((p.N + ROWS - 1) / ROWS);
    p.vec = p.N % 4 == 0;
    const long long blocks = (long long)p.nblocks * ((p.M + TOK - 1) / TOK);
    // K is split until there is a CTA to an SM, with 64 columns at least for each warp: every CTA builds
    // its table, so two to an SM took 44 us where this takes 38 us (2 tokens, 4096 x 11008)
    p.split = 1;
    while (p.split < 8 && blocks * p.split < num_sms() && p.K >= 8ll * 32 * 2 * p.split) p.split *= 2;
    if (blocks * p.split > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * p.split));
    cfg.blockDim = dim3(gq::GA_THREADS);
    cfg.dynamicSmemBytes = std::max((TABLE ? (size_t)p.ng * ROWS * 4 : 0) + PARKED, (size_t)SUMS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

template <int BITS, typename XT>
cudaError_t gemv_act_run(const gq::GemvArgs& p, cudaStream_t st) {
    if ((long long)p.ng * gq::GA_ROWS * 4 > gq::GA_TABLE) return gemv_act_launch<BITS, XT, 1, false>(p, st);
    if (p.M <= 8) return gemv_act_launch<BITS, XT, 1, true>(p, st);
    if (p.M <= 16) return gemv_act_launch<BITS, XT, 2, true>(p, st);
    return gemv_act_launch<BITS, XT, 4, true>(p, st);
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
    switch (p.bits) {
        case 2: return gemv_act_run<2, XT>(p, st);
        case 3: return gemv_act_run<3, XT>(p, st);
        case 4: return gemv_act_run<4, XT>(p, st);
        default: return gemv_act_run<8, XT>(p, st);
    }
}

inline cudaError_t gemv_run(const gq::GemvArgs& p, bool x_e4m3, cudaStream_t st) {
    return x_e4m3 ? gemv_run_x<__nv_fp8_e4m3>(p, st) : gemv_run_x<__nv_bfloat16>(p, st);
}

}  // namespace gqh
