// Dequantizing GEMM on e4m3 activations:
//
//   Y[m, n] = xs[m] sum_g s_g[n] P_g[n, m],   P_g[n, m] = sum_{k in g} (q[n, k] - z_g[n]) X8[m, k]
//
// q - z of 2, 3 and 4 bits is exact in e4m3, so P_g is formed by the 8-bit tensor
// instructions (twice the bf16 rate) from exact products with fp32 accumulation; s_g and xs are
// applied in fp32.  No rounded copy of W_hat is made.
//
// The weights are the A operand (128 rows n of a tile) and sit in tensor memory: a converter
// thread owns one row, turns its packed codes into e4m3 bytes and stores them with tcgen05.st, so
// shared memory carries only X8 (the B operand) and the packed words.  With rows on the lanes, a
// group's scale is one register of an epilogue thread.
//
// A tile is 128 rows x TT tokens (64 up to 64 tokens, else 128), K advances by 128.  One CTA per SM,
// 20 warps:
//   warps 0-7    converters, two sets that take turns, a thread per row, a ring of three A operands;
//   warps 8-15   epilogue: two warps per lane quadrant, TT / 2 tokens each, running sums in
//                registers: y += s_g P_g;
//   warp 16      TMA: X8 tile (TT tokens x 128 bytes, 128-byte swizzle) and packed words
//                (4 BITS words x 128 rows) into a ring of stages;
//   warp 17      MMA issuer: per quantization group one accumulator segment, in a ring of
//                accumulators of tensor memory;
//   warp 18      the groups' fp16 scales and packed zero points by asynchronous copies into a
//                ring of their own (they outlive the stage: the epilogue scales later).
// The epilogue takes registers that the others give up (setmaxnreg).  Every wait is bounded
// (GPTQ_ERR_TIMEOUT).  No TMA multicast.
//
// Codes to e4m3: a byte b < 16 read as e4m3 is b 2^-9 (the subnormals and the first binade are one
// arithmetic sequence), so |q - z|, with the sign in bit 7, is (q - z) 2^-9.  A group's 2^BITS bytes come
// as 4 registers from a table of 16 zero points in shared memory, and byte permutes look four codes up.
// The MMAs then sum exact products of q - z: P_g carries the rounding of sums of |q - z| |X8| and is 0
// where every code is at the zero point.  (Spread codes as they are and a second pass of MMAs with -z
// would round sums of (q + z) |X8|, which for codes near z can be hundreds of times larger.)
//
// What bounds it: no unit is full.  A 128-column K tile takes about 1070 clocks (2048 tokens x 4096 x 4096),
// of which the MMAs are 260 (four of 65 clocks); 66 % of the issue slots are used, most by the converters and
// the epilogue, whose latencies add up along the ring of operands.  4-bit groups of 128: 2048
// tokens x 4096 x 4096 in 76 us (900 TFLOP/s), 8192 tokens x 11008 x 4096 in 663 us (1115 TFLOP/s, 34 % of
// the 8-bit rate); groups of 64 and 32 take 104 and 169 us for the former, as every group is an accumulator
// to drain.  Looking q - z up takes 11 instructions for 8 codes of 4 bits (3 or 2 bits: 3 after spreading
// them to nibbles), spreading alone 5, which with the second pass of MMAs took 74 and 729 us.
//
// Few tiles: the K range is split over a cluster of S CTAs, whose partial sums are joined
// through distributed shared memory in rank order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "host_once.h"
#include "pack.cuh"

namespace gq {

constexpr int D8_THREADS = 640;
constexpr int D8_EPI_WARP0 = 8, D8_PROD_WARP = 16;   // converters 0-7, epilogue 8-15, TMA 16, MMA 17, scales 18
constexpr int D8_AST = 3, D8_PST = 8, D8_LAG = 2;
// Registers a thread after setmaxnreg, per warpgroup.  A split above what the launch gave would wait
// forever, so the launch checks that the kernel was compiled to D8_REGS.
constexpr int D8_REGS = 96, D8_REGS_CONV = 56, D8_REGS_EPI = 160, D8_REGS_MISC = 48;
static_assert(2 * D8_REGS_CONV + 2 * D8_REGS_EPI + D8_REGS_MISC <= D8_THREADS / 128 * D8_REGS, "register split");
constexpr int D8_PAR_S = 1024, D8_PAR_Z = 256;   // bytes of scales and zero points of four groups
constexpr int D8_LUT = 256;                      // bytes of (q - z) 2^-9 as e4m3 for 16 z, 16 q
constexpr int D8_SEG_TILES = 4;   // K tiles per segment for one group per row: 16 MMAs in place

template <int BITS, int TT>
struct D8Cfg {
    static constexpr int KW = 4 * BITS;               // packed words per row and K tile
    static constexpr int X_BYTES = TT * 128;
    static constexpr int P_BYTES = KW * 128 * 4;
    static constexpr int STAGE_BYTES = X_BYTES + P_BYTES;
    static constexpr int FIT = (206 * 1024) / STAGE_BYTES;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int C = TT / 2;                  // tokens per epilogue warp
    static constexpr int ND = 384 / TT;               // accumulators
    static constexpr int SMEM =
        1024 + STAGES * STAGE_BYTES + D8_PST * (D8_PAR_S + D8_PAR_Z) + D8_LUT + 8 * TT + 512;
    static_assert(STAGE_BYTES % 1024 == 0, "the swizzled tiles stay 1024-byte aligned");
    static_assert(TT * 128 * 4 <= STAGES * STAGE_BYTES, "partial sums fit the ring");
};

// Tensor memory: accumulators in front, then a ring of D8_AST operands of 32 columns.
constexpr int D8_ACC_COLS = 384, D8_A_COLS = 32;
static_assert(D8_ACC_COLS + D8_AST * D8_A_COLS <= 512, "TMEM");

struct D8Args {
    const __half* scales;    // [n_groups, N]
    const int32_t* qzeros;   // [n_groups, ceil(N BITS / 32)] or null
    const float* x_scale;    // [M]
    void* Y;                 // [M, N]
    int y_bf16;
    int M, N, K;
    int spt;                 // segments per K tile (groups of 32, 64, 128), 0 for one group per row
    int tiles_n, tiles;      // tiles_n x token tiles, n fastest
    int split;               // cluster size
};

__device__ __forceinline__ void umma_e4m3_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc));
}

// Whether a barrier's phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// 32 lanes x 16 consecutive columns, one column per register.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t s) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(s));
    return r;
}
// The 32 codes of BITS words as 8 words of one e4m3 byte per code, taken from t, whose byte q stands for
// code q.
template <int BITS>
__device__ __forceinline__ void codes_to_bytes(const uint32_t (&w)[BITS], const uint4& t, uint32_t* out) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t v;   // eight codes, one per nibble
        if constexpr (BITS == 4)
            v = w[c];
        else if constexpr (BITS == 2)
            v = codes_to_nibbles<2>((w[c >> 1] >> (16 * (c & 1))) & 0xFFFFu);
        else
            v = codes_to_nibbles<3>(
                (c == 0 ? w[0] : c == 3 ? w[2] >> 8 : __funnelshift_r(w[c - 1], w[c], c == 1 ? 24 : 16)) & 0xFFFFFFu);
        // a selector takes four nibbles, of which bits 0-2 pick one of eight bytes and bit 3 must be 0
        if constexpr (BITS == 4) {
            const uint32_t low = v & 0x77777777u, high = ((v >> 1) & 0x44444444u) | 0x32103210u;
            out[2 * c] = byte_perm(byte_perm(t.x, t.y, low), byte_perm(t.z, t.w, low), high);
            out[2 * c + 1] = byte_perm(byte_perm(t.x, t.y, low >> 16), byte_perm(t.z, t.w, low >> 16), high >> 16);
        } else {
            out[2 * c] = byte_perm(t.x, t.y, v);
            out[2 * c + 1] = byte_perm(t.x, t.y, v >> 16);
        }
    }
}

// One lane's column of C rows of Y, scaled; rows past the end are left alone.
__device__ __forceinline__ void put(float* y, float v) { *y = v; }
__device__ __forceinline__ void put(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }
template <int C, typename YT>
__device__ __forceinline__ void store_rows(YT* y, int ld, int rows, const float (&acc)[C], const float* xs) {
#pragma unroll
    for (int j = 0; j < C; j += 4) {
        const float4 x = *reinterpret_cast<const float4*>(xs + j);
        const float xv[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (j + i < rows) put(y, acc[j + i] * xv[i]);
            y += ld;
        }
    }
}

// A warp waits for up to three barriers (those with a true, warp-uniform flag).  They are tried
// together, so that their latencies overlap.  Every lane waits: lanes must not part ways in front of
// the tcgen05 loads and stores, which need the warp converged.  Warp-uniform.
__device__ __forceinline__ bool warp_wait(int where, uint64_t* b0, uint32_t p0, bool w0, uint64_t* b1, uint32_t p1,
                                          bool w1, uint64_t* b2, uint32_t p2, bool w2) {
    const bool r0 = !w0 || mbar_try_wait(b0, p0), r1 = !w1 || mbar_try_wait(b1, p1), r2 = !w2 || mbar_try_wait(b2, p2);
    return __all_sync(~0u, (r0 || mbar_wait(b0, p0, where)) && (r1 || mbar_wait(b1, p1, where)) &&
                               (r2 || mbar_wait(b2, p2, where)));
}
__device__ __forceinline__ bool warp_wait(int where, uint64_t* b, uint32_t p) {
    return __all_sync(~0u, mbar_wait(b, p, where));
}

template <int BITS, int TT>
__global__ void __launch_bounds__(D8_THREADS, 1)
    dq_gemm_e4m3_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mP, const D8Args p) {
    using Cfg = D8Cfg<BITS, TT>;
    constexpr int STAGES = Cfg::STAGES, C = Cfg::C, ND = Cfg::ND;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);   // an offset, so that accesses stay shared-memory ones
    uint8_t* par = smem + STAGES * Cfg::STAGE_BYTES;   // [PST] scales [4][128] fp16, zero points [4][16] words
    uint8_t* lut = par + D8_PST * (D8_PAR_S + D8_PAR_Z);   // [16 zero points][16 codes]
    // [2][TT] scales of the tokens of this tile and the next
    float* xs = reinterpret_cast<float*>(lut + D8_LUT);
    uint64_t* full = reinterpret_cast<uint64_t*>(xs + 2 * TT);   // [STAGES] TMA landed
    uint64_t* empty = full + STAGES;                         // [STAGES] MMAs of the stage done
    uint64_t* conv = empty + STAGES;                         // [AST] A operand written
    uint64_t* aempty = conv + D8_AST;                        // [AST] A operand read
    uint64_t* dfull = aempty + D8_AST;                       // [ND] segment complete
    uint64_t* dempty = dfull + ND;                        // [ND] segment drained
    uint64_t* pfull = dempty + ND;                        // [PST] scales and zero points landed
    uint64_t* pempty = pfull + D8_PST;                       // [PST] scales and zero points used
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pempty + D8_PST);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < D8_AST; ++s) {
            mbar_init(&conv[s], 4);
            mbar_init(&aempty[s], 1);
        }
        for (int s = 0; s < ND; ++s) {
            mbar_init(&dfull[s], 1);
            mbar_init(&dempty[s], 8);
        }
        for (int s = 0; s < D8_PST; ++s) {
            mbar_init(&pfull[s], 1);
            mbar_init(&pempty[s], 9);
        }
        fence_mbar_init();
    }
    if (threadIdx.x < D8_LUT) {
        const int d = (int)(threadIdx.x & 15) - (int)(threadIdx.x >> 4);
        lut[threadIdx.x] = (uint8_t)(d < 0 ? 0x80 | -d : d);
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t a_ring = tmem + D8_ACC_COLS;

    // K tiles of this CTA, and the segments in them
    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int nkt_all = (p.K + 127) / 128;
    const int kt0 = (int)((long long)nkt_all * rank / p.split);
    const int nkt = (int)((long long)nkt_all * (rank + 1) / p.split) - kt0;
    const int step = (int)gridDim.x / p.split, first = (int)blockIdx.x / p.split;
    // the last K tile may hold fewer groups than spt
    const int nseg = p.spt ? min((kt0 + nkt) * p.spt, p.K / (128 / p.spt)) - kt0 * p.spt
                           : (nkt + D8_SEG_TILES - 1) / D8_SEG_TILES;

    if (warp < D8_EPI_WARP0) {
        // ---------------- converters: thread t of a set owns row n0 + t; the two sets take turns
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(D8_REGS_CONV));
        const int qd = warp & 3, t = 32 * qd + lane;
        const uint32_t set = warp >> 2;
        const uint32_t a_row = a_ring + ((uint32_t)(32 * qd) << 16);
        // units of four groups in a tile; one without groups in it (one group per row) is a single unit
        const uint32_t units = p.spt ? (nseg + 3) / 4 : 1;
        const uint4* table = reinterpret_cast<const uint4*>(lut);
        uint4 lookup = table[1 << (BITS - 1)];
        uint32_t it0 = 0, unit0 = 0, seen = ~0u;   // of the tile; last unit waited for
        bool ok = true;
        for (int w = first; w < p.tiles && ok; w += step, it0 += nkt, unit0 += units) {
            for (int kt = (int)((it0 ^ set) & 1); kt < nkt; kt += 2) {
                const uint32_t it = it0 + kt, s = it % STAGES, a = it % D8_AST;
                const int grp = kt * p.spt;   // the K tile's first group, counted from the CTA's first
                const uint32_t unit = unit0 + (uint32_t)grp / 4;
                const bool fresh = p.qzeros != nullptr && unit != seen;
                ok = warp_wait(w, &full[s], (it / STAGES) & 1, true, &aempty[a], ((it / D8_AST) & 1) ^ 1, true,
                               &pfull[unit % D8_PST], (unit / D8_PST) & 1, fresh);
                if (!ok) break;
                seen = unit;
                tc_fence_after();
                const uint32_t* col =
                    reinterpret_cast<const uint32_t*>(smem + s * Cfg::STAGE_BYTES + Cfg::X_BYTES) + t;
                const uint32_t dst = a_row + D8_A_COLS * a;
                const uint8_t* zq = par + (unit % D8_PST) * (D8_PAR_S + D8_PAR_Z) + D8_PAR_S;
                auto zero_point = [&](int q) {   // of a group, counted as grp is
                    const uint32_t* zw = reinterpret_cast<const uint32_t*>(zq + 64 * (q & 3));
                    const int b = t * BITS;
                    uint32_t z = zw[b >> 5] >> (b & 31);
                    if (BITS == 3 && (b & 31) > 29) z |= zw[(b >> 5) + 1] << (32 - (b & 31));
                    return z & ((1u << BITS) - 1u);
                };
                uint32_t words[4][BITS];
#pragma unroll
                for (int i = 0; i < 4 * BITS; ++i) words[i / BITS][i % BITS] = col[i * 128];
                if (p.qzeros != nullptr && p.spt <= 1) lookup = table[zero_point(grp)];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[16];
                    // groups of 64 and 32: the table changes within the K tile
                    if (p.qzeros != nullptr && p.spt > 1) lookup = table[zero_point(grp + (p.spt >> 1) * h)];
                    codes_to_bytes<BITS>(words[2 * h], lookup, r);
                    if (p.qzeros != nullptr && p.spt > 2) lookup = table[zero_point(grp + 2 * h + 1)];
                    codes_to_bytes<BITS>(words[2 * h + 1], lookup, r + 8);
                    tmem_st_32x32b_x16(dst + 16 * h, r);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&conv[a]);
                __syncwarp();
            }
        }
    } else if (warp < D8_PROD_WARP) {
        // ---------------- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(D8_REGS_EPI));
        const int ew = warp - D8_EPI_WARP0, qd = warp & 3, half = ew >> 2;
        const uint32_t lane_off = (uint32_t)(32 * qd) << 16;
        const uint32_t col0 = (uint32_t)(half * C);   // columns of the accumulator
        const int et = threadIdx.x - 32 * D8_EPI_WARP0;
        uint32_t buf = 0, dph = 0, unit = 0;   // accumulator and its phase
        bool ok = true;   // once false, the loop goes on without waiting: its barriers need every warp
        // The tokens' scales are fetched a tile ahead, as their way from memory is longer than a K tile.
        auto token_scale = [&](int w) {
            const int m = (w / p.tiles_n) * TT + et;
            return et < TT && w < p.tiles && m < p.M ? p.x_scale[m] : 0.f;
        };
        int xs_off = 0;
        float xs_next = token_scale(first);
        for (int w = first; w < p.tiles; w += step, xs_off ^= TT) {
            const int n = (w % p.tiles_n) * 128 + 32 * qd + lane, m0 = (w / p.tiles_n) * TT;
            // the other half is free: every warp has passed the barrier below since it was read
            if (et < TT) xs[xs_off + et] = xs_next;
            xs_next = token_scale(w + step);
            float acc[C];
#pragma unroll
            for (int j = 0; j < C; ++j) acc[j] = 0.f;
            // the scales of four groups, the next one in the low half of .x
            uint2 sq = {0, 0};
            auto scales = [&] {
                ok = warp_wait(w, &pfull[unit % D8_PST], (unit / D8_PST) & 1);
                const uint16_t* sp = reinterpret_cast<const uint16_t*>(par + (unit % D8_PST) * (D8_PAR_S + D8_PAR_Z)) +
                                     32 * qd + lane;
                sq.x = sp[0] | (uint32_t)sp[128] << 16;
                sq.y = sp[256] | (uint32_t)sp[384] << 16;
                __syncwarp();
                if (lane == 0) mbar_arrive(&pempty[unit % D8_PST]);
                __syncwarp();
                ++unit;
            };
            if (ok) scales();
            bool ready = false;   // the next accumulator was complete when last looked at
            for (int sg = 0; sg < nseg && ok; ++sg) {
                const float s = 512.f * __half2float(__ushort_as_half((uint16_t)sq.x));   // P_g comes as 2^-9 P_g
                if (!ready) {
                    ok = warp_wait(w, &dfull[buf], dph);
                    if (!ok) break;
                }
                tc_fence_after();
                uint32_t r[C / 32][32];
#pragma unroll
                for (int c = 0; c < C / 32; ++c) tmem_ld_32x32b_x32(tmem + buf * TT + col0 + 32 * c + lane_off, r[c]);
                if (p.spt && sg + 1 < nseg) {
                    if ((sg & 3) == 3) {
                        scales();
                    } else {
                        sq.x = sq.x >> 16 | sq.y << 16;
                        sq.y >>= 16;
                    }
                }
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&dempty[buf]);
                __syncwarp();
                if (++buf == ND) {
                    buf = 0;
                    dph ^= 1;
                }
                // looked at here, the barrier's latency passes under the multiplications
                ready = __all_sync(~0u, mbar_test_wait(&dfull[buf], dph));
#pragma unroll
                for (int j = 0; j < C; ++j) acc[j] = fmaf(s, __uint_as_float(r[j / 32][j % 32]), acc[j]);
            }
            const int j0 = half * C;   // this warp's first token of the tile
            asm volatile("bar.sync 1, 256;" ::: "memory");   // the tokens' scales are written
            if (p.split == 1) {
                if (ok && n < p.N) {
                    const int rows = p.M - m0 - j0;
                    const long long at = (long long)(m0 + j0) * p.N + n;
                    if (p.y_bf16)
                        store_rows<C>(reinterpret_cast<__nv_bfloat16*>(p.Y) + at, p.N, rows, acc, xs + xs_off + j0);
                    else
                        store_rows<C>(reinterpret_cast<float*>(p.Y) + at, p.N, rows, acc, xs + xs_off + j0);
                }
            } else {
                // One tile per cluster.  The partial sums take the ring's place once the last MMAs
                // have read it.
                float* red = reinterpret_cast<float*>(smem);   // [TT][128]
                if (ok) ok = mbar_wait(&empty[(nkt - 1) % STAGES], ((nkt - 1) / STAGES) & 1, w);
                if (ok) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        red[(j0 + j) * 128 + 32 * qd + lane] = acc[j];
                }
                __syncwarp();
                cluster_sync_all();
                // rank r finishes the tokens r, r + split, ..., a warp a token; N is a multiple of 8
                const int c = 4 * lane, nn = (w % p.tiles_n) * 128 + c;
                for (int j = rank + p.split * ew; j < TT && m0 + j < p.M; j += 8 * p.split) {
                    if (nn < p.N) {
                        const float4 y = cluster_sum4(smem_u32(red + j * 128 + c), p.split);
                        const float x = xs[xs_off + j];
                        store_y4(p.Y, p.y_bf16, (long long)(m0 + j) * p.N + nn,
                                 make_float4(y.x * x, y.y * x, y.z * x, y.w * x));
                    }
                }
                __syncwarp();
                cluster_sync_all();   // no CTA leaves while its partial sums are being read
            }
        }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(D8_REGS_MISC));
      if (warp == D8_PROD_WARP && lane == 0) {
        // ---------------- producer: X8 and packed words by TMA
        prefetch_tmap(&mX);
        prefetch_tmap(&mP);
        uint32_t it = 0;
        bool ok = true;
        for (int w = first; w < p.tiles && ok; w += step) {
            const int n0 = (w % p.tiles_n) * 128, m0 = (w / p.tiles_n) * TT;
            for (int kt = 0; kt < nkt; ++kt, ++it) {
                const uint32_t s = it % STAGES;
                ok = mbar_wait(&empty[s], ((it / STAGES) & 1) ^ 1, w);
                if (!ok) break;
                uint8_t* st = smem + s * Cfg::STAGE_BYTES;
                mbar_arrive_expect_tx(&full[s], Cfg::STAGE_BYTES);
                tma_load_2d(st + Cfg::X_BYTES, &mP, &full[s], n0, (kt0 + kt) * Cfg::KW);
                tma_load_2d(st, &mX, &full[s], (kt0 + kt) * 128, m0);
            }
        }
        // after a wait that ran out, the copies still in flight land before the CTA leaves
        for (uint32_t b = it > STAGES ? it - STAGES : 0; !ok && b < it; ++b)
            (void)mbar_wait(&full[b % STAGES], (b / STAGES) & 1, -1);
      } else if (warp == D8_PROD_WARP + 2) {
        // ---------------- scales and zero points, four groups to a unit, by asynchronous copies of
        // 16 and 4 bytes a lane; a unit is handed over when it has landed, D8_LAG units later, so
        // that the copies overlap
        const long long zwords = ((long long)p.N * BITS + 31) / 32;
        const int groups = p.spt ? nseg : 1;
        uint32_t it = 0, done = 0;
        bool ok = true;
        auto hand_over = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[done % D8_PST]);
            ++done;
        };
        for (int w = first; w < p.tiles && ok; w += step) {
            const int n = (w % p.tiles_n) * 128 + 8 * lane;
            const long long zk = (long long)(w % p.tiles_n) * (4 * BITS) + lane;
            const uint32_t s_bytes = lane < 16 && n < p.N ? 16 : 0, z_bytes = zk < zwords ? 4 : 0;
            const long long g0 = p.spt ? (long long)kt0 * p.spt : 0;
            const __half* sp = p.scales + g0 * p.N + (s_bytes ? n : 0);
            const int32_t* zp = p.qzeros + g0 * zwords + (z_bytes ? zk : 0);
            const bool zlane = p.qzeros != nullptr && lane < 4 * BITS;
            for (int g = 0; g < groups; g += 4, ++it) {
                ok = warp_wait(w, &pempty[it % D8_PST], ((it / D8_PST) & 1) ^ 1);
                if (!ok) break;
                const uint32_t dst = smem_u32(par + (it % D8_PST) * (D8_PAR_S + D8_PAR_Z));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (g + q < groups) {
                        if (lane < 16) cp_async_zfill<16>(dst + 256 * q + 16 * lane, sp, s_bytes);
                        if (zlane) cp_async_zfill<4>(dst + D8_PAR_S + 64 * q + 4 * lane, zp, z_bytes);
                        sp += p.N;
                        zp += zwords;
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (it >= D8_LAG) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(D8_LAG) : "memory");
                    hand_over();
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        while (done < it) hand_over();
      } else if (warp == D8_PROD_WARP + 1) {
        // ---------------- MMA issuer: the whole warp waits, one elected lane issues
        constexpr uint32_t idesc = make_idesc(0u, 128, TT);   // e4m3 x e4m3 -> fp32
        const bool lead = elect_one();
        uint32_t it = 0, buf = 0, dph = 1, unit = 0;
        bool ok = true;
        // One K tile: MM = MMAs (32 columns each) per segment.  A segment of every group opens
        // and closes within the tile; with one group per row it spans D8_SEG_TILES tiles.
        // The barriers are tried together and every descriptor is a constant away from the
        // stage's, as each wait or chain of address arithmetic costs the issuer about 100 clocks.
        auto issue = [&](auto mm, uint32_t s, uint32_t a, int segs, bool open, bool close, int w) {
            constexpr int MM = decltype(mm)::value;
            const uint64_t xdesc = desc_sw128_kmajor(smem_u32(smem + s * Cfg::STAGE_BYTES));
            const uint32_t at = a_ring + D8_A_COLS * a;
#pragma unroll
            for (int sg = 0; sg < 4 / MM; ++sg) {
                if (sg >= segs) break;
                // the converters' arrival on conv follows their own wait for the stage's TMA
                // copies, X8 included
                if (!warp_wait(w, &conv[a], (it / D8_AST) & 1, sg == 0, &dempty[buf], dph, open, &dempty[buf], dph,
                               false))
                    return false;
                tc_fence_after();
                if (lead) {
                    const uint32_t d = tmem + buf * TT;
#pragma unroll
                    for (int j = 0; j < MM; ++j)
                        umma_e4m3_ta(d, at + 8 * (sg * MM + j), xdesc + (uint64_t)(2 * (sg * MM + j)), idesc,
                                     j > 0 ? 1u : open ? 0u : 1u);
                    if (close) umma_commit(&dfull[buf]);
                }
                if (lead && sg == segs - 1) {
                    umma_commit(&empty[s]);
                    umma_commit(&aempty[a]);
                }
                if (close && ++buf == ND) {
                    buf = 0;
                    dph ^= 1;
                }
            }
            return true;
        };
        for (int w = first; w < p.tiles && ok; w += step) {
            for (int kt = 0; kt < nkt && ok; ++kt, ++it) {
                const uint32_t s = it % STAGES, a = it % D8_AST;
                if (p.spt <= 1) {
                    const bool open = p.spt || kt % D8_SEG_TILES == 0;
                    const bool close = p.spt || kt % D8_SEG_TILES == D8_SEG_TILES - 1 || kt == nkt - 1;
                    ok = issue(std::integral_constant<int, 4>{}, s, a, 1, open, close, w);
                } else {
                    const int segs = min(p.spt, nseg - kt * p.spt);
                    ok = p.spt == 2 ? issue(std::integral_constant<int, 2>{}, s, a, segs, true, true, w)
                                    : issue(std::integral_constant<int, 1>{}, s, a, segs, true, true, w);
                }
                // the products of a unit's last K tile come after its zero points were read
                if (kt == nkt - 1 || (p.spt && ((kt + 1) * p.spt & 3) == 0)) {
                    if (lead && ok) umma_commit(&pempty[unit % D8_PST]);
                    ++unit;
                }
            }
        }
    }
    }
    __syncwarp();
    if (p.split > 1 && (warp < D8_EPI_WARP0 || warp >= D8_PROD_WARP)) {
        cluster_sync_all();   // these warps' part in the epilogue's cluster barriers
        cluster_sync_all();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace gq

namespace gqh {

// Tensor maps are encoded anew on every call: a shared cache would tie concurrent callers together.
static bool tmap_2d(CUtensorMap* map, const void* base, CUtensorMapDataType type, int elem_bytes, uint64_t rows,
                    uint64_t cols, uint32_t box_rows, uint32_t box_cols, bool swizzle) {
    static KeepFound<PFN_cuTensorMapEncodeTiled_v12000> found;
    const auto encode = found.get([] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (!encode) return false;
    cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * (uint64_t)elem_bytes};
    cuuint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
    return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The setmaxnreg split relies on the registers that the kernel was launched with: with fewer it would wait
// forever, so such a build is refused.
template <auto Kernel>
static cudaError_t d8_registers_fit() {
    static KeepFound<int> found;
    cudaError_t e = cudaSuccess;
    const int regs = found.get([&e] {
        cudaFuncAttributes at = {};
        e = cudaFuncGetAttributes(&at, reinterpret_cast<const void*>(Kernel));
        return e == cudaSuccess ? at.numRegs : 0;
    });
    if (regs == 0) {
        (void)cudaGetLastError();   // a failed query must not leak into later checks
        return e;
    }
    return regs >= gq::D8_REGS ? cudaSuccess : cudaErrorInvalidKernelImage;
}

int num_sms();

template <int BITS, int TT>
cudaError_t dq_gemm_e4m3_launch(const uint8_t* X8, const int32_t* qweight, gq::D8Args p, cudaStream_t st) {
    using Cfg = gq::D8Cfg<BITS, TT>;
    CUtensorMap mx, mp;
    if (!tmap_2d(&mx, X8, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)p.M, (uint64_t)p.K, TT, 128, true) ||
        !tmap_2d(&mp, qweight, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, (uint64_t)((long long)p.K * BITS / 32),
                 (uint64_t)p.N, Cfg::KW, 128, false))
        return cudaErrorInvalidValue;
    constexpr auto kern = gq::dq_gemm_e4m3_kernel<BITS, TT>;
    GQ_TRY((d8_registers_fit<kern>()));
    GQ_TRY((smem_attr_once<kern, Cfg::SMEM>()));
    p.tiles_n = (p.N + 127) / 128;
    const long long tiles = (long long)p.tiles_n * ((p.M + TT - 1) / TT);
    if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.tiles = (int)tiles;
    // K is split where the tiles leave half of the SMs idle, at two K tiles per CTA at least
    p.split = 1;
    while (p.split < 8 && tiles * p.split * 2 <= num_sms() && (p.K + 127) / 128 >= 4 * p.split) p.split *= 2;
    TimedScope ts__("dequant_gemm_e4m3", st);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : std::min<long long>(tiles, num_sms())));
    cfg.blockDim = dim3(gq::D8_THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mx, mp, p);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

// Up to 64 tokens a tile of 64: 64 x 4096 x 4096 takes 11.0 us, 128 tokens in a tile of 128 13.3 us.
template <int BITS>
cudaError_t dq_gemm_e4m3_run(const uint8_t* X8, const int32_t* qweight, const gq::D8Args& p, cudaStream_t st) {
    if (p.M <= 64) return dq_gemm_e4m3_launch<BITS, 64>(X8, qweight, p, st);
    return dq_gemm_e4m3_launch<BITS, 128>(X8, qweight, p, st);
}

}  // namespace gqh
