// Dequantizing GEMM on e4m3 activations:
//
//   Y[m, n] = xs[m] sum_g s_g[n] P_g[n, m],   P_g[n, m] = sum_{k in g} (q[n, k] - z_g[n]) X8[m, k]
//
// q - z of 2, 3 and 4 bits lies in [-15, 15] and is exact in e4m3, so P_g is formed by the 8-bit
// tensor instructions (twice the bf16 rate) from exact products with fp32 accumulation; s_g and
// xs are applied in fp32.  No rounded copy of W_hat is made.
//
// The weights are the A operand (128 rows n of a tile) and sit in tensor memory: a converter
// thread owns one row, turns its packed codes into e4m3 bytes and stores them with one
// tcgen05.st, so shared memory carries only X8 (the B operand) and the packed words.  With rows
// on the lanes, a group's scale is one register of an epilogue thread.
//
// A tile is 128 rows x TT tokens, K advances by 128.  One CTA per SM, 16 warps:
//   warp 0       TMA: X8 tile (TT tokens x 128 bytes, 128-byte swizzle) and packed words
//                (4 BITS words x 128 rows) into a ring of stages;
//   warp 1       MMA issuer: per quantization group one accumulator segment for each half of
//                up to 128 tokens, in a ring of three accumulators of tensor memory;
//   warps 4-7    converters, one thread per row, a ring of four A operands of 32 columns;
//   warps 8-15   epilogue: two warps per lane quadrant, TT / 2 tokens each, running sums in
//                registers: y += s_g P_g, two at a time.
// Warps 8-15 take the registers that the others give up (setmaxnreg: 56 + 88 + 2 x 184 of
// 4 x 128).  Every wait is bounded (GPTQ_ERR_TIMEOUT).  No TMA multicast.
//
// Codes to e4m3: the values q - z of one group and row are a table of 2^BITS bytes in registers
// that byte permutes index with the codes themselves: two lookups by the low three bits and a
// third permute that picks by bit 3 for 4 bits, one lookup for 2 and 3 bits.
//
// Few tiles: the K range is split over a cluster of S CTAs, whose partial sums are joined
// through distributed shared memory in rank order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "pack.cuh"

namespace gq {

constexpr int D8_THREADS = 512;
constexpr int D8_AST = 4, D8_ND = 3;
constexpr int D8_SEG_TILES = 4;   // K tiles per segment for one group per row: 16 MMAs in place

template <int BITS, int TT>
struct D8Cfg {
    static constexpr int KW = 4 * BITS;               // packed words per row and K tile
    static constexpr int X_BYTES = TT * 128;
    static constexpr int P_BYTES = KW * 128 * 4;
    static constexpr int STAGE_BYTES = X_BYTES + P_BYTES;
    static constexpr int FIT = (220 * 1024) / STAGE_BYTES;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int H = TT == 256 ? 2 : 1;       // accumulators per segment
    static constexpr int DW = TT / H;                 // tokens per accumulator
    static constexpr int C = TT / 2;                  // tokens per epilogue warp
    static constexpr int A_COL = D8_ND * 128;         // A ring behind the accumulators
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 256 + 4 * TT + 512;
    static_assert(STAGE_BYTES % 1024 == 0, "the swizzled tiles stay 1024-byte aligned");
    static_assert(TT * 128 * 4 <= STAGES * STAGE_BYTES, "partial sums fit the ring");
};

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

__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t s) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(s));
    return r;
}
// Eight BITS-wide codes in the low 8 BITS bits of v, one per nibble.
template <int BITS>
__device__ __forceinline__ uint32_t codes_to_nibbles(uint32_t v) {
    if constexpr (BITS == 2) {
        v = (v | (v << 8)) & 0x00FF00FFu;
        v = (v | (v << 4)) & 0x0F0F0F0Fu;
        v = (v | (v << 2)) & 0x33333333u;
    } else if constexpr (BITS == 3) {
        v = (v & 0x00000FFFu) | ((v & 0x00FFF000u) << 4);
        v = (v & 0x003F003Fu) | ((v & 0x0FC00FC0u) << 2);
        v = (v & 0x07070707u) | ((v & 0x38383838u) << 1);
    }
    return v;
}
// Table bytes of eight nibble codes, in order.
template <int BITS>
__device__ __forceinline__ void table_bytes(uint32_t nib, const uint4& t, uint32_t& b0, uint32_t& b1) {
    if constexpr (BITS == 4) {
        const uint32_t m = nib & 0x77777777u, k = ((nib >> 1) & 0x44444444u) | 0x32103210u;
        b0 = byte_perm(byte_perm(t.x, t.y, m), byte_perm(t.z, t.w, m), k);
        b1 = byte_perm(byte_perm(t.x, t.y, m >> 16), byte_perm(t.z, t.w, m >> 16), k >> 16);
    } else {
        b0 = byte_perm(t.x, t.y, nib);
        b1 = byte_perm(t.x, t.y, nib >> 16);
    }
}
// The 32 codes of BITS words as 8 words of table bytes.
template <int BITS>
__device__ __forceinline__ void table_bytes_32(const uint32_t (&w)[BITS], const uint4& t, uint32_t* out) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t v;
        if constexpr (BITS == 4)
            v = w[c];
        else if constexpr (BITS == 2)
            v = (w[c >> 1] >> (16 * (c & 1))) & 0xFFFFu;
        else
            v = (c == 0 ? w[0] : c == 3 ? w[2] >> 8 : __funnelshift_r(w[c - 1], w[c], c == 1 ? 24 : 16)) & 0xFFFFFFu;
        table_bytes<BITS>(codes_to_nibbles<BITS>(v), t, out[2 * c], out[2 * c + 1]);
    }
}

__device__ __forceinline__ void fma2(float2& acc, float s, uint32_t a, uint32_t b) {
    asm("{\n\t.reg .b64 s, v, c;\n\t"
        "mov.b64 s, {%2, %2};\n\tmov.b64 v, {%3, %4};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, s, v, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(acc.x), "+f"(acc.y)
        : "f"(s), "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
        : "=f"(v)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

__device__ __forceinline__ void store_y(void* Y, int bf16, long long at, float y) {
    if (bf16)
        reinterpret_cast<__nv_bfloat16*>(Y)[at] = __float2bfloat16_rn(y);
    else
        reinterpret_cast<float*>(Y)[at] = y;
}

template <int BITS, int TT>
__global__ void __launch_bounds__(D8_THREADS, 1)
    dq_gemm_e4m3_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mP, const D8Args p) {
    using Cfg = D8Cfg<BITS, TT>;
    constexpr int STAGES = Cfg::STAGES, H = Cfg::H, DW = Cfg::DW, C = Cfg::C;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint4* lut = reinterpret_cast<uint4*>(smem + STAGES * Cfg::STAGE_BYTES);   // [16] table of each zero point
    float* xs = reinterpret_cast<float*>(lut + 16);                            // [TT] scales of the tile's tokens
    uint64_t* full = reinterpret_cast<uint64_t*>(xs + TT);   // [STAGES] TMA landed
    uint64_t* empty = full + STAGES;                         // [STAGES] MMAs of the stage done
    uint64_t* conv = empty + STAGES;                         // [AST] A operand written
    uint64_t* aempty = conv + D8_AST;                        // [AST] A operand read
    uint64_t* dfull = aempty + D8_AST;                       // [ND] segment complete
    uint64_t* dempty = dfull + D8_ND;                        // [ND] segment drained
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dempty + D8_ND);

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
        for (int s = 0; s < D8_ND; ++s) {
            mbar_init(&dfull[s], 1);
            mbar_init(&dempty[s], 8 / H);
        }
        fence_mbar_init();
    }
    if (threadIdx.x < 256) {   // byte c of table z: e4m3(c - z)
        const int z = threadIdx.x >> 4, c = threadIdx.x & 15;
        reinterpret_cast<uint8_t*>(lut)[threadIdx.x] =
            (uint8_t)__nv_cvt_float_to_fp8((float)(c - z), __NV_SATFINITE, __NV_E4M3);
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
    pdl_wait();

    // K tiles of this CTA, and the segments in them
    const int rank = p.split > 1 ? (int)cluster_rank() : 0;
    const int nkt_all = (p.K + 127) / 128;
    const int kt0 = (int)((long long)nkt_all * rank / p.split);
    const int kt1 = (int)((long long)nkt_all * (rank + 1) / p.split);
    const int nkt = kt1 - kt0;
    const int step = (int)gridDim.x / p.split, first = (int)blockIdx.x / p.split;
    // the last K tile may hold fewer groups than spt
    const int nseg = p.spt ? min(kt1 * p.spt, p.K / (128 / p.spt)) - kt0 * p.spt
                           : (nkt + D8_SEG_TILES - 1) / D8_SEG_TILES;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0 && lane == 0) {
            // ---------------- TMA producer
            prefetch_tmap(&mX);
            prefetch_tmap(&mP);
            uint32_t it = 0;
            bool ok = true;
            for (int w = first; w < p.tiles && ok; w += step) {
                const int n0 = (w % p.tiles_n) * 128, m0 = (w / p.tiles_n) * TT;
                for (int kt = kt0; kt < kt1; ++kt, ++it) {
                    const uint32_t s = it % STAGES;
                    if (!mbar_wait(&empty[s], ((it / STAGES) & 1) ^ 1, w)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = smem + s * Cfg::STAGE_BYTES;
                    mbar_arrive_expect_tx(&full[s], Cfg::STAGE_BYTES);
                    tma_load_2d(st + Cfg::X_BYTES, &mP, &full[s], n0, kt * Cfg::KW);
                    tma_load_2d(st, &mX, &full[s], kt * 128, m0);
                }
            }
            // after a wait that ran out, the copies still in flight land before the CTA leaves
            for (uint32_t b = it > STAGES ? it - STAGES : 0; !ok && b < it; ++b)
                (void)mbar_wait(&full[b % STAGES], (b / STAGES) & 1, -1);
        } else if (warp == 1 && lane == 0) {
            // ---------------- MMA issuer
            constexpr uint32_t idesc = make_idesc(0u, 128, DW);   // e4m3 x e4m3 -> fp32
            uint32_t it = 0, seg = 0;
            bool ok = true;
            for (int w = first; w < p.tiles && ok; w += step) {
                for (int kt = 0; kt < nkt && ok; ++kt, ++it) {
                    const uint32_t s = it % STAGES, a = it % D8_AST;
                    if (!mbar_wait(&full[s], (it / STAGES) & 1, w) || !mbar_wait(&conv[a], (it / D8_AST) & 1, w)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t xb = smem_u32(smem + s * Cfg::STAGE_BYTES);
                    const uint32_t at = tmem + Cfg::A_COL + 32 * a;
                    const int segs = p.spt ? min(p.spt, nseg - kt * p.spt) : 1;
                    const int mmas = p.spt ? 4 / p.spt : 4;
                    const bool open = p.spt || kt % D8_SEG_TILES == 0;
                    const bool close = p.spt || kt % D8_SEG_TILES == D8_SEG_TILES - 1 || kt == nkt - 1;
                    for (int sg = 0; sg < segs && ok; ++sg) {
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            const uint32_t dc = seg * H + h, buf = dc % D8_ND;
                            if (open) {
                                if (!mbar_wait(&dempty[buf], ((dc / D8_ND) & 1) ^ 1, w)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                            }
                            for (int j = 0; j < mmas; ++j) {
                                const int kk = sg * mmas + j;   // which 32 columns of the K tile
                                umma_e4m3_ta(tmem + buf * 128, at + 8 * kk,
                                             desc_sw128_kmajor(xb + h * (DW * 128) + 32 * kk), idesc,
                                             (open && j == 0) ? 0u : 1u);
                            }
                            if (close) umma_commit(&dfull[buf]);
                        }
                        if (close) ++seg;
                    }
                    umma_commit(&empty[s]);
                    umma_commit(&aempty[a]);
                }
            }
        }
    } else if (warp < 8) {
        // ---------------- converters: thread t owns row n0 + t
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        const int t = threadIdx.x - 128, qd = warp & 3;
        const long long zwords = ((long long)p.N * BITS + 31) / 32;
        const int qps = p.spt ? 4 / p.spt : 4;    // 32-column quarters per table
        uint32_t it = 0;
        bool ok = true;
        for (int w = first; w < p.tiles && ok; w += step) {
            const int n = (w % p.tiles_n) * 128 + t;
            const bool live = p.qzeros != nullptr && n < p.N;
            int z[4], zn[4];
            // zero points of a K tile, fetched one tile ahead
            auto fetch = [&](int kt, int (&zz)[4]) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    zz[q] = 1 << (BITS - 1);
                    const int gi = p.spt ? kt * p.spt + q / qps : 0;
                    if (live && q % qps == 0 && (p.spt == 0 || gi * (128 / p.spt) < p.K))
                        zz[q] = (int)stream_code(p.qzeros + gi * zwords, 1, n, BITS);
                }
            };
            fetch(kt0, zn);
            for (int kt = kt0; kt < kt1; ++kt, ++it) {
                const uint32_t s = it % STAGES, a = it % D8_AST;
#pragma unroll
                for (int q = 0; q < 4; ++q) z[q] = zn[q];
                if (p.spt && kt + 1 < kt1) fetch(kt + 1, zn);
                if (!mbar_wait(&full[s], (it / STAGES) & 1, w) ||
                    !mbar_wait(&aempty[a], ((it / D8_AST) & 1) ^ 1, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t* col = reinterpret_cast<const uint32_t*>(smem + s * Cfg::STAGE_BYTES + Cfg::X_BYTES) + t;
                uint32_t r[32];
                uint4 tab = lut[z[0]];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t words[BITS];
#pragma unroll
                    for (int i = 0; i < BITS; ++i) words[i] = col[(q * BITS + i) * 128];
                    if (q > 0 && q % qps == 0) tab = lut[z[q]];
                    table_bytes_32<BITS>(words, tab, r + 8 * q);
                }
                tmem_st_32x32b_x32(tmem + Cfg::A_COL + 32 * a + ((uint32_t)(32 * qd) << 16), r);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&conv[a]);
            }
        }
    } else {
        // ---------------- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int ew = warp - 8, qd = warp & 3, half = ew >> 2;
        const uint32_t lane_off = (uint32_t)(32 * qd) << 16;
        const uint32_t col0 = H == 2 ? 0 : (uint32_t)(half * C);   // columns of the accumulator
        const int et = threadIdx.x - 256;
        uint32_t seg = 0;
        bool ok = true;   // once false, the loop goes on without waiting: its barriers need every warp
        for (int w = first; w < p.tiles; w += step) {
            const int n = (w % p.tiles_n) * 128 + 32 * qd + lane, m0 = (w / p.tiles_n) * TT;
            asm volatile("bar.sync 1, 256;" ::: "memory");   // the previous tile's scales are read
            if (et < TT) xs[et] = m0 + et < p.M ? p.x_scale[m0 + et] : 0.f;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            float2 acc[C / 2];
#pragma unroll
            for (int j = 0; j < C / 2; ++j) acc[j] = make_float2(0.f, 0.f);
            const long long g0 = p.spt ? (long long)kt0 * p.spt : 0;
            const __half* sp = p.scales + g0 * p.N + n;
            float s_next = n < p.N ? __half2float(sp[0]) : 0.f;
            for (int sg = 0; sg < nseg && ok; ++sg, ++seg) {
                const float s = s_next;
                if (p.spt && sg + 1 < nseg && n < p.N) {
                    sp += p.N;
                    s_next = __half2float(*sp);
                }
                const uint32_t dc = H == 2 ? seg * 2 + half : seg, buf = dc % D8_ND;
                ok = mbar_wait(&dfull[buf], (dc / D8_ND) & 1, w);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < C / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tmem + buf * 128 + col0 + 32 * c + lane_off, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) fma2(acc[16 * c + j], s, r[2 * j], r[2 * j + 1]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&dempty[buf]);
            }
            const int j0 = half * C;   // this warp's first token of the tile
            if (p.split == 1) {
                if (ok && n < p.N) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (m0 + j0 + j < p.M)
                            store_y(p.Y, p.y_bf16, (long long)(m0 + j0 + j) * p.N + n,
                                    ((j & 1) ? acc[j / 2].y : acc[j / 2].x) * xs[j0 + j]);
                }
            } else {
                // One tile per cluster.  The partial sums take the ring's place once the last MMAs
                // have read it (a segment of one half completes before those of the other).
                float* red = reinterpret_cast<float*>(smem);   // [TT][128]
                if (ok) ok = mbar_wait(&empty[(nkt - 1) % STAGES], ((nkt - 1) / STAGES) & 1, w);
                if (ok) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        red[(j0 + j) * 128 + 32 * qd + lane] = (j & 1) ? acc[j / 2].y : acc[j / 2].x;
                }
                cluster_sync_all();
                // rank r finishes the tokens r, r + split, ...
                const int c = et & 127, nn = (w % p.tiles_n) * 128 + c;
                for (int j = rank + p.split * (et >> 7); j < TT; j += 2 * p.split) {
                    if (m0 + j < p.M && nn < p.N) {
                        float y = 0.f;
                        for (int r = 0; r < p.split; ++r)
                            y += ld_cluster_f32(smem_u32(red + j * 128 + c), (uint32_t)r);
                        store_y(p.Y, p.y_bf16, (long long)(m0 + j) * p.N + nn, y * xs[j]);
                    }
                }
                cluster_sync_all();   // no CTA leaves while its partial sums are being read
            }
        }
    }
    __syncwarp();
    if (warp < 8 && p.split > 1) {   // the other warps' part in the epilogue's cluster barriers
        cluster_sync_all();
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
inline bool tmap_2d(CUtensorMap* map, const void* base, CUtensorMapDataType type, int elem_bytes, uint64_t rows,
                    uint64_t cols, uint32_t box_rows, uint32_t box_cols, bool swizzle) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode) return false;
    cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * (uint64_t)elem_bytes};
    cuuint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
    return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// MaxDynamicSharedMemorySize of one kernel, set once per device; safe from several threads (the
// attribute is set again if two race, which changes nothing).
template <auto Kernel, int BYTES>
cudaError_t smem_attr_once() {
    static std::atomic<bool> done[128];
    int dev = 0;
    GQ_TRY(cudaGetDevice(&dev));
    if (dev < 128 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    GQ_TRY(cudaFuncSetAttribute(reinterpret_cast<const void*>(Kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                BYTES));
    if (dev < 128) done[dev].store(true, std::memory_order_release);
    return cudaSuccess;
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

template <int BITS>
cudaError_t dq_gemm_e4m3_run(const uint8_t* X8, const int32_t* qweight, const gq::D8Args& p, cudaStream_t st) {
    if (p.M <= 64) return dq_gemm_e4m3_launch<BITS, 64>(X8, qweight, p, st);
    if (p.M <= 128) return dq_gemm_e4m3_launch<BITS, 128>(X8, qweight, p, st);
    return dq_gemm_e4m3_launch<BITS, 256>(X8, qweight, p, st);
}

}  // namespace gqh
