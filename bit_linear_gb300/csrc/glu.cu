// Gated feed-forward layer on ternary weights: both projections, the activation and the product.
//
//   g | u = scale (X T), T = ternary weight [K][2N], the gate's columns first
//   H     = act(g) u
//   dY    = dH u act'(g) | dH act(g)      the dY [M][2N] that tern_linear_bwd takes for the same weight
//
// Many rows: one persistent tcgen05 GEMM whose tile holds the gate's and the value's columns of the same
// HN outputs side by side (accumulator columns 0..HN-1 and HN..2HN-1), so that the epilogue has both
// and g, u never reach memory.  A pair of CTAs (256 rows) splits the B operand the same way: the
// leader copies the gate's columns, its peer the value's.  Operands as in the ternary forward: X
// (K-major) and the bf16 plane T (MN-major), by TMA with the 128-byte swizzle; products with -1, 0
// and 1 are exact and sums fp32.  The epilogue rounds H once.  For training it also stores the
// factors u act'(g) | act(g) as bf16, which leaves the gradient a product: that costs a second
// rounding (2^-8 at most each) and four bytes an element, where g and u in fp32 would cost eight and
// recomputing them the whole GEMM again.  The gradient without stored factors is that: the same
// GEMM, with dH read and dY written in the epilogue, rounded once.
//
// A few rows (single tokens): the 2-bit codes are read, an eighth of T's bytes.  See glu_codes below.
//
// 32768 x 4096 x 6144 (3.3 TFLOP): 1.64 ms, 2010 TFLOP/s, above cuBLAS's measured burst; with the factors stored
// 1.75 ms, and the product with dH 0.30 ms (0.92 of the copy rate).  8192 x 512 x 1360: 24 us, with factors 29, the
// gradient recomputed 35, where the products alone would take 12: eight of it before and after the tiles (no
// launch overlaps another), then 4.6 rounds of tiles in five whose epilogue (stores of 32 bytes a lane, rows 2 N
// apart) takes longer than their 512-deep products.  Copying dH ahead of the products changed nothing.
#include <algorithm>
#include <cmath>
#include <mutex>

#include <cuda_bf16.h>

#include "mma.cuh"
#include "pairs.cuh"
#include "rows.cuh"

namespace tern {

__device__ int g_glu_status;

namespace {

constexpr int kBM = 128;   // rows of X per CTA

__device__ __forceinline__ float pow2(float x) {   // 2^x, from the special function unit
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ F2 each(F2 x, float (*f)(float)) {
    float a, b;
    split(x, a, b);
    return pair(f(a), f(b));
}
__device__ __forceinline__ float magnitude(float x) { return fabsf(x); }
__device__ __forceinline__ float positive(float x) { return x < 0.f ? 0.f : x; }   // NaN passes
__device__ __forceinline__ float bounded(float x) {                               // by 127; NaN passes
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(127.f));
    return y;
}

// act(g) and, with D, act'(g), of two neighbours.  The special functions' errors (2^-22 relative each) are
// far below the outputs' rounding to bf16.  So is GELU's approximation but for its lower tail, where it is
// relative to Phi 1.6e-3 at g = -5, 3.6e-3 at -6 (the rounding's 2^-8 from there on) and 1e-2 at -8, of
// values below 1e-8; 1 + erf in fp32 has nothing left there.
template <int ACT, bool D>
__device__ __forceinline__ void activate(F2 g, F2& a, F2& d) {
    if constexpr (ACT == TERN_ACT_RELU2) {
        const F2 r = each(g, positive);
        a = mul2(r, r);
        if (D) d = add2(r, r);
    } else if constexpr (ACT == TERN_ACT_GELU) {
        // g Phi(g): the upper tail's approximation by Hastings (Abramowitz and Stegun 7.1.26, 1.5e-7
        // absolute in erf), whose exponential the density shares
        const F2 z = each(g, magnitude);
        const F2 t = each(fma2(z, both(0.3275911f * 0.70710678f), both(1.f)), reciprocal);
        const F2 e = each(mul2(mul2(g, g), both(-0.72134752f)), pow2);   // exp(-g^2 / 2)
        F2 p = fma2(both(0.5f * 1.061405429f), t, both(0.5f * -1.453152027f));
        p = fma2(p, t, both(0.5f * 1.421413741f));
        p = fma2(p, t, both(0.5f * -0.284496736f));
        p = fma2(p, t, both(0.5f * 0.254829592f));
        const F2 tail = mul2(mul2(p, t), e), rest = fma2(tail, both(-1.f), both(1.f));   // Phi(-|g|), Phi(|g|)
        float t0, t1, r0, r1, g0, g1;
        split(tail, t0, t1);
        split(rest, r0, r1);
        split(g, g0, g1);
        const F2 cdf = pair(g0 < 0.f ? t0 : r0, g1 < 0.f ? t1 : r1);
        a = mul2(g, cdf);
        if (D) d = fma2(mul2(g, both(0.39894228f)), e, cdf);
    } else {
        // s = 1 / (1 + e) and its complement e / (1 + e); e = exp(-g) kept finite.  At its bound s is 0 (the
        // reciprocal, 2^-127, is flushed), so that no gate, however far, leaves a product with it.
        const F2 e = each(each(mul2(g, both(-1.44269504f)), bounded), pow2);
        const F2 s = each(add2(e, both(1.f)), reciprocal), c = mul2(e, s);
        if constexpr (ACT == TERN_ACT_SIGMOID) {
            a = s;
            if (D) d = mul2(s, c);
        } else {
            a = mul2(g, s);
            if (D) d = fma2(a, c, s);
        }
    }
}

struct GluArgs {
    CUtensorMap mX, mT;
    const float* scale;     // [2N]
    const uint16_t* dH;     // [M][N]: the gradient is computed; else H
    uint16_t* H;            // [M][N]
    uint16_t* pair;         // [M][2N]: the factors (with H; may be null), or dY (with dH)
    int M, N, K, act;
    int tiles_m, tiles_n, num_kb;
    bool whole;             // H and pair are 32-byte aligned
};

// CG CTAs share a tile of 128 CG rows by HN outputs: 2 HN accumulator columns.
template <int CG_, int HN_, int STAGES_>
struct GluCfg {
    static constexpr int CG = CG_, HN = HN_, STAGES = STAGES_, BK = 64, BN = 2 * HN;
    static constexpr int TILE_M = kBM * CG;
    static constexpr int B_COLS = BN / CG;
    static constexpr int A_BYTES = kBM * BK * 2, B_BYTES = B_COLS * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int RASTER = 16 / CG;      // as in the ternary forward
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int EPI_WARPS = 16, THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 256;
    static_assert(TMEM_COLS == 256 || TMEM_COLS == 512, "TMEM allocation must be a power of two");
    static_assert(SMEM_BYTES <= 232448 && B_COLS % 64 == 0, "stage");
};

__device__ __forceinline__ bool glu_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, bool watch) {
    return wait_limited(bar, parity, abort_flag, watch, kWaitLimitNs, [] { atomicExch(&g_glu_status, 1); });
}

// A lane's 16 bf16 of a row, 32 bytes: one access where rows are aligned to that (`whole`).
__device__ __forceinline__ void store_row(uint16_t* to, const uint32_t (&w)[8], bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                     "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(F2 x) {
    float a, b;
    split(x, a, b);
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// 16 outputs of a lane's row, columns c0..c0+15, from the accumulators at TMEM columns tg (the gate's)
// and tu (the value's): H, or H and the factors, or dY.
template <int ACT, bool BACK, bool TWO>
__device__ __forceinline__ void glu_chunk(const GluArgs& a, uint32_t tg, uint32_t tu, int wrow, int c0, int lane) {
    const int64_t row = wrow + lane;
    const bool in = row < a.M;
    uint32_t h[8], p[8], q[8];
    uint32_t rg[16], ru[16];
    ptx::tmem_ld_32x32b_x16(tg, rg);
    ptx::tmem_ld_32x32b_x16(tu, ru);
    Raw<__nv_bfloat16, 16> dh;
    if (BACK) dh = load_raw<__nv_bfloat16, 16>(reinterpret_cast<const __nv_bfloat16*>(a.dH) + (in ? row : wrow) * a.N + c0);
    const float4* pg = reinterpret_cast<const float4*>(a.scale + c0);
    const float4* pu = reinterpret_cast<const float4*>(a.scale + a.N + c0);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int b = 0; b < 4; ++b) {   // four columns
        const float4 sg = __ldg(pg + b), su = __ldg(pu + b);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = 2 * b + i;   // two of them
            const F2 g = mul2(pair(__uint_as_float(rg[2 * o]), __uint_as_float(rg[2 * o + 1])), i ? pair(sg.z, sg.w) : pair(sg.x, sg.y));
            const F2 u = mul2(pair(__uint_as_float(ru[2 * o]), __uint_as_float(ru[2 * o + 1])), i ? pair(su.z, su.w) : pair(su.x, su.y));
            F2 f, d;
            activate<ACT, TWO>(g, f, d);
            if constexpr (!BACK) h[o] = pack_bf16(mul2(f, u));
            if constexpr (TWO) {
                d = mul2(d, u);
                if constexpr (BACK) {
                    const F2 x = pair(raw_at<__nv_bfloat16, 16>(dh, 2 * o), raw_at<__nv_bfloat16, 16>(dh, 2 * o + 1));
                    d = mul2(d, x);
                    f = mul2(f, x);
                }
                p[o] = pack_bf16(d);
                q[o] = pack_bf16(f);
            }
        }
    }
    if (!in) return;
    if constexpr (!BACK) store_row(a.H + row * a.N + c0, h, a.whole);
    if constexpr (TWO) {
        uint16_t* to = a.pair + row * 2 * a.N + c0;
        store_row(to, p, a.whole);
        store_row(to + a.N, q, a.whole);
    }
}

template <bool BACK, bool TWO>
__device__ __forceinline__ void glu_act(const GluArgs& a, uint32_t tg, uint32_t tu, int wrow, int c0, int lane) {
    switch (a.act) {
    case TERN_ACT_SILU: glu_chunk<TERN_ACT_SILU, BACK, TWO>(a, tg, tu, wrow, c0, lane); break;
    case TERN_ACT_GELU: glu_chunk<TERN_ACT_GELU, BACK, TWO>(a, tg, tu, wrow, c0, lane); break;
    case TERN_ACT_RELU2: glu_chunk<TERN_ACT_RELU2, BACK, TWO>(a, tg, tu, wrow, c0, lane); break;
    default: glu_chunk<TERN_ACT_SIGMOID, BACK, TWO>(a, tg, tu, wrow, c0, lane); break;
    }
}

// Roles as in the ternary forward: warp 0 copies, warp 1 allocates TMEM and (in the leader) issues the
// MMAs, warps 2-17 are the epilogue, four for each 32 rows (with two, the epilogue's latencies showed
// where K is small: 8192 x 512 x 1360 with gelu 31 us, its gradient 40).  Two accumulators, so that a tile's
// epilogue runs beside the next tile's products.
template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) tern_glu_gemm(const __grid_constant__ GluArgs a) {
    constexpr int CG = C::CG;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + (base - raw) + C::STAGES * C::STAGE_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t FULL0 = ptx::smem_u32(bars), EMPTY0 = FULL0 + 8u * C::STAGES;
    const uint32_t TFULL0 = FULL0 + 16u * C::STAGES, TEMPTY0 = TFULL0 + 16u, DRAIN = TFULL0 + 32u;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0u;   // 0 = leader of the pair
    const int unit = static_cast<int>(blockIdx.x) / CG, units = static_cast<int>(gridDim.x) / CG;
    const int total = a.tiles_m * a.tiles_n;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(FULL0 + 8u * s, 1);
            ptx::mbar_init(EMPTY0 + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(TFULL0 + 8u * b, 1);
            ptx::mbar_init(TEMPTY0 + 8u * b, C::EPI_WARPS * CG);
        }
        ptx::mbar_init(DRAIN, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before();
    if constexpr (CG == 2) ptx::cluster_sync(); else __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    ptx::pdl_trigger();   // TMEM is allocated everywhere: small kernels may follow
    ptx::pdl_wait();

    uint32_t issued = 0, issued_parity = 0;
    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ copies
        ptx::tma_prefetch_desc(&a.mX);
        ptx::tma_prefetch_desc(&a.mT);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = unit; ok && tile < total; tile += units) {
            int mt, nt;
            tile_coords<C::RASTER>(tile, a.tiles_m, a.tiles_n, mt, nt);
            const int arow = mt * C::TILE_M + static_cast<int>(rank) * kBM;
            for (int kb = 0; kb < a.num_kb; ++kb) {
                if (!glu_wait(EMPTY0 + 8u * stage, phase ^ 1u, abort_flag, true)) {
                    ok = false;
                    break;
                }
                const uint32_t full = FULL0 + 8u * stage;
                const uint32_t full_at = CG == 2 ? ptx::mapa_shared(full, 0) : full;   // a pair counts on the leader's
                const uint32_t sA = base + stage * C::STAGE_BYTES, sB = sA + C::A_BYTES;
                if (rank == 0) ptx::mbar_arrive_expect_tx(full, CG * C::STAGE_BYTES);
                auto load = [&](uint32_t dst, const CUtensorMap* m, int x, int y) {
                    if constexpr (CG == 2) ptx::tma_load_2d_pair(dst, m, x, y, full_at);
                    else ptx::tma_load_2d(dst, m, x, y, full_at);
                };
                load(sA, &a.mX, kb * C::BK, arow);
#pragma unroll
                for (int j = 0; j < C::B_COLS / 64; ++j) {
                    // column of the accumulator, the gate's below HN; N is a multiple of 16, so that x is
                    // aligned.  A last tile's columns past N are the value's first (or zeros): not stored.
                    const int c = static_cast<int>(rank) * C::B_COLS + j * 64;
                    const int x = c < C::HN ? nt * C::HN + c : a.N + nt * C::HN + c - C::HN;
                    load(sB + j * 64 * C::BK * 2, &a.mT, x, kb * C::BK);
                }
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // every stage's release has arrived before the CTA may exit
        if (ok)
            for (int s = 0; s < C::STAGES; ++s)
                if (issued & (1u << s)) glu_wait(EMPTY0 + 8u * s, (issued_parity >> s) & 1u, abort_flag, true);
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ------------------------------------------------------------ products
        constexpr uint32_t IDESC = make_idesc(C::TILE_M, C::BN, false, true);
        int stage = 0, local = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = unit; ok && tile < total; tile += units, ++local) {
            const int acc = local & 1;
            if (!glu_wait(TEMPTY0 + 8u * acc, ((local >> 1) & 1) ^ 1u, abort_flag, true)) break;
            ptx::tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * C::BN;
            for (int kb = 0; kb < a.num_kb; ++kb) {
                if (!glu_wait(FULL0 + 8u * stage, phase, abort_flag, true)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t sA = base + stage * C::STAGE_BYTES, sB = sA + C::A_BYTES;
#pragma unroll
                for (int kk = 0; kk < C::BK / 16; ++kk) {
                    const uint64_t da = op_desc<false, C::BK>(sA, kk), db = op_desc<true, C::BK>(sB, kk);
                    const uint32_t more = kb != 0 || kk != 0;
                    if constexpr (CG == 2) ptx::mma_bf16_pair(d_tmem, da, db, IDESC, more);
                    else ptx::mma_bf16(d_tmem, da, db, IDESC, more);
                }
                if constexpr (CG == 2) ptx::mma_commit_pair_mc(EMPTY0 + 8u * stage, 0x3);
                else ptx::mma_commit(EMPTY0 + 8u * stage);
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            if constexpr (CG == 2) ptx::mma_commit_pair_mc(TFULL0 + 8u * acc, 0x3);
            else ptx::mma_commit(TFULL0 + 8u * acc);
        }
        if constexpr (CG == 2) ptx::mma_commit_pair(DRAIN); else ptx::mma_commit(DRAIN);
        glu_wait(DRAIN, 0, abort_flag, false);
        if (ok && !*abort_flag) {   // the epilogues' last releases have arrived
            for (int acc = 0; acc < 2; ++acc) {
                if (local <= acc) continue;
                const int last = (local - 1) - (((local - 1) - acc) & 1);
                glu_wait(TEMPTY0 + 8u * acc, static_cast<uint32_t>(last >> 1) & 1u, abort_flag, true);
            }
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue
        const int quad = warp & 3;   // a warp may touch TMEM lanes 32 (warp % 4) .. + 31
        const uint32_t tempty_leader = CG == 2 ? ptx::mapa_shared(TEMPTY0, 0) : TEMPTY0;   // shared::cta addresses are its own block's shared::cluster ones
        constexpr int CHUNKS = C::HN / 16 / (C::EPI_WARPS / 4);   // of 16 columns, a warp's
        const int j0 = ((warp - 2) / 4) * CHUNKS;
        int local = 0;
        for (int tile = unit; tile < total; tile += units, ++local) {
            const int acc = local & 1;
            const bool full = glu_wait(TFULL0 + 8u * acc, (local >> 1) & 1, abort_flag, true);
            if (!__all_sync(0xffffffffu, full)) break;   // one decision a warp: the loads are the warp's
            ptx::tc_fence_after();
            int mt, nt;
            tile_coords<C::RASTER>(tile, a.tiles_m, a.tiles_n, mt, nt);
            const int wrow = mt * C::TILE_M + static_cast<int>(rank) * kBM + quad * 32;
            if (wrow < a.M) {
                const uint32_t trow = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * C::BN;
#pragma unroll 1
                for (int j = j0; j < j0 + CHUNKS; ++j) {
                    const int c0 = nt * C::HN + j * 16;
                    if (c0 >= a.N) break;   // N % 16 == 0
                    const uint32_t tg = trow + j * 16, tu = tg + C::HN;
                    if (a.dH) glu_act<true, true>(a, tg, tu, wrow, c0, lane);
                    else if (a.pair) glu_act<false, true>(a, tg, tu, wrow, c0, lane);
                    else glu_act<false, false>(a, tg, tu, wrow, c0, lane);
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                // Relaxed: what it tells is that the accumulator has been read.  A release would wait for the
                // tile's stores to memory (8192 x 512 x 1360: 37.5 us for the gradient).
                asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(tempty_leader + 8u * acc) : "memory");
            }
        }
    }

    ptx::tc_fence_before();
    if constexpr (CG == 2) ptx::cluster_sync(); else __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        if constexpr (CG == 2) ptx::tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
    if (warp == 0 && lane == 0 && *abort_flag) {
        // after an abort, copies still in flight must land before the shared memory is released
        if constexpr (CG == 1) {
            for (int s = 0; s < C::STAGES; ++s)
                if (issued & (1u << s)) glu_wait(FULL0 + 8u * s, (issued_parity >> s) & 1u, abort_flag, false);
        } else {
            const uint64_t t0 = ptx::globaltimer();   // a pair's copies count on the leader's barriers: give them time
            while (ptx::globaltimer() - t0 < 100000ull) {
            }
        }
    }
}

using GluPair = GluCfg<2, 128, 7>;
using GluOne = GluCfg<1, 128, 4>;
using GluPairNarrow = GluCfg<2, 64, 9>;   // for outputs of few tiles
using GluOneNarrow = GluCfg<1, 64, 6>;

// ------------------------------------------------------------------------------ a few rows
//
// glu_codes: 16 rows a block from the 2-bit codes.  A code's two bits as the upper two bits of a bf16 are
// twice its value (00: 0, 01: 0x4000 = 2, 11: 0xC000 = -2), so an operand register of two weights
// takes a shift and a mask.  The products run on mma.sync (m16n8k16), with the weights as the 16-row
// operand and the tokens as the 8 columns: with so few rows the time is that of reading and
// expanding codes, a tcgen05 tile of 128 rows would be mostly padding and would want the operand
// written to shared memory.  Element order within an MMA is free as long as both operands agree:
// lane (g, t) = (lane / 4, lane % 4) reads the words of 16 columns 16 g.. at the four weight rows
// 4 t.. of a block of 16 rows, and MMA j takes its columns 16 g + j and 16 g + j + 8.
//
// 1 x 4096 x 6144 7.6 us, 8 rows 8.8, 16 rows (two MMAs for each operand) 12.2, of which a launch is 3.6 and the
// codes' bytes would be 1.9.  No unit is at its limit: at 16 rows the tensor pipe is busy for 23% of the time,
// the issue slots for 35%, and per issue 2.1 warps wait for a result of fixed latency, 2.1 for a global load and
// 0.8 for a pipe.  So latency bounds it, at two blocks an SM; and 240 blocks for 304 places leave 64 SMs with one.
//
// A block has 128 outputs: half of its eight warps take the gate's 128 columns, half the value's, and share
// the weight's rows; where there are fewer blocks than SMs, the blocks of a cluster share them too.
// Sums are added in a fixed order: a warp's blocks of rows, the warps of a block, the blocks of a cluster.
constexpr int kCodeOut = 128, kCodeWarps = 4;       // warps for each of the two
constexpr int kCodePad = kCodeOut + 4;              // the pad keeps a warp's stores free of conflicts
constexpr int kCodeRows = 16;                       // rows of X that a block takes

struct CodeArgs {
    const uint16_t* X;
    const uint32_t* packed;
    const float* scale;
    uint16_t* H;
    int M, N, K, act, tiles;
};

__device__ __forceinline__ void mma_tokens(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes of eight columns at two rows: the lower (upper) halves of two words side by side.
__device__ __forceinline__ uint32_t halves(uint32_t w0, uint32_t w1, bool upper) { return __byte_perm(w0, w1, upper ? 0x7632 : 0x5410); }

template <int MT, int AHEAD>   // tokens in eights; blocks of 16 weight rows that a warp asks for at once
__global__ void __launch_bounds__(kCodeWarps * 64, 2) glu_codes(const __grid_constant__ CodeArgs args) {
    // [2][warps][8 MT][kCodePad] sums of the warps; then what the cluster's blocks push: [blocks][columns of one][2 M]
    extern __shared__ float part[];
    constexpr int SUMS = 8 * MT * kCodePad;
    float* pushed = part + 2 * kCodeWarps * SUMS;
    const int warp = (threadIdx.x >> 5) & (kCodeWarps - 1), side = threadIdx.x / (32 * kCodeWarps);   // 0: the gate
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t rank, size;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(size));
    if (size > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    ptx::pdl_trigger();
    const int unit = static_cast<int>(blockIdx.x / size), group = unit / args.tiles;
    CodeArgs a = args;   // of the block's rows
    a.X += group * kCodeRows * static_cast<int64_t>(a.K);
    a.H += group * kCodeRows * static_cast<int64_t>(a.N);
    a.M = min(kCodeRows, a.M - group * kCodeRows);
    const int n0 = (unit - group * a.tiles) * kCodeOut;
    const int words = a.N / 8;                       // of a weight row: 2N / 16
    const bool live = n0 + 16 * g < a.N;             // N % 16 == 0
    float acc[8][MT][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][m][i] = 0.f;
    const int step = static_cast<int>(size) * kCodeWarps, b0 = static_cast<int>(rank) * kCodeWarps + warp;
    const uint32_t* wp = a.packed + side * (a.N / 16) + (live ? n0 / 16 + g : 0) + (16 * static_cast<int64_t>(b0) + 4 * t) * words;
    const int64_t wstep = 16 * static_cast<int64_t>(step) * words;
    const uint16_t* xp = a.X + 16 * b0 + 4 * t + (g < a.M ? g : 0) * static_cast<int64_t>(a.K);
    const int64_t up = 8 * static_cast<int64_t>(a.K);
    const bool in0 = g < a.M, in1 = MT > 1 && 8 + g < a.M;
    ptx::pdl_wait();
    for (int left = (a.K / 16 - b0 + step - 1) / step; left > 0; left -= AHEAD) {   // this warp's blocks
        uint32_t w[AHEAD][4];
        uint2 x[AHEAD][MT];
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const bool in = q < left;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[q][i] = in && live ? __ldg(wp + i * words) : 0u;
            x[q][0] = in && in0 ? __ldg(reinterpret_cast<const uint2*>(xp)) : make_uint2(0u, 0u);
            if constexpr (MT > 1) x[q][MT - 1] = in && in1 ? __ldg(reinterpret_cast<const uint2*>(xp + up)) : make_uint2(0u, 0u);
            wp += wstep;
            xp += 16 * step;
        }
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            if (q < left) {
                const uint32_t l0 = halves(w[q][0], w[q][1], false), h0 = halves(w[q][0], w[q][1], true);
                const uint32_t l1 = halves(w[q][2], w[q][3], false), h1 = halves(w[q][2], w[q][3], true);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    constexpr uint32_t TOP = 0xC000C000u;
                    const int sh = 14 - 2 * j;
                    const uint32_t a0 = (l0 << sh) & TOP, a1 = (h0 << sh) & TOP, a2 = (l1 << sh) & TOP, a3 = (h1 << sh) & TOP;
#pragma unroll
                    for (int m = 0; m < MT; ++m) mma_tokens(acc[j][m], a0, a1, a2, a3, x[q][m].x, x[q][m].y);
                }
            }
        }
    }
    // column 16 g + c lies at 8 c + g: lanes of a store in different banks
    float* mine = part + (side * kCodeWarps + warp) * SUMS;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int token = 8 * m + 2 * t + i;
            if (token < a.M) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    mine[token * kCodePad + 8 * j + g] = acc[j][m][i];
                    mine[token * kCodePad + 8 * (j + 8) + g] = acc[j][m][i + 2];
                }
            }
        }
    __syncthreads();
    const int per = (kCodeOut + static_cast<int>(size) - 1) / static_cast<int>(size);   // columns that a block finishes
    if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every block has started
    // the warps' sums, to the block that finishes the column
    for (int e = threadIdx.x; e < 2 * a.M * kCodeOut; e += 64 * kCodeWarps) {
        const int at0 = e % kCodeOut, c = (at0 >> 3) + 16 * (at0 & 7), m = e / kCodeOut, of = m >= a.M, token = m - of * a.M;
        const float* from = part + of * kCodeWarps * SUMS + token * kCodePad + at0;
        float v = from[0];
#pragma unroll
        for (int w = 1; w < kCodeWarps; ++w) v += from[w * SUMS];
        const int to = c / per;
        const uint32_t at = ptx::smem_u32(pushed + (static_cast<int>(rank) * 2 * a.M + m) * per + c - to * per);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ptx::mapa_shared(at, to)), "f"(v) : "memory");
    }
    __syncwarp();
    if (size > 1) ptx::cluster_sync(); else __syncthreads();
    for (int e = threadIdx.x; e < per * a.M; e += 64 * kCodeWarps) {
        const int m = e / per, q = e - m * per, c = q + static_cast<int>(rank) * per, n = n0 + c;
        if (c >= kCodeOut || n >= a.N) continue;
        // half of the sums: the operand was twice the weight
        const float sg = 0.5f * __ldg(a.scale + n), su = 0.5f * __ldg(a.scale + a.N + n);
        float vg = 0.f, vu = 0.f;
#pragma unroll 4
        for (int r = 0; r < static_cast<int>(size); ++r) {
            vg += pushed[(r * 2 * a.M + m) * per + q];
            vu += pushed[(r * 2 * a.M + a.M + m) * per + q];
        }
        vg *= sg;
        vu *= su;
        F2 f, d;
        const F2 g2 = both(vg);
        switch (a.act) {
        case TERN_ACT_SILU: activate<TERN_ACT_SILU, false>(g2, f, d); break;
        case TERN_ACT_GELU: activate<TERN_ACT_GELU, false>(g2, f, d); break;
        case TERN_ACT_RELU2: activate<TERN_ACT_RELU2, false>(g2, f, d); break;
        default: activate<TERN_ACT_SIGMOID, false>(g2, f, d); break;
        }
        float act, same;
        split(f, act, same);
        a.H[m * static_cast<int64_t>(a.N) + n] = __bfloat16_as_ushort(__float2bfloat16_rn(act * vu));
    }
}

// ------------------------------------------------------------------------------ gradient from factors
// dY = dH f_g | dH f_u, eight elements of a row a thread; dY may lie in place of the factors.
__global__ void __launch_bounds__(256) glu_factors(const uint16_t* __restrict__ dH, const uint16_t* saved, uint16_t* dY, int64_t rows, int N) {
    using B = __nv_bfloat16;
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int units = N / 8;
    const int64_t total = rows * units, step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total; e += step) {
        const int64_t row = e / units;
        const int c = static_cast<int>(e - row * units) * 8;
        const auto d = load_raw<B, 8>(reinterpret_cast<const B*>(dH) + row * N + c);
        const int64_t at = row * 2 * N + c;
        const uint4* ps = reinterpret_cast<const uint4*>(saved + at);
        const uint4 fg = *ps, fu = *reinterpret_cast<const uint4*>(saved + at + N);
        Raw<B, 8> rg, ru;
        rg.w[0] = fg.x, rg.w[1] = fg.y, rg.w[2] = fg.z, rg.w[3] = fg.w;
        ru.w[0] = fu.x, ru.w[1] = fu.y, ru.w[2] = fu.z, ru.w[3] = fu.w;
        float vg[8], vu[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = raw_at<B, 8>(d, i);
            vg[i] = x * raw_at<B, 8>(rg, i);
            vu[i] = x * raw_at<B, 8>(ru, i);
        }
        store_as<B, 8>(reinterpret_cast<B*>(dY) + at, vg);
        store_as<B, 8>(reinterpret_cast<B*>(dY) + at + N, vu);
    }
}

// ------------------------------------------------------------------------------ host side
template <class C>
int glu_units(int num_sms, int* units) {
    static std::once_flag once[64];
    static cudaError_t status[64];
    static int pairs[64];
    int dev = 0;
    TERN_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return TERN_ERR_DEVICE;
    std::call_once(once[dev], [&] {
        status[dev] = cudaFuncSetAttribute(tern_glu_gemm<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
        if (status[dev] != cudaSuccess || C::CG == 1) return;
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2 * (num_sms / 2));
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::SMEM_BYTES;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        status[dev] = cudaOccupancyMaxActiveClusters(&n, tern_glu_gemm<C>, &cfg);
        pairs[dev] = n > 0 ? n : 1;
    });
    TERN_CUDA_TRY(status[dev]);
    *units = C::CG == 2 ? pairs[dev] : num_sms;
    return TERN_OK;
}

// Launched as the other GEMMs: after every earlier kernel of the stream has completed.
template <class C>
int glu_gemm(GluArgs& a, const uint16_t* X, const uint16_t* T, int num_sms, cudaStream_t s) {
    a.tiles_m = (a.M + C::TILE_M - 1) / C::TILE_M;
    a.tiles_n = (a.N + C::HN - 1) / C::HN;
    a.num_kb = (a.K + C::BK - 1) / C::BK;
    if (int st = tensor_map_2d(&a.mX, X, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.K, a.M, C::BK, kBM, CU_TENSOR_MAP_SWIZZLE_128B)) return st;
    if (int st = tensor_map_2d(&a.mT, T, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2 * static_cast<int64_t>(a.N), a.K, 64, C::BK, CU_TENSOR_MAP_SWIZZLE_128B))
        return st;
    int units = 0;
    if (int st = glu_units<C>(num_sms, &units)) return st;
    const int grid = C::CG * static_cast<int>(std::min<int64_t>(static_cast<int64_t>(a.tiles_m) * a.tiles_n, units));
    return launch_cluster(tern_glu_gemm<C>, grid, C::THREADS, C::SMEM_BYTES, C::CG, false, s, a);
}

template <class C>
int64_t glu_rounds(const GluArgs& a, int num_sms) {
    const int64_t tiles = static_cast<int64_t>((a.M + C::TILE_M - 1) / C::TILE_M) * ((a.N + C::HN - 1) / C::HN), units = num_sms / C::CG;
    return (tiles + units - 1) / units;
}
template <class Wide, class Narrow>
int glu_width(GluArgs& a, const uint16_t* X, const uint16_t* T, int num_sms, cudaStream_t s) {
    // a narrow tile takes a little more than half of a wide one's time
    if (glu_rounds<Narrow>(a, num_sms) * 5 < glu_rounds<Wide>(a, num_sms) * 9) return glu_gemm<Narrow>(a, X, T, num_sms, s);
    return glu_gemm<Wide>(a, X, T, num_sms, s);
}
int glu_many(GluArgs& a, const uint16_t* X, const uint16_t* T, int num_sms, cudaStream_t s) {
    a.whole = ((reinterpret_cast<uintptr_t>(a.H) | reinterpret_cast<uintptr_t>(a.pair)) & 31) == 0;   // N % 16 == 0: every row then
    return a.M > kBM ? glu_width<GluPair, GluPairNarrow>(a, X, T, num_sms, s) : glu_width<GluOne, GluOneNarrow>(a, X, T, num_sms, s);
}

constexpr int kCodeMost = 8;   // blocks of a cluster

template <int MT>
size_t code_smem(int M, int c) {
    const int per = (kCodeOut + c - 1) / c;
    return (static_cast<size_t>(2 * kCodeWarps) * 8 * MT * kCodePad + static_cast<size_t>(c) * 2 * M * per) * sizeof(float);
}

// Clusters of c blocks that are resident at once (with the shared memory of the most rows).
template <int MT, int AHEAD>
int code_room(int c, int* clusters) {
    static std::once_flag once[64];
    static cudaError_t status[64];
    static int room[64][kCodeMost + 1];
    int dev = 0;
    TERN_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return TERN_ERR_DEVICE;
    std::call_once(once[dev], [&] {
        const size_t most = code_smem<MT>(8 * MT, 1) + 8 * MT * 64;   // the columns of uneven shares
        status[dev] = cudaFuncSetAttribute(glu_codes<MT, AHEAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
        for (int k = 1; k <= kCodeMost && status[dev] == cudaSuccess; ++k) {
            cudaLaunchConfig_t cfg{};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = k;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(64 * k);
            cfg.blockDim = dim3(kCodeWarps * 64);
            cfg.dynamicSmemBytes = code_smem<MT>(8 * MT, k);
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            status[dev] = cudaOccupancyMaxActiveClusters(&room[dev][k], glu_codes<MT, AHEAD>, &cfg);
        }
    });
    TERN_CUDA_TRY(status[dev]);
    *clusters = room[dev][c];
    return TERN_OK;
}

// Clusters as large as leave every block resident at once and every warp a block of rows.
template <int MT, int AHEAD>
int glu_few(CodeArgs a, cudaStream_t s) {
    a.tiles = (a.N + kCodeOut - 1) / kCodeOut;
    const int blocks = a.K / 16;
    const int64_t units = static_cast<int64_t>(a.tiles) * ((a.M + kCodeRows - 1) / kCodeRows);
    int c = 1, room = 0;
    for (int k = 2; k <= kCodeMost && blocks > (k - 1) * kCodeWarps; ++k) {
        if (int st = code_room<MT, AHEAD>(k, &room)) return st;
        if (units <= room) c = k;
    }
    return launch_cluster(glu_codes<MT, AHEAD>, static_cast<unsigned>(units * c), kCodeWarps * 64, code_smem<MT>(std::min(a.M, kCodeRows), c), c, true, s, a);
}

// Whether M rows (17 .. 128) go through the codes, from what both take in us: sixteen rows at a time
// (4096 x 12288 weights: 8.6 each beside a launch) against the GEMM's longer set-up with its rounds of
// tiles, 0.27 for each 64 of K, or the bytes of the bf16 plane.  40 x 3872 x 192: 6.5 us by the codes, 22.5
// in the GEMM; 64 x 4096 x 6144: 25 us in the GEMM, 38 by the codes.
bool few_by_codes(const GluArgs& a, int num_sms) {
    const double groups = (a.M + kCodeRows - 1) / kCodeRows;
    const int64_t wide = glu_rounds<GluOne>(a, num_sms), narrow = glu_rounds<GluOneNarrow>(a, num_sms);
    const double rounds = std::min(static_cast<double>(wide), 0.55 * static_cast<double>(narrow));
    const double weights = 2.0 * a.K * a.N;
    return groups * weights * 0.17e-6 < 2.5 + std::max(0.27 * a.K / 64 * rounds, weights * 2 / 6.5e6);
}

bool glu_dims(int64_t M, int64_t K, int64_t N) {
    // 2N columns within 31 bits; rows of dY and of the weight within the tensor maps' limits
    return M >= 0 && K >= 16 && N >= 16 && M < (1ll << 31) - 1024 && K < (1ll << 31) - 1024 && N < (1ll << 30) - 1024 && M * K < (1ll << 40) &&
           K * N < (1ll << 39) && M * N < (1ll << 39) &&
           ((M + 127) / 128) * ((N + 63) / 64) < (1ll << 31) - 1024;
}

}  // namespace

int glu_status_read(int clear) {
    int v = 0;
    TERN_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_glu_status, sizeof(int)));
    if (clear) {
        const int zero = 0;
        TERN_CUDA_TRY(cudaMemcpyToSymbol(g_glu_status, &zero, sizeof(int)));
    }
    return v ? TERN_ERR_TIMEOUT : TERN_OK;
}

}  // namespace tern

using namespace tern;

extern "C" int tern_glu_fwd(const uint16_t* X, const tern_tiles* W, const float* scale, int act, uint16_t* H, uint16_t* saved, int64_t M,
                            int64_t K, int64_t N, void* stream) {
    if (!glu_dims(M, K, N) || act < TERN_ACT_SILU || act > TERN_ACT_SIGMOID) return TERN_ERR_ARG;
    if (K % 16 || N % 16) return TERN_ERR_ALIGN;
    if (M == 0) return TERN_OK;
    if (!X || !W || !scale || !H) return TERN_ERR_ARG;
    const bool can = M <= kBM && !saved && W->packed;   // the codes serve few rows
    if (!can && !W->t_bf16) return TERN_ERR_ARG;
    if (!aligned16(X) || !aligned16(scale) || !aligned16(H) || !aligned16(saved) || (can && !aligned16(W->packed)) || !aligned16(W->t_bf16))
        return TERN_ERR_ALIGN;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    GluArgs a{};
    a.scale = scale, a.H = H, a.pair = saved;
    a.M = static_cast<int>(M), a.N = static_cast<int>(N), a.K = static_cast<int>(K), a.act = act;
    if (can && (M <= kCodeRows || !W->t_bf16 || few_by_codes(a, num_sms))) {
        const CodeArgs c{X, W->packed, scale, H, a.M, a.N, a.K, act, 0};
        return M <= 8 ? glu_few<1, 4>(c, s) : glu_few<2, 3>(c, s);
    }
    return glu_many(a, X, W->t_bf16, num_sms, s);
}

extern "C" int tern_glu_bwd(const uint16_t* dH, const uint16_t* saved, const uint16_t* X, const tern_tiles* W, const float* scale, int act,
                            uint16_t* dY, int64_t M, int64_t K, int64_t N, void* stream) {
    if (!glu_dims(M, saved ? 16 : K, N) || (!saved && (act < TERN_ACT_SILU || act > TERN_ACT_SIGMOID))) return TERN_ERR_ARG;
    if (N % 16 || (!saved && K % 16)) return TERN_ERR_ALIGN;
    if (M == 0) return TERN_OK;
    if (!dH || !dY || (!saved && (!X || !W || !W->t_bf16 || !scale))) return TERN_ERR_ARG;
    if (!aligned16(dH) || !aligned16(dY) || !aligned16(saved)) return TERN_ERR_ALIGN;
    if (!saved && (!aligned16(X) || !aligned16(W->t_bf16) || !aligned16(scale))) return TERN_ERR_ALIGN;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (saved) {
        const int64_t units = M * (N / 8);
        const int grid = static_cast<int>(std::min<int64_t>((units + 255) / 256, static_cast<int64_t>(num_sms) * 8));
        return launch_pdl(glu_factors, dim3(grid), dim3(256), 0, s, dH, saved, dY, M, static_cast<int>(N));
    }
    GluArgs a{};
    a.scale = scale, a.dH = dH, a.pair = dY;
    a.M = static_cast<int>(M), a.N = static_cast<int>(N), a.K = static_cast<int>(K), a.act = act;
    return glu_many(a, X, W->t_bf16, num_sms, s);
}
