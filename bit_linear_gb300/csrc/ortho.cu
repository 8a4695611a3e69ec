// Orthogonalised update of a weight's gradient by Newton-Schulz products.
//
//   X = G / (|G|_F + eps), then `steps` times  A = X X^T,  M = a I + b A + c A A,  X = M X
//
// with (a, b, c) = (3.4445, -4.7750, 2.0315): an odd quintic applied to every singular value,
// which takes those of X (at most 1) to about 1 (0.7 to 1.2) and leaves the singular vectors
// alone.  For K > N the products are taken on the other side (A = X^T X, X = X M), so A is always
// of the smaller side, and G is never transposed.
//
// Precision.  A singular value of 1e-3 of the largest grows by up to 3.4445 a step, 480 times in
// five, and with it whatever noise the roundings before left in its directions: one binary16 or
// bf16 plane per operand (2^-12, 2^-9) would leave directions of a real gradient's weak singular
// values to chance.  Every matrix is therefore kept as two binary16 planes hi + lo, 22 bits, and a
// product is three tensor-core passes into one fp32 accumulator, hi*hi + hi*lo + lo*hi; the
// dropped lo*lo is 2^-22 of the product.  The sum is less exact than its terms: the tensor cores cut
// each of its 3 depth / 16 additions towards zero.  With exact sums out would be 4e-7 of its norm from
// the fp64 result before its rounding; as it is, one element in a hundred is a bf16 step off the rounded
// fp64 result at 512 x 2048, one in 36 at 1100 x 4200 and one in 22 at 4096 x 12288 (one in 350 to 500
// with fp32 arithmetic, one in three with one binary16 plane), and |out - fp64| / |fp64| is there 1.6580e-3
// where rounding alone gives 1.6561e-3.  Scales of powers of two keep both planes normal numbers:
// |X| <= 1.21 is stored times 2^14, |A| <= 1.46 and |M| <= 3.45 times 2^13 (bounds of the quintic
// on [0, 1] and its image), so a lo plane's smallest spacing is 2^-38 of 1.  Where |G|_F is below eps, X
// starts below 1/2 and would lose its low bits there: it is stored times 2^k more, with the k that takes
// its norm to between 1/2 and 1, and A times 2^2k.  A step multiplies by up to 3.4445, so k falls with the
// steps to 0, where X has reached the rest of the quintic; the products' factors undo it (Factors).
//
// Two steps at once, for m (n - m) of a million and more (and at 1024 rows from n = 1536 on): with M0 =
// p(A), the next step's A is M0 A M0 = (M0 M0) A, as all of these commute, and X = (M1 M0) X, so
// the pair needs one product of X in place of two: 3 m^2 n / 2 + 5 m^3 / 2 multiply-adds against
// 3 m^2 n + m^3.  More than two would pass the
// square of the amplification on to A's rounding.  The weak directions stay sound: where the
// eigenvalue of A is lost in A's rounding M is still a, and they are X's own.
//
// Cost: A and M are symmetric, so half of their tiles are computed (and mirrored), and a step is
// m^2 n + m^3 + 2 m^2 n multiply-adds of one plane, three times that in tensor-core work; bounded
// by the tensor cores for m >= 2048, by the launches of 3 * steps products for m of some hundreds.
//
// The GEMM: a persistent kernel, operands by TMA with the 128-byte swizzle (K-major or MN-major,
// as the products need), accumulators in TMEM, two of them so that the epilogue of a tile overlaps
// the next one's main loop.  warp 0 copies, warp 1 issues the MMAs, warps 2-9 drain (two per TMEM
// lane quarter).  The four operand tiles of a 64-deep k-block feed twelve MMAs: one and a half
// times the work per byte of shared memory of a plain product.  256 x 256 tiles by CTA pairs where
// they fill the GPU, else 128 x 128 or 128 x 64 by single CTAs, and clusters that share the
// contraction of a few tiles.
//
// 4096 x 12288: 5.2 ms; a product of X runs at 1.82 PFLOP/s of executed passes (0.95 of the measured
// cuBLAS burst rate, tensor pipe busy 0.84), the symmetric ones at 0.77 of that: 136 tiles on 76
// pairs are two rounds, the second one of 60.  512 x 2048: 143 us, eight a product: the end of the
// launch before it 2, the first copies 1.3, the k-blocks 0.45 each (operands at 87 B/ns into an SM),
// the exchange and the stores 3.
#include <algorithm>
#include <cmath>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mma.cuh"

namespace tern {

__device__ int g_ortho_status;   // 1 once a bounded wait gave up

namespace {

constexpr int kRows = 128;       // rows of A (and of D) per CTA
constexpr int kBK = 64;
constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 16384.0f, kScaleA = 8192.0f, kScaleM = 8192.0f;
constexpr float kScaleQ = 4096.0f;   // of products of two M, at most 11.9

enum { OUT_SYM, OUT_POLY, OUT_X, OUT_FINAL };

struct OrthoArgs {
    CUtensorMap ah, al, bh, bl;
    int rows, cols, ld;           // D: rows x cols, planes with rows of ld elements (ld % 8 == 0)
    int tiles_m, tiles_n, units, num_kb, split;
    int kind;
    __half *oh, *ol;              // D's planes
    const __half *ch, *cl;        // OUT_POLY: A's planes
    float alpha, pa, pb;          // OUT_POLY: pa I + pb A + alpha acc; else alpha acc
    const int* k_first;           // k of the first X
    int k_in, k_out;              // steps' worth of k gone by: of what is read, and of D
    __nv_bfloat16* out;           // OUT_FINAL: [rows][cols]
};

// CG CTAs share one MMA (a pair has the tile's 256 rows between them).  SPLIT: one tile per cluster,
// whose CTAs each take a part of the contraction.
template <int CG_, int BN_, bool A_MN_, bool B_MN_, bool SPLIT_ = false>
struct OCfg {
    static constexpr int CG = CG_, BN = BN_;
    static constexpr bool A_MN = A_MN_, B_MN = B_MN_, SPLIT = SPLIT_;
    static constexpr int THREADS = 64 + 256;
    static constexpr int TILE_M = kRows * CG, B_ROWS = BN / CG;
    static constexpr int A_BYTES = kRows * kBK * 2, B_BYTES = B_ROWS * kBK * 2;   // of one plane
    static constexpr int STAGE_BYTES = 2 * (A_BYTES + B_BYTES);
    static constexpr int STAGES = 196608 / STAGE_BYTES;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 256;
    static constexpr int RASTER = 16 / CG;
    static_assert(2 * SMEM_BYTES > 233472, "one CTA per SM");
    static_assert(B_ROWS % 64 == 0 && TMEM_COLS <= 512 && SMEM_BYTES <= 232448, "tile");
};

// The symmetric products' tiles: those with an element on or above the diagonal, row by row.
template <class C>
__host__ __device__ __forceinline__ int sym_first(int mt) { return mt * C::TILE_M / C::BN; }

template <class C>
__device__ __forceinline__ void unit_tile(const OrthoArgs& a, int unit, int& mt, int& nt) {
    if (a.kind == OUT_SYM || a.kind == OUT_POLY) {
        mt = 0;
        int n = a.tiles_n;
        while (unit >= n) {
            unit -= n;
            ++mt;
            n = a.tiles_n - sym_first<C>(mt);
        }
        nt = sym_first<C>(mt) + unit;
    } else {
        tile_coords<C::RASTER>(unit, a.tiles_m, a.tiles_n, mt, nt);
    }
}

// The accumulator's factor and A's with the powers of two by which operands and D are stored.  OUT_FINAL,
// which stores X itself, has its power in two halves (pb and post), numbers of their own where it is none.
struct Factors {
    float alpha, pb, post;
};
__device__ __forceinline__ Factors factors(const OrthoArgs& a) {
    const int k0 = *a.k_first, k = max(k0 - a.k_in, 0), to = max(k0 - a.k_out, 0);
    Factors f{a.alpha, a.kind == OUT_FINAL ? 1.0f : a.pb, 1.0f};
    if (k == 0) return f;
    if (a.kind == OUT_POLY) f.alpha = ldexpf(a.alpha, -4 * k), f.pb = ldexpf(a.pb, -2 * k);   // A A and A, of 2^2k each
    if (a.kind == OUT_SYM) f.alpha = ldexpf(a.alpha, 2 * (to - k));                           // A's next (else k_in = k_out)
    if (a.kind == OUT_X) f.alpha = ldexpf(a.alpha, to - k);
    if (a.kind == OUT_FINAL) f.post = ldexpf(1.0f, -(k / 2)), f.pb = ldexpf(1.0f, -(k - k / 2));
    return f;
}

__device__ __forceinline__ void split16(float v, __half& hi, __half& lo) {
    hi = __float2half_rn(v);
    lo = __float2half_rn(v - __half2float(hi));
}

// Lane i of each eight holds row i of an 8 x 8 block, x its columns; afterwards column i, x its rows.
__device__ __forceinline__ void transpose8(uint32_t (&x)[8], int lane) {
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1) {
        const bool upper = (lane & d) != 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i & d) continue;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? x[i] : x[i | d], d);
            if (upper) x[i] = other;
            else x[i | d] = other;
        }
    }
}

// Eight columns c..c+7 (c % 8 == 0) of row `row`, from the accumulator's values; called by whole
// warps, whose lanes hold 32 consecutive rows.  Of a symmetric product, the 8 x 8 blocks above the
// diagonal are stored twice, as they are and transposed (in registers: stores of single elements
// took 3.5 us to drain, most of a small product's time), those on it once.
__device__ __forceinline__ bool group_here(const OrthoArgs& a, int row, int c) {
    return row < a.rows && c < a.ld && ((a.kind != OUT_SYM && a.kind != OUT_POLY) || c >= (row & ~7));
}
// OUT_POLY: A's planes there.
__device__ __forceinline__ void group_load(const OrthoArgs& a, int row, int c, uint4& h, uint4& l) {
    h = l = make_uint4(0u, 0u, 0u, 0u);
    if (a.kind == OUT_POLY && group_here(a, row, c)) {
        h = *reinterpret_cast<const uint4*>(a.ch + static_cast<int64_t>(row) * a.ld + c);
        l = *reinterpret_cast<const uint4*>(a.cl + static_cast<int64_t>(row) * a.ld + c);
    }
}
__device__ __forceinline__ void ortho_group(const OrthoArgs& a, const Factors& f, const float (&acc)[8], const uint4& h0, const uint4& l0, int row, int c,
                                            int lane) {
    const bool sym = a.kind == OUT_SYM || a.kind == OUT_POLY;
    const int row8 = row & ~7;
    const bool here = group_here(a, row, c);
    if (a.kind == OUT_FINAL) {
        if (!here) return;
        __nv_bfloat16* o = a.out + static_cast<int64_t>(row) * a.cols + c;
        if (a.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(f.alpha * acc[2 * k] * f.pb * f.post, f.alpha * acc[2 * k + 1] * f.pb * f.post);
                u[k] = *reinterpret_cast<const uint32_t*>(&t);
            }
            *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k < a.cols) o[k] = __float2bfloat16_rn(f.alpha * acc[k] * f.pb * f.post);
        }
        return;
    }
    const int64_t base = static_cast<int64_t>(row) * a.ld + c;
    __align__(16) __half hi[8], lo[8];
    if (a.kind == OUT_POLY) {
        __align__(16) __half ah[8], al[8];
        *reinterpret_cast<uint4*>(ah) = h0;
        *reinterpret_cast<uint4*>(al) = l0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = __half2float(ah[k]) + __half2float(al[k]);
            split16(fmaf(f.alpha, acc[k], f.pb * x) + (c + k == row ? a.pa : 0.0f), hi[k], lo[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) split16(f.alpha * acc[k], hi[k], lo[k]);
    }
    if (here) {
        *reinterpret_cast<uint4*>(a.oh + base) = *reinterpret_cast<const uint4*>(hi);
        *reinterpret_cast<uint4*>(a.ol + base) = *reinterpret_cast<const uint4*>(lo);
    }
    if (sym) {
        uint32_t x[8], h[4], l[4];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = static_cast<uint32_t>(__half_as_ushort(hi[k])) | static_cast<uint32_t>(__half_as_ushort(lo[k])) << 16;
        transpose8(x, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = __byte_perm(x[2 * k], x[2 * k + 1], 0x5410);
            l[k] = __byte_perm(x[2 * k], x[2 * k + 1], 0x7632);
        }
        const int mrow = c + (lane & 7);   // rows past the last are zeros, which the columns past it want
        if (c > row8 && row8 < a.rows && mrow < a.rows) {
            const int64_t at = static_cast<int64_t>(mrow) * a.ld + row8;
            *reinterpret_cast<uint4*>(a.oh + at) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(a.ol + at) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) tern_ortho_gemm(const __grid_constant__ OrthoArgs a) {
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
    const int part = C::SPLIT ? static_cast<int>(ptx::cluster_ctarank()) : 0;
    const int group = C::SPLIT ? a.split : CG;                     // CTAs per unit
    const int unit0 = static_cast<int>(blockIdx.x) / group, stride = static_cast<int>(gridDim.x) / group;
    const int kb0 = C::SPLIT ? a.num_kb * part / a.split : 0, kb1 = C::SPLIT ? a.num_kb * (part + 1) / a.split : a.num_kb;
    auto wait = [&](uint32_t bar, uint32_t parity, bool watch = true) {
        return wait_limited(bar, parity, abort_flag, watch, kWaitLimitNs, [&] { atomicExch(&g_ortho_status, 1); });
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(FULL0 + 8u * s, 1);
            ptx::mbar_init(EMPTY0 + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(TFULL0 + 8u * b, 1);
            ptx::mbar_init(TEMPTY0 + 8u * b, 8 * CG);   // every epilogue warp of the group
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
    if (threadIdx.x == 0)
        for (const CUtensorMap* m : {&a.ah, &a.al, &a.bh, &a.bl}) ptx::tma_prefetch_desc(m);
    ptx::pdl_trigger();
    ptx::pdl_wait();

    Factors f{};
    if (warp >= 2) f = factors(a);
    uint32_t issued = 0, issued_parity = 0;   // producer: stages with a copy issued, and its phase
    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = unit0; ok && u < a.units; u += stride) {
            int mt, nt;
            unit_tile<C>(a, u, mt, nt);
            const int arow = mt * C::TILE_M + static_cast<int>(rank) * kRows;
            const int brow = nt * C::BN + static_cast<int>(rank) * C::B_ROWS;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait(EMPTY0 + 8u * stage, phase ^ 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t full = FULL0 + 8u * stage;
                const uint32_t full_at = CG == 2 ? ptx::mapa_shared(full, 0) : full;   // the pair counts on the leader's
                const uint32_t sA = base + stage * C::STAGE_BYTES, sB = sA + 2 * C::A_BYTES;
                if (rank == 0) ptx::mbar_arrive_expect_tx(full, CG * C::STAGE_BYTES);
                auto load = [&](uint32_t dst, const CUtensorMap* m, bool mn, int rows, int r0) {
                    const int k0 = kb * kBK;
                    if (mn) {
                        for (int j = 0; j < rows / 64; ++j) {
                            if constexpr (CG == 2) ptx::tma_load_2d_pair(dst + j * 64 * kBK * 2, m, r0 + j * 64, k0, full_at);
                            else ptx::tma_load_2d(dst + j * 64 * kBK * 2, m, r0 + j * 64, k0, full_at);
                        }
                    } else {
                        if constexpr (CG == 2) ptx::tma_load_2d_pair(dst, m, k0, r0, full_at);
                        else ptx::tma_load_2d(dst, m, k0, r0, full_at);
                    }
                };
                load(sA, &a.ah, C::A_MN, kRows, arow);
                load(sB, &a.bh, C::B_MN, C::B_ROWS, brow);
                load(sB + C::B_BYTES, &a.bl, C::B_MN, C::B_ROWS, brow);
                load(sA + C::A_BYTES, &a.al, C::A_MN, kRows, arow);
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == C::STAGES) stage = 0, phase ^= 1u;
            }
        }
        // Until the MMA has released every stage filled above: the release is an asynchronous
        // arrival that may otherwise land in the barriers of the next CTA on this SM.
        if (ok) {
            for (int s = 0; s < C::STAGES; ++s)
                if (issued & (1u << s)) wait(EMPTY0 + 8u * s, (issued_parity >> s) & 1u);
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ------------------------------------------------------------ MMA issuer (leader only)
        constexpr uint32_t IDESC = make_idesc(C::TILE_M, C::BN, C::A_MN, C::B_MN, 0u);   // binary16 operands
        auto mma = [&](uint32_t d, uint64_t da, uint64_t db, uint32_t acc) {
            if constexpr (CG == 2) ptx::mma_bf16_pair(d, da, db, IDESC, acc);
            else ptx::mma_bf16(d, da, db, IDESC, acc);
        };
        auto commit = [&](uint32_t bar) {
            if constexpr (CG == 2) ptx::mma_commit_pair_mc(bar, 0x3);
            else ptx::mma_commit(bar);
        };
        int stage = 0, local = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = unit0; ok && u < a.units; u += stride, ++local) {
            const int acc = local & 1;
            if (!wait(TEMPTY0 + 8u * acc, ((local >> 1) & 1) ^ 1u)) break;
            ptx::tc_fence_after();
            const uint32_t d = tmem_base + acc * C::BN;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait(FULL0 + 8u * stage, phase)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t sA = base + stage * C::STAGE_BYTES, sB = sA + 2 * C::A_BYTES;
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk) {
                    const uint64_t ah = op_desc<C::A_MN, kBK>(sA, kk), al = op_desc<C::A_MN, kBK>(sA + C::A_BYTES, kk);
                    const uint64_t bh = op_desc<C::B_MN, kBK>(sB, kk), bl = op_desc<C::B_MN, kBK>(sB + C::B_BYTES, kk);
                    mma(d, ah, bl, kb != kb0 || kk != 0 ? 1u : 0u);
                    mma(d, al, bh, 1u);
                    mma(d, ah, bh, 1u);
                }
                commit(EMPTY0 + 8u * stage);
                if (++stage == C::STAGES) stage = 0, phase ^= 1u;
            }
            if (!ok) break;
            commit(TFULL0 + 8u * acc);
        }
        // every MMA issued completes before TMEM and shared memory go away
        if constexpr (CG == 2) ptx::mma_commit_pair(DRAIN); else ptx::mma_commit(DRAIN);
        wait(DRAIN, 0, false);
        // and the epilogues' release of each accumulator's last use has landed
        if (ok && !*abort_flag) {
            for (int acc = 0; acc < 2; ++acc) {
                if (local <= acc) continue;
                const int last = (local - 1) - (((local - 1) - acc) & 1);
                wait(TEMPTY0 + 8u * acc, static_cast<uint32_t>(last >> 1) & 1u);
            }
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue
        const int quad = warp & 3;   // TMEM lanes 32*quad .. +31
        const uint32_t tempty = CG == 2 ? ptx::mapa_shared(TEMPTY0, 0) : TEMPTY0;
        constexpr int JPW = C::BN / 64;   // 32-column chunks per warp: each quarter's two warps take half
        const int j0 = ((warp - 2) / 4) * JPW;
        int local = 0;
        for (int u = unit0; u < a.units; u += stride, ++local) {
            const int acc = local & 1;
            const bool full = wait(TFULL0 + 8u * acc, (local >> 1) & 1);
            if (!__all_sync(0xffffffffu, full)) break;   // one decision per warp: the loads are collective
            ptx::tc_fence_after();
            int mt, nt;
            unit_tile<C>(a, u, mt, nt);
            const int row0 = mt * C::TILE_M + static_cast<int>(rank) * kRows;
            const uint32_t trow = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * C::BN;
            const bool sym = a.kind == OUT_SYM || a.kind == OUT_POLY;
            if constexpr (C::SPLIT) {
                // the partial tile to shared memory, over the operand stages (all read by now): four columns
                // of all rows side by side, so that a warp's reads from a peer are of neighbouring bytes
                // (of rows 272 bytes apart they took 3 us a tile)
                uint4* p = reinterpret_cast<uint4*>(smem_raw + (base - raw)) + quad * 32 + lane;
#pragma unroll 1
                for (int j = j0; j < j0 + JPW; ++j) {
                    uint32_t r[32];
                    ptx::tmem_ld_32x32b_x32(trow + j * 32, r);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        p[(j * 8 + k / 4) * kRows] = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
                }
            } else if (row0 < a.rows) {
#pragma unroll 1
                for (int j = j0; j < j0 + JPW; ++j) {
                    const int c0 = nt * C::BN + j * 32;
                    if (c0 >= a.ld) break;
                    if (sym && c0 + 31 < row0 + quad * 32) continue;   // wholly below the diagonal
                    uint32_t r[32];
                    ptx::tmem_ld_32x32b_x32(trow + j * 32, r);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r[8 * g + k]);
                        uint4 ph, pl;
                        group_load(a, row0 + quad * 32 + lane, c0 + 8 * g, ph, pl);
                        ortho_group(a, f, v, ph, pl, row0 + quad * 32 + lane, c0 + 8 * g, lane);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) ptx::mbar_arrive_cluster(tempty + 8u * acc);
                else ptx::mbar_arrive(TEMPTY0 + 8u * acc);
            }
        }
    }

    if constexpr (C::SPLIT) {
        // each CTA adds up its share of the tile's columns over the partial tiles, in order
        const int share = C::BN / a.split, r = (warp & 3) * 32 + lane;
        int mt = 0, nt = 0;
        if (unit0 < a.units) unit_tile<C>(a, unit0, mt, nt);
        const int row = mt * C::TILE_M + r;
        const int g0 = (warp - 2) / 4;      // the first of this warp's groups of eight columns
        uint4 ph, pl;                       // its planes of A are on their way during the exchange
        if (warp >= 2 && unit0 < a.units) group_load(a, row, nt * C::BN + part * share + 8 * g0, ph, pl);
        __syncwarp();
        ptx::cluster_sync();
        if (warp >= 2 && unit0 < a.units) {
            for (int g = g0; g < share / 8; g += 2) {
                const int col = part * share + 8 * g;
                const uint32_t at = base + static_cast<uint32_t>(col / 4 * kRows + r) * 16u;
                if (g != g0) group_load(a, row, nt * C::BN + col, ph, pl);
                float x[8][8], v[8] = {};
#pragma unroll
                for (int k = 0; k < 8; ++k) {   // all in flight together
                    if (k >= a.split) break;
                    const uint32_t peer = ptx::mapa_shared(at, k);
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(x[k][0]), "=f"(x[k][1]), "=f"(x[k][2]), "=f"(x[k][3]) : "r"(peer) : "memory");
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(x[k][4]), "=f"(x[k][5]), "=f"(x[k][6]), "=f"(x[k][7]) : "r"(peer + kRows * 16u) : "memory");
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (k >= a.split) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += x[k][i];
                }
                ortho_group(a, f, v, ph, pl, row, nt * C::BN + col, lane);
            }
        }
    }
    ptx::tc_fence_before();
    if constexpr (C::SPLIT) {
        // The peers have read this CTA's partial tile (and used what they read).  Nothing is published
        // here, so the barrier need not wait for the stores.
        __syncwarp();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    } else if constexpr (CG == 2) {
        ptx::cluster_sync();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        if constexpr (CG == 2) ptx::tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
    if (warp == 0 && lane == 0 && *abort_flag) {
        // after an abort, copies still in flight must land before the shared memory is released
        if constexpr (CG == 1) {
            for (int s = 0; s < C::STAGES; ++s)
                if (issued & (1u << s)) wait(FULL0 + 8u * s, (issued_parity >> s) & 1u, false);
        } else {
            // a pair's copies complete on the leader's barriers; give them time to land
            const uint64_t t0 = ptx::globaltimer();
            for (uint32_t i = 0; i < (1u << 24) && ptx::globaltimer() - t0 < 100000ull; ++i) {
            }
        }
    }
}

}  // namespace

// Sum of squares of G, a partial sum per block in fp64 (fixed chunks and order).  Sixteen squares
// at a time are added in fp32, whose rounding is then that of sixteen terms, unless their range
// does not allow it: fp64 throughout would take as long as the arithmetic, not the reads
// (227 us against 44 us for the 4096 x 12288 gradient).
constexpr int kSumBlocks = 304;
__global__ void __launch_bounds__(256) tern_ortho_sumsq_kernel(const float* __restrict__ G, int64_t n, double* __restrict__ partial) {
    __shared__ double red[256];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const bool wide = (reinterpret_cast<uintptr_t>(G) & 15u) == 0;
    double sum = 0.0;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256 * 16;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < n; i += stride) {
        // four groups of four, a block's threads side by side in each
        float v[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t at = i + static_cast<int64_t>(q) * gridDim.x * 1024;
            if (wide && at + 4 <= n) {
                const float4 t = __ldg(reinterpret_cast<const float4*>(G + at));
                v[4 * q] = t.x, v[4 * q + 1] = t.y, v[4 * q + 2] = t.z, v[4 * q + 3] = t.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[4 * q + k] = at + k < n ? __ldg(G + at + k) : 0.0f;
            }
        }
        float top = 0.0f, s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            top = fmaxf(top, fabsf(v[k]));
            s = fmaf(v[k], v[k], s);
        }
        // squares between 2^-100 (what underflows is 2^-26 of the largest) and 2^120; a NaN is in s
        if (top > 8.9e-16f && top < 1e18f) sum += static_cast<double>(s);
        else if (top != 0.0f || s != s) {
#pragma unroll
            for (int k = 0; k < 16; ++k) sum += static_cast<double>(v[k]) * static_cast<double>(v[k]);
        }
    }
    red[threadIdx.x] = sum;
    __syncthreads();
    for (int k = 128; k > 0; k >>= 1) {
        if (threadIdx.x < k) red[threadIdx.x] += red[threadIdx.x + k];
        __syncthreads();
    }
    if (threadIdx.x == 0) partial[blockIdx.x] = red[0];
}

// X's planes from G: rows of ld columns, zeros past the last; and X's k.  Every block adds up the
// partial sums for itself, in the same order.
__global__ void __launch_bounds__(256) tern_ortho_load_kernel(const float* __restrict__ G, int64_t rows, int cols, int ld,
                                                              const double* __restrict__ partial, int parts, float eps,
                                                              __half* __restrict__ hi, __half* __restrict__ lo, int* k_first) {
    __shared__ double red[256];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    double sum = 0.0;
    for (int k = threadIdx.x; k < parts; k += 256) sum += partial[k];
    red[threadIdx.x] = sum;
    __syncthreads();
    for (int k = 128; k > 0; k >>= 1) {
        if (threadIdx.x < k) red[threadIdx.x] += red[threadIdx.x + k];
        __syncthreads();
    }
    const double norm = sqrt(red[0]), size = norm + static_cast<double>(eps);
    double scale = static_cast<double>(kScaleX) / size;
    int k = 0, over = 0;
    if (norm > 0.0 && norm <= static_cast<double>(eps) && isfinite(size)) {
        k = ilogb(size / norm);   // |X| 2^k: above 1/2, at most 1
        scale = ldexp(scale, k);
        over = max(ilogb(scale) - 120, 0);   // of norms below 2^-106 the factor would pass fp32's range
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *k_first = k;
    const float inv = static_cast<float>(over == 0 ? scale : ldexp(scale, -over)), more = ldexpf(1.0f, over);
    const int per_row = ld / 8;
    const bool wide = cols % 4 == 0 && (reinterpret_cast<uintptr_t>(G) & 15u) == 0;
    const int64_t total = rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / per_row;
        const int c = static_cast<int>(i - row * per_row) * 8;
        const float* g = G + row * cols + c;
        float v[8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (wide) {
                float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c + 4 * q < cols) t = __ldg(reinterpret_cast<const float4*>(g + 4 * q));
                v[4 * q] = t.x, v[4 * q + 1] = t.y, v[4 * q + 2] = t.z, v[4 * q + 3] = t.w;
            } else {
#pragma unroll
                for (int k = 4 * q; k < 4 * q + 4; ++k) v[k] = c + k < cols ? __ldg(g + k) : 0.0f;
            }
        }
        __align__(16) __half h[8], l[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) split16(v[k] * inv * more, h[k], l[k]);
        *reinterpret_cast<uint4*>(hi + row * ld + c) = *reinterpret_cast<const uint4*>(h);
        *reinterpret_cast<uint4*>(lo + row * ld + c) = *reinterpret_cast<const uint4*>(l);
    }
}

// ------------------------------------------------------------------------------ host side
namespace {

// Configures a GEMM kernel once per device; the co-resident CTAs (or pairs).
template <class C>
int ortho_units(int num_sms, int* units) {
    static std::once_flag once[64];
    static int status[64], clusters[64];
    int dev = 0;
    TERN_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return TERN_ERR_DEVICE;
    std::call_once(once[dev], [&] {
        status[dev] = TERN_ERR_CUDA;
        if (cudaFuncSetAttribute(tern_ortho_gemm<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
            return;
        clusters[dev] = num_sms;
        if (C::CG == 2) {
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
            if (cudaOccupancyMaxActiveClusters(&n, tern_ortho_gemm<C>, &cfg) != cudaSuccess) return;
            clusters[dev] = std::max(n, 1);
        }
        status[dev] = TERN_OK;
    });
    *units = clusters[dev];
    return status[dev];
}

// An operand: two planes of [outer][inner] binary16, read K-major (inner is the contraction) or MN-major.
struct Operand {
    const __half *hi, *lo;
    int64_t inner, outer;
};

int map_planes(CUtensorMap* hi, CUtensorMap* lo, const Operand& x, bool mn, int rows) {
    for (int p = 0; p < 2; ++p) {
        const int st = tensor_map_2d(p == 0 ? hi : lo, p == 0 ? x.hi : x.lo, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x.inner, x.outer,
                                     64, mn ? kBK : rows, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != TERN_OK) return st;
    }
    return TERN_OK;
}

template <class C>
int ortho_gemm(OrthoArgs& a, const Operand& A, const Operand& B, int64_t depth, int num_sms, cudaStream_t s, int split = 1) {
    int max_units = 0;
    if (int st = ortho_units<C>(num_sms, &max_units)) return st;
    if (int st = map_planes(&a.ah, &a.al, A, C::A_MN, kRows)) return st;
    if (int st = map_planes(&a.bh, &a.bl, B, C::B_MN, C::B_ROWS)) return st;
    a.tiles_m = (a.rows + C::TILE_M - 1) / C::TILE_M;
    a.tiles_n = (a.ld + C::BN - 1) / C::BN;
    a.num_kb = static_cast<int>((depth + kBK - 1) / kBK);
    a.units = a.tiles_m * a.tiles_n;
    if (a.kind == OUT_SYM || a.kind == OUT_POLY) {
        a.units = 0;
        for (int mt = 0; mt < a.tiles_m; ++mt) a.units += a.tiles_n - sym_first<C>(mt);
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.numAttrs = 0;
    a.split = C::SPLIT ? split : 1;
    const int group = C::SPLIT ? split : C::CG;
    if (group > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = group;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    if (C::CG == 1) {
        // A chain of products of some hundred rows is bound by launches: let each set itself up while
        // the one before it runs.  Two of these CTAs never share an SM (each takes most of its shared
        // memory), and a grid lets the next one launch only once all its own CTAs hold their TMEM, so
        // no allocation waits on a grid that waits in turn.  The pairs start, as the library's other
        // pair GEMMs, once every earlier kernel on the stream has completed.
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = dim3(C::SPLIT ? a.units * split : C::CG * std::min(a.units, max_units));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    TERN_CUDA_TRY(cudaLaunchKernelEx(&cfg, tern_ortho_gemm<C>, static_cast<const OrthoArgs&>(a)));
    return TERN_OK;
}

// The tile by the time that its rounds take.  A k-block takes 1.1 us in a 256 x 256 tile of a pair, 0.6
// in a 128 x 128 tile and 0.45 in a 128 x 64 one, but 0.95 and 0.65 where every SM has one, which then
// share what L2 delivers; the last tile's stores take 5, 3 and 1.5 us.  (2500 x 2500: the symmetric
// products in 55 large tiles, one round, or 210 of 128 x 128, two: 1035 and 1248 us; 1500 x 4000: in 78
// of 128 x 128 or 156 of 128 x 64: 570 and 761 us; 2049 x 2049: the products of X in 81 large tiles or
// 289: 845 and 799 us; 2048 x 2048: in 64 or 256: 509 and 525 us; 512 x 2048: in 64 of 128 x 128 or 128
// of 128 x 64: 159 and 143 us.)
template <bool A_MN, bool B_MN>
int ortho_product(OrthoArgs& a, const Operand& A, const Operand& B, int64_t depth, int num_sms, cudaStream_t s) {
    const bool sym = a.kind == OUT_SYM || a.kind == OUT_POLY;
    auto tiles = [&](int64_t tm, int64_t tn) {
        const int64_t m = (a.rows + tm - 1) / tm, n = (a.ld + tn - 1) / tn;
        return m * n - (sym ? m * (m - 1) / 2 * (tm / tn) : 0);
    };
    // Few tiles: clusters of S CTAs share each one's contraction, at least a k-block a CTA.  Clusters of
    // 8, 4 and 2 CTAs of this size fit 16, 36 and 76 times.  (512 x 2048: 174 us without, 142 us; 256 x
    // 1024: 111 us with at least two k-blocks a CTA, 105 us.)
    const int64_t n = tiles(128, 64), kb = (depth + kBK - 1) / kBK;
    const int S = n <= 16 && kb >= 8 ? 8 : n <= 36 && kb >= 4 ? 4 : n <= 76 && kb >= 2 ? 2 : 1;
    if (S > 1) return ortho_gemm<OCfg<1, 64, A_MN, B_MN, true>>(a, A, B, depth, num_sms, s, S);
    auto time = [&](int64_t n, int64_t at_once, int64_t full, int64_t least, int64_t stores) {   // in 10 ns
        const int64_t rest = n % at_once;
        return kb * (n / at_once * full + (rest != 0 ? std::max(least, full * rest / at_once) : 0)) + stores;
    };
    const int64_t large = time(tiles(256, 256), num_sms / 2, 110, 110, 500);
    const int64_t middle = time(tiles(128, 128), num_sms, 95, 60, 300);
    const int64_t small = time(n, num_sms, 65, 45, 150);
    if (large <= middle && large <= small) return ortho_gemm<OCfg<2, 256, A_MN, B_MN>>(a, A, B, depth, num_sms, s);
    if (middle <= small) return ortho_gemm<OCfg<1, 128, A_MN, B_MN>>(a, A, B, depth, num_sms, s);
    return ortho_gemm<OCfg<1, 64, A_MN, B_MN>>(a, A, B, depth, num_sms, s);
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

struct OrthoPlan {
    int64_t m, ldx, ldm;                     // smaller side; elements between rows of X and of A, M
    int64_t sums, k, x, mat[4], bytes;         // parts of the workspace, in bytes (x: two X of two planes; A, M and two more for pairs of steps)
    int64_t x_plane, m_plane;                // bytes of one plane
    bool pairs;                              // steps two at a time
};

OrthoPlan ortho_plan(int64_t K, int64_t N) {
    OrthoPlan p{};
    p.m = std::min(K, N);
    p.ldx = round_up(N, 8);
    p.ldm = round_up(p.m, 8);
    p.x_plane = round_up(K * p.ldx * 2, 256);
    p.m_plane = round_up(p.m * p.ldm * 2, 256);
    p.sums = 0;
    p.k = kSumBlocks * static_cast<int64_t>(sizeof(double));
    p.x = round_up(p.k + static_cast<int64_t>(sizeof(int)), 256);
    // From about a million on the products of X that a pair of steps saves, m m (n - m) each, are worth
    // more than its additional products of the smaller side: 512 x 4096 180 us, in pairs 168; 900 x 4000 311
    // and 273; 4096 x 5000 3358 and 3143.  Just below, either may be the faster (512 x 2400 153 and 151, 600 x
    // 2200 181 and 176, 896 x 1900 235 both, 1100 x 1900 313 and 326, 1152 x 2040 310 and 323), and far below
    // single steps are (600 x 1500 166 and 171, 1000 x 1530 234 and 239, 1280 x 1920 315 and 333, 2048 x 2048
    // 508 and 534, 3000 x 3180 1584 and 1672).  At 1024 rows, the most whose symmetric products share their
    // contractions over clusters of two, pairs are as good from n = 1.5 m on: 1024 x 1536 216 both, 1024 x 1800
    // 227 and 224, 2040 x 1024 225 and 221 (1100 x 1650, without the clusters, 310 and 325).
    const int64_t n = std::max(K, N);
    p.pairs = p.m * (n - p.m) >= 1 << 20 || (p.m == 1024 && n >= 1536);
    p.bytes = p.x + 4 * p.x_plane;
    for (int i = 0; i < (p.pairs ? 4 : 2); ++i) p.mat[i] = p.bytes, p.bytes += 2 * p.m_plane;
    return p;
}

bool ortho_sizes_ok(int64_t K, int64_t N) { return K >= 0 && N >= 0 && K < (1 << 30) && N < (1 << 30) && (N == 0 || K <= (1ll << 40) / N); }

}  // namespace

int ortho_status_read(int clear) {
    int v = 0;
    TERN_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_ortho_status, sizeof(v)));
    const int zero = 0;
    if (v != 0 && clear) TERN_CUDA_TRY(cudaMemcpyToSymbol(g_ortho_status, &zero, sizeof(zero)));
    return v != 0 ? TERN_ERR_TIMEOUT : TERN_OK;
}

}  // namespace tern

using namespace tern;

extern "C" size_t tern_orthogonalize_workspace(int64_t K, int64_t N) {
    return ortho_sizes_ok(K, N) && K > 0 && N > 0 ? static_cast<size_t>(ortho_plan(K, N).bytes) : 0;
}

extern "C" int tern_orthogonalize(const float* G, int64_t K, int64_t N, int steps, float eps, float gain, uint16_t* out,
                                  void* workspace, size_t ws_bytes, void* stream) {
    if (!ortho_sizes_ok(K, N) || steps < 1 || steps > 64 || !(eps >= 1e-30f)) return TERN_ERR_ARG;
    if (K == 0 || N == 0) return TERN_OK;
    if (!G || !out) return TERN_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(G) % 4 || reinterpret_cast<uintptr_t>(out) % 2) return TERN_ERR_ALIGN;
    const OrthoPlan p = ortho_plan(K, N);
    if (!workspace || ws_bytes < static_cast<size_t>(p.bytes)) return TERN_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) % 128) return TERN_ERR_ALIGN;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    double* sums = reinterpret_cast<double*>(ws + p.sums);
    int* k_first = reinterpret_cast<int*>(ws + p.k);
    auto half = [&](int64_t at) { return reinterpret_cast<__half*>(ws + at); };
    __half* x[2][2];
    for (int q = 0; q < 2; ++q)
        for (int i = 0; i < 2; ++i) x[i][q] = half(p.x + (2 * i + q) * p.x_plane);
    const int parts = static_cast<int>(std::min<int64_t>((K * N + 4095) / 4096, kSumBlocks));
    if (int st = launch_pdl(tern_ortho_sumsq_kernel, dim3(parts), dim3(256), 0, s, G, K * N, sums)) return st;
    const int64_t chunks = K * (p.ldx / 8);
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((chunks + 255) / 256, 8 * num_sms));
    if (int st = launch_pdl(tern_ortho_load_kernel, dim3(blocks), dim3(256), 0, s, G, K, static_cast<int>(N),
                            static_cast<int>(p.ldx), static_cast<const double*>(sums), parts, eps, x[0][0], x[0][1], k_first))
        return st;
    // that many steps' worth of k: X grows by up to 3.4445 in each
    auto grown = [](int t) { return static_cast<int>(std::ceil(t * std::log2(static_cast<double>(kA)))); };
    const bool tall = K > N;
    Operand mat[4];   // symmetric, by commuting factors: A, M, and for pairs of steps M0 M0 then M1, and the second A
    for (int i = 0; i < (p.pairs ? 4 : 2); ++i) mat[i] = Operand{half(p.mat[i]), half(p.mat[i] + p.m_plane), p.ldm, p.m};
    auto to = [](OrthoArgs& a, const Operand& d) { a.oh = const_cast<__half*>(d.hi), a.ol = const_cast<__half*>(d.lo); };
    // Of a product that reads the t-th step's X or A, and whose D is the next-th's.
    auto steps_args = [&](int t, int next) {
        OrthoArgs a{};
        a.k_first = k_first, a.k_in = grown(t), a.k_out = grown(next);
        return a;
    };
    // D = alpha L R, of which half the tiles are computed
    auto product = [&](const Operand& L, const Operand& R, const Operand& D, float alpha, int t, int next) {
        OrthoArgs a = steps_args(t, next);
        a.rows = static_cast<int>(p.m), a.cols = a.rows, a.ld = static_cast<int>(p.ldm);
        a.kind = OUT_SYM, a.alpha = alpha;
        to(a, D);
        return ortho_product<false, false>(a, L, R, p.ldm, num_sms, s);
    };
    // D = a I + b A + c A A
    auto poly = [&](const Operand& A, const Operand& D, int t) {
        OrthoArgs a = steps_args(t, t);
        a.rows = static_cast<int>(p.m), a.cols = a.rows, a.ld = static_cast<int>(p.ldm);
        a.kind = OUT_POLY, a.ch = A.hi, a.cl = A.lo;
        a.alpha = kScaleM * kC / (kScaleA * kScaleA), a.pa = kScaleM * kA, a.pb = kScaleM * kB / kScaleA;
        to(a, D);
        return ortho_product<false, false>(a, A, A, p.ldm, num_sms, s);
    };
    int cur = 0;
    for (int t = 0; t < steps; cur ^= 1) {
        const Operand X{x[cur][0], x[cur][1], p.ldx, K};
        const int t0 = t;
        OrthoArgs a = steps_args(t0, t0);
        a.rows = static_cast<int>(p.m), a.cols = a.rows, a.ld = static_cast<int>(p.ldm);
        a.kind = OUT_SYM, a.alpha = kScaleA / (kScaleX * kScaleX);
        to(a, mat[0]);
        if (int st = tall ? ortho_product<true, true>(a, X, X, K, num_sms, s) : ortho_product<false, false>(a, X, X, p.ldx, num_sms, s))
            return st;
        if (int st = poly(mat[0], mat[1], t0)) return st;
        Operand Q = mat[1];
        float q_scale = kScaleM;
        t += 1;
        if (p.pairs && t < steps) {
            if (int st = product(mat[1], mat[1], mat[2], kScaleQ / (kScaleM * kScaleM), t0, t0)) return st;   // M0 M0
            if (int st = product(mat[2], mat[0], mat[3], 1.0f / kScaleQ, t0, t0 + 1)) return st;              // the second A
            if (int st = poly(mat[3], mat[2], t0 + 1)) return st;                                             // M1
            if (int st = product(mat[2], mat[1], mat[0], kScaleQ / (kScaleM * kScaleM), t0, t0)) return st;   // M1 M0
            Q = mat[0], q_scale = kScaleQ;
            t += 1;
        }
        a = steps_args(t0, t);
        a.rows = static_cast<int>(K), a.cols = static_cast<int>(N), a.ld = static_cast<int>(p.ldx);
        a.kind = t == steps ? OUT_FINAL : OUT_X;
        a.oh = x[cur ^ 1][0], a.ol = x[cur ^ 1][1], a.out = reinterpret_cast<__nv_bfloat16*>(out);
        a.alpha = a.kind == OUT_FINAL ? gain / (q_scale * kScaleX) : 1.0f / q_scale;
        if (int st = tall ? ortho_product<false, false>(a, X, Q, p.ldm, num_sms, s) : ortho_product<false, true>(a, Q, X, p.m, num_sms, s))
            return st;
    }
    return TERN_OK;
}
