// Gated linear recurrence over sequences, its gradient, and its single-token step.
//
//   a_t = sigmoid(f_t + bias), h_t = a_t h_{t-1} + (1 - a_t) v_t, y_t = sigmoid(r_t) h_t
//
// per sequence b and channel d; h_{t-1} is read as 0 at a document start, and rows at or past
// lengths[b] are padding (never read: a = 1, no input, y = 0, gradients 0).
//
// The map of one row, h -> a h + b, composes: rows i..j act as h -> A h + H with A = prod a and
// H the state reached from 0.  A block takes 32*VEC channels and ROWS consecutive rows, RPT rows
// per warp (lane = VEC channels, so a warp's loads are whole lines), all held in registers:
//   1. each thread folds its RPT rows into (A, H) and leaves the pair in shared memory;
//   2. after a barrier it folds the pairs of the warps before it onto the block's incoming state;
//   3. it runs its rows again from that state and writes y.
// A block walks T in steps of ROWS.  Where sequences times channel tiles are too few blocks to
// fill the GPU, a cluster of S blocks takes S consecutive steps at a time and exchanges the
// blocks' totals through distributed shared memory, one cluster barrier per S steps.  Every
// fold has a fixed order, so results do not depend on the schedule; nothing polls memory.
//
// The gradient runs the same way from the end of the sequence, with e_t = a_t dh_t as its state:
//   dh_t = g_t + e_{t+1}, e_t = a_t dh_t, g_t = sigmoid(r_t) dy_t, e_T = dhT
//   dv = (1 - a) dh, df = dh (h_{t-1} - v) a (1 - a), dr = dy h s (1 - s), dh0 = e_0
// and recomputes h inside its 64 rows from the states the forward saved every 64 rows (1/16 B
// per element beside the 22 B of a forward and a backward in bf16).
//
// Bounded by HBM (each input read once, each output written once) with the special-function
// unit next: four operations per element (two sigmoids) against the 5.4 per element that its
// rate allows at 8 B per element.  Gates and states are fp32; outputs are rounded once.
#include <cuda_bf16.h>

#include "common.cuh"

namespace tern {
namespace {

constexpr int kSaveRows = 64;    // rows between saved states; the backward's block step
constexpr int kMaxCluster = 8;   // portable cluster size

// --------------------------------------------------------------- element access
template <class T, int VEC>
struct Io;
template <>
struct Io<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw load(const void* p, int64_t i) {
        return __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p) + i));
    }
    static __device__ __forceinline__ void get(Raw r, float (&x)[2]) {
        x[0] = __uint_as_float(r << 16);
        x[1] = __uint_as_float(r & 0xFFFF0000u);
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&x)[2]) {
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p) + i) = __floats2bfloat162_rn(x[0], x[1]);
    }
};
template <>
struct Io<__nv_bfloat16, 1> {
    using Raw = unsigned short;
    static __device__ __forceinline__ Raw load(const void* p, int64_t i) {
        return __ldg(static_cast<const unsigned short*>(p) + i);
    }
    static __device__ __forceinline__ void get(Raw r, float (&x)[1]) { x[0] = __uint_as_float(static_cast<uint32_t>(r) << 16); }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&x)[1]) {
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x[0]);
    }
};
template <>
struct Io<float, 2> {
    using Raw = float2;
    static __device__ __forceinline__ Raw load(const void* p, int64_t i) {
        return __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(p) + i));
    }
    static __device__ __forceinline__ void get(Raw r, float (&x)[2]) { x[0] = r.x, x[1] = r.y; }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&x)[2]) {
        *reinterpret_cast<float2*>(static_cast<float*>(p) + i) = make_float2(x[0], x[1]);
    }
};
template <>
struct Io<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ Raw load(const void* p, int64_t i) { return __ldg(static_cast<const float*>(p) + i); }
    static __device__ __forceinline__ void get(Raw r, float (&x)[1]) { x[0] = r; }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&x)[1]) { static_cast<float*>(p)[i] = x[0]; }
};

// s = sigmoid(x) and n = sigmoid(-x), each to a few units in the last place (n is not formed
// as 1 - s, which loses it where s is near 1).  e = exp(-x) is capped at 2^125 so that s and
// e*s stay normal numbers: for x below -86 (-inf included) s is 2^-125 and n is 1.  A NaN
// stays one.
__device__ __forceinline__ void gate(float x, float& s, float& n) {
    float e = __expf(-x);
    asm("min.NaN.f32 %0, %1, 0f7E000000;" : "=f"(e) : "f"(e));
    s = __fdividef(1.0f, 1.0f + e);
    n = e * s;
}

// A row map whose A carries the sign bit ignores the state before it (a document start lies in
// its rows): -0 keeps its sign through products with the a >= 0 of later rows, and no value of
// an earlier document, NaN included, passes.
__device__ __forceinline__ bool cuts(float A) { return (__float_as_uint(A) >> 31) != 0; }
__device__ __forceinline__ float apply(float A, float H, float h) { return cuts(A) ? H : fmaf(A, h, H); }

struct Strided {
    const void* p;
    int64_t sb, st;   // elements between sequences and between rows
};
struct ScanArgs {
    Strided f, v, r, y;   // y: the forward's output, or the backward's dy
    const float* f_bias;
    const int32_t* lengths;
    const uint8_t* starts;
    float* saved;         // [B][ceil(T/64)][D]
    const float* h_in;    // h0 (forward) or dhT (backward); may be null
    float* h_out;         // hT or dh0; may be null
    int T, D, tiles, S;
};
struct GradArgs {
    ScanArgs s;
    Strided df, dv, dr;
    float* partial;       // [B*S][D] sums of df, or null
};

__device__ __forceinline__ int rows_live(const ScanArgs& a, int b) {
    return a.lengths != nullptr ? min(max(a.lengths[b], 0), a.T) : a.T;
}
// bit i: row0 + i (of the nl live rows of this warp) starts a document
__device__ __forceinline__ uint32_t start_bits(const ScanArgs& a, int64_t b, int row0, int nl, int lane) {
    if (a.starts == nullptr) return 0;
    const int st = lane < nl ? a.starts[b * a.T + row0 + lane] : 0;
    return __ballot_sync(0xffffffffu, st != 0);
}

// N consecutive floats of this block's shared memory at `p`, read from block `rank` of the cluster.
template <int N>
__device__ __forceinline__ void load_peer(const float* p, uint32_t rank, float (&x)[N]) {
    const uint32_t at = ptx::mapa_shared(ptx::smem_u32(p), rank);
    if constexpr (N == 4) {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(at) : "memory");
    } else {
        static_assert(N == 2, "two or four");
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(at) : "memory");
    }
}

}  // namespace

// ------------------------------------------------------------------------------ forward
// CL: the S blocks of a cluster take S consecutive steps at a time; otherwise S is 1.
template <class T, int VEC, int RPT, int WARPS, bool CL>
__global__ void __launch_bounds__(WARPS * 32, 2) tern_scan_fwd_kernel(const __grid_constant__ ScanArgs a) {
    using X = Io<T, VEC>;
    constexpr int ROWS = RPT * WARPS;
    static_assert(kSaveRows % RPT == 0 && RPT <= 32, "saved states fall on warp boundaries");
    __shared__ alignas(16) float agg[2][WARPS][32][2 * VEC];
    __shared__ alignas(16) float tot[2][32][2 * VEC];      // CL: this block's (A, H)
    __shared__ float carry_s[2][32][VEC];                  // not CL: the state after a step
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cl = blockIdx.x / a.S, rank = blockIdx.x - cl * a.S;
    const int64_t b = cl / a.tiles;
    const int d = (cl - static_cast<int>(b) * a.tiles) * (32 * VEC) + lane * VEC;
    const bool on = d < a.D;
    const int len = rows_live(a, static_cast<int>(b));
    const int64_t nsaved = (static_cast<int64_t>(a.T) + kSaveRows - 1) / kSaveRows;
    const int64_t fo = b * a.f.sb + d, vo = b * a.v.sb + d, ro = b * a.r.sb + d, yo = b * a.y.sb + d;

    float bias[VEC], carry[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        bias[j] = on && a.f_bias != nullptr ? a.f_bias[d + j] : 0.0f;
        carry[j] = on && a.h_in != nullptr ? a.h_in[b * a.D + d + j] : 0.0f;
    }
    const int steps = (a.T + ROWS - 1) / ROWS;
    const int iters = (steps + a.S - 1) / a.S;
    for (int it = 0; it < iters; ++it) {
        const int p = it & 1;
        const int64_t first = static_cast<int64_t>(it * a.S + rank) * ROWS + w * RPT;
        const int row0 = first < a.T ? static_cast<int>(first) : a.T;
        const int nl = min(max(len - row0, 0), RPT);   // live rows of this warp
        const uint32_t cut = start_bits(a, b, row0, nl, lane);
        typename X::Raw rf[RPT], rv[RPT], rr[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            rf[i] = typename X::Raw{}, rv[i] = typename X::Raw{}, rr[i] = typename X::Raw{};
            if (on && i < nl) {
                const int64_t t = row0 + i;
                rf[i] = X::load(a.f.p, fo + t * a.f.st);
                rv[i] = X::load(a.v.p, vo + t * a.v.st);
                rr[i] = X::load(a.r.p, ro + t * a.r.st);
            }
        }
        // (A, H) of this thread's rows
        float ga[RPT][VEC], gb[RPT][VEC], A[VEC], H[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) A[j] = 1.0f, H[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            float f[VEC], v[VEC];
            X::get(rf[i], f);
            X::get(rv[i], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float s, n;
                gate(f[j] + bias[j], s, n);
                ga[i][j] = i < nl ? s : 1.0f;
                gb[i][j] = i < nl ? n * v[j] : 0.0f;
            }
        }
        if (cut == 0) {
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) A[j] *= ga[i][j], H[j] = fmaf(ga[i][j], H[j], gb[i][j]);
        } else {
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const bool c = (cut >> i) & 1u;
                    A[j] = c ? -0.0f : A[j] * ga[i][j];
                    H[j] = c ? gb[i][j] : fmaf(ga[i][j], H[j], gb[i][j]);
                }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) agg[p][w][lane][j] = A[j], agg[p][w][lane][VEC + j] = H[j];
        __syncthreads();
        // the state before this block's rows
        float h[VEC];
        if constexpr (CL) {
            if (w == WARPS - 1) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) A[j] = 1.0f, H[j] = 0.0f;
#pragma unroll
                for (int k = 0; k < WARPS; ++k)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float Ak = agg[p][k][lane][j], Hk = agg[p][k][lane][VEC + j];
                        H[j] = apply(Ak, Hk, H[j]);
                        A[j] = cuts(Ak) ? Ak : A[j] * Ak;
                    }
#pragma unroll
                for (int j = 0; j < VEC; ++j) tot[p][lane][j] = A[j], tot[p][lane][VEC + j] = H[j];
            }
            ptx::cluster_sync();
            for (int k = 0; k < a.S; ++k) {
                float x[2 * VEC];
                load_peer(&tot[p][lane][0], k, x);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (k == rank) h[j] = carry[j];
                    carry[j] = apply(x[j], x[VEC + j], carry[j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) h[j] = it == 0 ? carry[j] : carry_s[p ^ 1][lane][j];
        }
        for (int k = 0; k < w; ++k)
#pragma unroll
            for (int j = 0; j < VEC; ++j) h[j] = apply(agg[p][k][lane][j], agg[p][k][lane][VEC + j], h[j]);
        if (a.saved != nullptr && on && row0 < a.T && row0 % kSaveRows == 0) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) a.saved[(b * nsaved + row0 / kSaveRows) * a.D + d + j] = h[j];
        }
        // the rows again, from the state before them
        if (cut == 0) {
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) h[j] = fmaf(ga[i][j], h[j], gb[i][j]), gb[i][j] = h[j];
        } else {
#pragma unroll
            for (int i = 0; i < RPT; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    h[j] = (cut >> i) & 1u ? gb[i][j] : fmaf(ga[i][j], h[j], gb[i][j]);
                    gb[i][j] = h[j];
                }
        }
        if constexpr (!CL) {
            if (w == WARPS - 1) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) carry_s[p][lane][j] = h[j];
            }
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            float r[VEC], y[VEC];
            X::get(rr[i], r);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float s, n;
                gate(r[j], s, n);
                y[j] = i < nl ? s * gb[i][j] : 0.0f;
            }
            if (on && row0 + i < a.T) X::store(const_cast<void*>(a.y.p), yo + static_cast<int64_t>(row0 + i) * a.y.st, y);
        }
    }
    if constexpr (CL) {
        ptx::cluster_sync();   // the peers have read this block's totals
    } else {
        __syncthreads();
        if (iters > 0) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) carry[j] = carry_s[(iters - 1) & 1][lane][j];
        }
    }
    if (a.h_out != nullptr && on && rank == 0 && w == 0) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) a.h_out[b * a.D + d + j] = carry[j];
    }
}

// ------------------------------------------------------------------------------ backward
template <class T, int VEC, bool CL>
__global__ void __launch_bounds__(256, 2) tern_scan_bwd_kernel(const __grid_constant__ GradArgs g) {
    using X = Io<T, VEC>;
    constexpr int RPT = 8, WARPS = 8, ROWS = RPT * WARPS;
    static_assert(ROWS == kSaveRows, "a step starts from a saved state");
    const ScanArgs& a = g.s;
    __shared__ alignas(16) float agg[2][WARPS][32][2 * VEC];   // A and G (the gradient's fold)
    __shared__ alignas(16) float aggh[2][WARPS][32][VEC];      // H (the state's fold)
    __shared__ alignas(16) float tot[2][32][2 * VEC];
    __shared__ float carry_s[2][32][VEC];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cl = blockIdx.x / a.S, rank = blockIdx.x - cl * a.S;
    const int64_t b = cl / a.tiles;
    const int d = (cl - static_cast<int>(b) * a.tiles) * (32 * VEC) + lane * VEC;
    const bool on = d < a.D;
    const int len = rows_live(a, static_cast<int>(b));
    const int steps = (a.T + ROWS - 1) / ROWS;
    const int iters = (steps + a.S - 1) / a.S;
    const int64_t fo = b * a.f.sb + d, vo = b * a.v.sb + d, ro = b * a.r.sb + d, yo = b * a.y.sb + d;
    const int64_t dfo = b * g.df.sb + d, dvo = b * g.dv.sb + d, dro = b * g.dr.sb + d;

    float bias[VEC], carry[VEC], dbias[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        bias[j] = on && a.f_bias != nullptr ? a.f_bias[d + j] : 0.0f;
        carry[j] = on && a.h_in != nullptr ? a.h_in[b * a.D + d + j] : 0.0f;
        dbias[j] = 0.0f;
    }
    for (int it = 0; it < iters; ++it) {
        const int p = it & 1;
        const int step = steps - 1 - (it * a.S + rank);   // below 0: nothing left for this block
        const int row0 = step >= 0 ? min(step * ROWS + w * RPT, a.T) : a.T;
        const int nl = min(max(len - row0, 0), RPT);
        const uint32_t cut = start_bits(a, b, row0, nl, lane);
        typename X::Raw rf[RPT], rv[RPT], rr[RPT], rd[RPT];
        float h[VEC];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            rf[i] = rv[i] = rr[i] = rd[i] = typename X::Raw{};
            if (on && i < nl) {
                const int64_t t = row0 + i;
                rf[i] = X::load(a.f.p, fo + t * a.f.st);
                rv[i] = X::load(a.v.p, vo + t * a.v.st);
                rr[i] = X::load(a.r.p, ro + t * a.r.st);
                rd[i] = X::load(a.y.p, yo + t * a.y.st);
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            h[j] = on && step >= 0 ? a.saved[(b * steps + step) * a.D + d + j] : 0.0f;
        // per row: s = a, n = 1 - a, o = g = sigmoid(r) dy, q = sigmoid(-r)
        float s[RPT][VEC], n[RPT][VEC], o[RPT][VEC], q[RPT][VEC];
        float A[VEC], H[VEC], G[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) A[j] = 1.0f, H[j] = 0.0f, G[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            float f[VEC], v[VEC], r[VEC], dy[VEC];
            X::get(rf[i], f);
            X::get(rv[i], v);
            X::get(rr[i], r);
            X::get(rd[i], dy);
            const bool c = (cut >> i) & 1u;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float so;
                gate(f[j] + bias[j], s[i][j], n[i][j]);
                gate(r[j], so, q[i][j]);
                o[i][j] = so * dy[j];
                if (i >= nl) s[i][j] = 1.0f, n[i][j] = 0.0f, o[i][j] = 0.0f;
                A[j] = c ? -0.0f : A[j] * s[i][j];
                H[j] = c ? n[i][j] * v[j] : fmaf(s[i][j], H[j], n[i][j] * v[j]);
            }
        }
#pragma unroll
        for (int i = RPT - 1; i >= 0; --i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) G[j] = (cut >> i) & 1u ? 0.0f : s[i][j] * (o[i][j] + G[j]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            agg[p][w][lane][j] = A[j], agg[p][w][lane][VEC + j] = G[j];
            aggh[p][w][lane][j] = H[j];
        }
        __syncthreads();
        float e[VEC];   // e after this thread's rows
        if constexpr (CL) {
            if (w == 0) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) A[j] = 1.0f, G[j] = 0.0f;
#pragma unroll
                for (int k = WARPS - 1; k >= 0; --k)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float Ak = agg[p][k][lane][j], Gk = agg[p][k][lane][VEC + j];
                        G[j] = apply(Ak, Gk, G[j]);
                        A[j] = cuts(Ak) ? Ak : A[j] * Ak;
                    }
#pragma unroll
                for (int j = 0; j < VEC; ++j) tot[p][lane][j] = A[j], tot[p][lane][VEC + j] = G[j];
            }
            ptx::cluster_sync();
            for (int k = 0; k < a.S; ++k) {
                float x[2 * VEC];
                load_peer(&tot[p][lane][0], k, x);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (k == rank) e[j] = carry[j];
                    carry[j] = apply(x[j], x[VEC + j], carry[j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) e[j] = it == 0 ? carry[j] : carry_s[p ^ 1][lane][j];
        }
        for (int k = WARPS - 1; k > w; --k)
#pragma unroll
            for (int j = 0; j < VEC; ++j) e[j] = apply(agg[p][k][lane][j], agg[p][k][lane][VEC + j], e[j]);
        for (int k = 0; k < w; ++k)
#pragma unroll
            for (int j = 0; j < VEC; ++j) h[j] = apply(agg[p][k][lane][j], aggh[p][k][lane][j], h[j]);
        // the states before and after each row: hp = h_{t-1}; q becomes dr = g h (1 - sigmoid(r))
        float hp[RPT][VEC];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            float v[VEC];
            X::get(rv[i], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                hp[i][j] = (cut >> i) & 1u ? 0.0f : h[j];
                h[j] = fmaf(s[i][j], hp[i][j], n[i][j] * v[j]);
                q[i][j] = i < nl ? o[i][j] * h[j] * q[i][j] : 0.0f;
            }
        }
#pragma unroll
        for (int i = RPT - 1; i >= 0; --i) {
            float v[VEC], df[VEC], dv[VEC];
            X::get(rv[i], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float dh = o[i][j] + e[j];
                const float e2 = s[i][j] * dh;
                dv[j] = i < nl ? n[i][j] * dh : 0.0f;
                df[j] = i < nl ? e2 * n[i][j] * (hp[i][j] - v[j]) : 0.0f;
                dbias[j] += df[j];
                e[j] = (cut >> i) & 1u ? 0.0f : e2;
            }
            if (on && row0 + i < a.T) {
                const int64_t t = row0 + i;
                X::store(const_cast<void*>(g.df.p), dfo + t * g.df.st, df);
                X::store(const_cast<void*>(g.dv.p), dvo + t * g.dv.st, dv);
                X::store(const_cast<void*>(g.dr.p), dro + t * g.dr.st, q[i]);
            }
        }
        if constexpr (!CL) {
            if (w == 0) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) carry_s[p][lane][j] = e[j];
            }
        }
    }
    if constexpr (CL) ptx::cluster_sync();   // the peers have read this block's totals
    __syncthreads();
    if constexpr (!CL) {
        if (iters > 0) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) carry[j] = carry_s[(iters - 1) & 1][lane][j];
        }
    }
    if (a.h_out != nullptr && on && rank == 0 && w == 0) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) a.h_out[b * a.D + d + j] = carry[j];
    }
    if (g.partial != nullptr) {   // this block's sum of df, warps in order
#pragma unroll
        for (int j = 0; j < VEC; ++j) aggh[0][w][lane][j] = dbias[j];
        __syncthreads();
        if (w == 0 && on) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < WARPS; ++k) sum += aggh[0][k][lane][j];
                g.partial[(b * a.S + rank) * a.D + d + j] = sum;
            }
        }
    }
}

// dbias[d] = sum of the blocks' partial sums: 8 warps take every eighth partial, then in order.
__global__ void __launch_bounds__(256) tern_scan_dbias_kernel(const float* __restrict__ partial, int64_t parts, int D,
                                                              float* __restrict__ dbias) {
    __shared__ float red[8][32];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int d = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (d < D) {
#pragma unroll 4
        for (int64_t k = w; k < parts; k += 8) sum += partial[k * D + d];
    }
    red[w][lane] = sum;
    __syncthreads();
    if (w == 0 && d < D) {
#pragma unroll
        for (int k = 1; k < 8; ++k) sum += red[k][lane];
        dbias[d] = sum;
    }
}

// ------------------------------------------------------------------------------ one token
struct StepArgs {
    const void *f, *v, *r;
    const float* f_bias;
    const float* h_in;
    float* h_out;
    void* y;
    int64_t rows, f_sb, v_sb, r_sb, y_sb;
    int D;
};

template <class T, int VEC>
__global__ void __launch_bounds__(128) tern_scan_step_kernel(const __grid_constant__ StepArgs a) {
    using X = Io<T, VEC>;
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int per_row = a.D / VEC;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    const int64_t b = i / per_row;
    if (b >= a.rows) return;
    const int d = static_cast<int>(i - b * per_row) * VEC;
    float f[VEC], v[VEC], r[VEC], y[VEC];
    X::get(X::load(a.f, b * a.f_sb + d), f);
    X::get(X::load(a.v, b * a.v_sb + d), v);
    X::get(X::load(a.r, b * a.r_sb + d), r);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float s, n, o, q;
        gate(f[j] + (a.f_bias != nullptr ? a.f_bias[d + j] : 0.0f), s, n);
        gate(r[j], o, q);
        const float h = fmaf(s, a.h_in[b * a.D + d + j], n * v[j]);
        a.h_out[b * a.D + d + j] = h;
        y[j] = o * h;
    }
    X::store(a.y, b * a.y_sb + d, y);
}

// ------------------------------------------------------------------------------ host side
namespace {

template <class... KArgs, class... Args>
int launch_cluster(void (*kernel)(KArgs...), unsigned grid, unsigned block, unsigned cluster, cudaStream_t s, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    TERN_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...));
    return TERN_OK;
}

size_t elem(int dtype) { return dtype == TERN_F32 ? 4 : 2; }

// TERN_OK when x can be read or written as `rows` of D elements, else the error; vec2 is cleared
// when its address or strides keep it from pairs of elements.
int check_act(const tern_act& x, int dtype, bool& vec2) {
    const size_t es = elem(dtype);
    if (x.p == nullptr || x.stride_b < 0 || x.stride_t < 0) return TERN_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(x.p) % es != 0) return TERN_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(x.p) % (2 * es) != 0 || x.stride_b % 2 != 0 || x.stride_t % 2 != 0) vec2 = false;
    return TERN_OK;
}
Strided strided(const tern_act& x) { return Strided{x.p, x.stride_b, x.stride_t}; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_scan(const tern_scan* s, bool& vec2) {
    if (s == nullptr || (s->dtype != TERN_BF16 && s->dtype != TERN_F32)) return TERN_ERR_ARG;
    if (s->B < 0 || s->T < 0 || s->D < 0 || s->T > INT32_MAX - 256 || s->D > INT32_MAX - 256 || s->B > INT32_MAX - 256) return TERN_ERR_ARG;
    vec2 = s->D % 2 == 0;
    if (s->B == 0 || s->D == 0) return TERN_OK;
    if (s->T > 0) {
        for (const tern_act* x : {&s->f, &s->v, &s->r})
            if (int st = check_act(*x, s->dtype, vec2)) return st;
    }
    if (!aligned4(s->f_bias) || !aligned4(s->lengths)) return TERN_ERR_ALIGN;
    return TERN_OK;
}

// Blocks per cluster: the smallest power of two that gives every SM two blocks, at most
// kMaxCluster and no more than there are steps.
int cluster_size(int64_t blocks, int64_t steps, int num_sms) {
    int S = 1;
    while (S < kMaxCluster && S < steps && blocks * S < 2 * num_sms) S *= 2;
    return S;
}

int64_t steps_of(int64_t T, int64_t rows) { return (T + rows - 1) / rows; }

template <class T, int VEC>
int launch_fwd(const ScanArgs& a0, int64_t B, int num_sms, cudaStream_t s) {
    constexpr int RPT = 16, WARPS = 8;
    ScanArgs a = a0;
    a.tiles = (a.D + 32 * VEC - 1) / (32 * VEC);
    const int64_t blocks = B * a.tiles;
    a.S = cluster_size(blocks, steps_of(a.T, RPT * WARPS), num_sms);
    if (blocks * a.S > INT32_MAX) return TERN_ERR_ARG;
    const unsigned grid = static_cast<unsigned>(blocks * a.S);
    if (a.S > 1) return launch_cluster(tern_scan_fwd_kernel<T, VEC, RPT, WARPS, true>, grid, WARPS * 32, a.S, s, a);
    return launch_cluster(tern_scan_fwd_kernel<T, VEC, RPT, WARPS, false>, grid, WARPS * 32, 1, s, a);
}

template <class T, int VEC>
int launch_bwd(const GradArgs& g0, int64_t B, int num_sms, float* dbias, cudaStream_t s) {
    GradArgs g = g0;
    g.s.tiles = (g.s.D + 32 * VEC - 1) / (32 * VEC);
    const int64_t blocks = B * g.s.tiles;
    g.s.S = cluster_size(blocks, steps_of(g.s.T, kSaveRows), num_sms);
    if (blocks * g.s.S > INT32_MAX) return TERN_ERR_ARG;
    const unsigned grid = static_cast<unsigned>(blocks * g.s.S);
    if (g.s.S > 1) {
        if (int st = launch_cluster(tern_scan_bwd_kernel<T, VEC, true>, grid, 256, g.s.S, s, g)) return st;
    } else if (int st = launch_cluster(tern_scan_bwd_kernel<T, VEC, false>, grid, 256, 1, s, g)) {
        return st;
    }
    if (dbias == nullptr) return TERN_OK;
    return launch_pdl(tern_scan_dbias_kernel, dim3(static_cast<unsigned>((g.s.D + 31) / 32)), dim3(256), 0, s,
                      static_cast<const float*>(g.partial), B * g.s.S, g.s.D, dbias);
}

ScanArgs scan_args(const tern_scan* s) {
    ScanArgs a{};
    a.f = strided(s->f), a.v = strided(s->v), a.r = strided(s->r);
    a.f_bias = s->f_bias, a.lengths = s->lengths, a.starts = s->starts;
    a.T = static_cast<int>(s->T), a.D = static_cast<int>(s->D);
    return a;
}

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" size_t tern_scan_saved(int64_t B, int64_t T, int64_t D) {
    if (B < 0 || T < 0 || D < 0) return 0;
    return static_cast<size_t>(B * steps_of(T, kSaveRows) * D) * sizeof(float);
}

extern "C" int tern_scan_fwd(const tern_scan* s, const float* h0, const tern_act* y, float* hT, float* saved,
                             size_t saved_bytes, void* stream) {
    bool vec2;
    if (int st = check_scan(s, vec2)) return st;
    if (s->B == 0 || s->D == 0) return TERN_OK;
    if (s->T > 0) {
        if (y == nullptr) return TERN_ERR_ARG;
        if (int st = check_act(*y, s->dtype, vec2)) return st;
    }
    if (!aligned4(h0) || !aligned4(hT) || !aligned4(saved)) return TERN_ERR_ALIGN;
    if (saved != nullptr && saved_bytes < tern_scan_saved(s->B, s->T, s->D)) return TERN_ERR_WORKSPACE;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    ScanArgs a = scan_args(s);
    if (s->T > 0) a.y = strided(*y);
    a.saved = saved, a.h_in = h0, a.h_out = hT;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (s->dtype == TERN_BF16)
        return vec2 ? launch_fwd<__nv_bfloat16, 2>(a, s->B, num_sms, cs) : launch_fwd<__nv_bfloat16, 1>(a, s->B, num_sms, cs);
    return vec2 ? launch_fwd<float, 2>(a, s->B, num_sms, cs) : launch_fwd<float, 1>(a, s->B, num_sms, cs);
}

extern "C" size_t tern_scan_bwd_workspace(int64_t B, int64_t T, int64_t D) {
    if (B < 0 || T < 0 || D < 0) return 0;
    return static_cast<size_t>(B * kMaxCluster * D) * sizeof(float);   // the blocks' sums of df
}

extern "C" int tern_scan_bwd(const tern_scan* s, const float* saved, const tern_act* dy, const float* dhT,
                             const tern_act* df, const tern_act* dv, const tern_act* dr, float* dbias, float* dh0,
                             void* workspace, size_t ws_bytes, void* stream) {
    bool vec2;
    if (int st = check_scan(s, vec2)) return st;
    if (s->B == 0 || s->D == 0) return s->D == 0 || dbias == nullptr ? TERN_OK : TERN_ERR_ARG;
    if (s->T > 0) {
        if (saved == nullptr) return TERN_ERR_ARG;
        for (const tern_act* x : {dy, df, dv, dr}) {
            if (x == nullptr) return TERN_ERR_ARG;
            if (int st = check_act(*x, s->dtype, vec2)) return st;
        }
    }
    if (!aligned4(saved) || !aligned4(dhT) || !aligned4(dbias) || !aligned4(dh0) || !aligned4(workspace)) return TERN_ERR_ALIGN;
    if (dbias != nullptr && (workspace == nullptr || ws_bytes < tern_scan_bwd_workspace(s->B, s->T, s->D)))
        return TERN_ERR_WORKSPACE;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    GradArgs g{};
    g.s = scan_args(s);
    g.s.saved = const_cast<float*>(saved), g.s.h_in = dhT, g.s.h_out = dh0;
    if (s->T > 0) g.s.y = strided(*dy), g.df = strided(*df), g.dv = strided(*dv), g.dr = strided(*dr);
    g.partial = dbias != nullptr ? static_cast<float*>(workspace) : nullptr;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (s->dtype == TERN_BF16)
        return vec2 ? launch_bwd<__nv_bfloat16, 2>(g, s->B, num_sms, dbias, cs) : launch_bwd<__nv_bfloat16, 1>(g, s->B, num_sms, dbias, cs);
    return vec2 ? launch_bwd<float, 2>(g, s->B, num_sms, dbias, cs) : launch_bwd<float, 1>(g, s->B, num_sms, dbias, cs);
}

namespace {
template <class T>
int launch_step(const StepArgs& a, bool vec2, cudaStream_t s) {
    const int64_t blocks = (a.rows * (vec2 ? a.D / 2 : a.D) + 127) / 128;
    if (blocks > INT32_MAX) return TERN_ERR_ARG;
    return launch_pdl(vec2 ? tern_scan_step_kernel<T, 2> : tern_scan_step_kernel<T, 1>, dim3(static_cast<unsigned>(blocks)),
                      dim3(128), 0, s, a);
}
}  // namespace

extern "C" int tern_scan_step(const tern_scan* s, const float* h_in, float* h_out, const tern_act* y, void* stream) {
    bool vec2;
    if (int st = check_scan(s, vec2)) return st;
    if (s->T != 1 || s->lengths != nullptr || s->starts != nullptr) return TERN_ERR_ARG;
    if (s->B == 0 || s->D == 0) return TERN_OK;
    if (h_in == nullptr || h_out == nullptr || y == nullptr) return TERN_ERR_ARG;
    if (int st = check_act(*y, s->dtype, vec2)) return st;
    if (!aligned4(h_in) || !aligned4(h_out)) return TERN_ERR_ALIGN;
    if (int st = check_device(nullptr)) return st;
    StepArgs a{};
    a.f = s->f.p, a.v = s->v.p, a.r = s->r.p, a.y = y->p;
    a.f_sb = s->f.stride_b, a.v_sb = s->v.stride_b, a.r_sb = s->r.stride_b, a.y_sb = y->stride_b;
    a.f_bias = s->f_bias, a.h_in = h_in, a.h_out = h_out;
    a.rows = s->B, a.D = static_cast<int>(s->D);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return s->dtype == TERN_BF16 ? launch_step<__nv_bfloat16>(a, vec2, cs) : launch_step<float>(a, vec2, cs);
}
