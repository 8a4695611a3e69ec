// Gated linear recurrence over sequences, its gradient, and its single-token step.
//
//   a_t = sigmoid(f_t + bias), h_t = a_t h_{t-1} + (1 - a_t) v_t, y_t = sigmoid(r_t) h_t
//
// per sequence b and channel d; h_{t-1} is read as 0 at a document start, and rows at or past
// lengths[b] are padding (a = 1, no input, y = 0, gradients 0; their values are never used, though
// copies by TMA bring those of a sequence's last live step along).
//
// The map of one row, h -> a h + b, composes: rows i..j act as h -> A h + H with A = prod a and
// H the state reached from 0.  A block takes a tile of channels and ROWS consecutive rows: a lane
// has four neighbouring channels (two in fp32) of RPT rows, a segment; LPR lanes side by side make
// a row's 64 bytes (32 in narrow tiles), and a warp holds 32/LPR segments.
//   1. each lane folds its RPT rows into (A, H); a warp's segments are joined by shuffles and
//      its pair left in shared memory;
//   2. after a barrier each lane folds what lies before it onto the block's incoming state;
//   3. it runs its rows again from that state, whose gates it kept in registers, and writes y.
// A block walks T in steps of ROWS, its inputs copied one step ahead by TMA.  Where sequences times
// channel tiles are too few blocks to fill the GPU, a cluster of S blocks takes S consecutive steps
// at a time, and each block pushes its total into the others' shared memory (a cluster barrier
// would wait for the block's stores each step: 414 against 165 us for a document of 65536).  Every
// fold has a fixed order, so results do not depend on the schedule.
//
// The gradient runs the same way from the end of the sequence, with e_t = a_t dh_t as its state:
//   dh_t = g_t + e_{t+1}, e_t = a_t dh_t, g_t = sigmoid(r_t) dy_t, e_T = dhT
//   dv = (1 - a) dh, df = dh (h_{t-1} - v) a (1 - a), dr = dy h s (1 - s), dh0 = e_0
// and recomputes h from the states the forward saved every 64 rows (1/8 B per element beside the
// 22 B of a forward and a gradient in bf16).
//
// HBM would allow 8 B per element in the forward and 14 B in the gradient (each input read once,
// each output written once).  8 x 2048 x 2048 in bf16 with packed documents: forward 59 us, 0.67 of
// the measured copy rate, gradient 127 us, 0.55; without documents 53 and 120 us; in fp32 86 us, 0.92, and
// 173 us, 0.80.  What binds in bf16 is latency, no unit: 31 and 72 instructions per element and lane, of
// which 17 and 32 are the arithmetic, take 48% and 54% of the issue slots, and DRAM is busy 51% and 43% of
// the time.  Of four warps on a scheduler, each on its own chain of exponential, reciprocal and fold, 1.6
// and 1.4 wait for a result of fixed latency when one issues, 1.3 and 1.4 for a global load (the start
// bytes and the gradient's saved states, loaded in the step that uses them), 0.8 and 0.4 for shared memory
// or a special function.  More warps with fewer rows each lost more to the folds than they hid (RPT 4: 77
// us), fewer with more rows hid less.  Gates and states are fp32; outputs are rounded once.
#include <algorithm>
#include <type_traits>
#include <utility>

#include <cuda_bf16.h>

#include "mma.cuh"
#include "pairs.cuh"

namespace tern {
namespace {

constexpr int kSaveRows = 64;     // rows between saved states
constexpr int kMaxCluster = 16;   // blocks of a cluster

__device__ int g_scan_status;     // 1 once a wait for a peer's totals gave up

__device__ __forceinline__ F2 shfl2(F2 a, int from) { return F2{__shfl_sync(0xffffffffu, a.v, from)}; }

// --------------------------------------------------------------- element access
// NP pairs of neighbouring elements of a row, eight bytes.  W is the alignment of every row, in
// bytes.  16 (WIDE): one access, and the sequences' inputs come by TMA.  Otherwise (odd widths,
// strides or addresses) words of W bytes, where a row's last lane may hold fewer elements: nch
// are there, loads repeat a word that is and stores leave the others out.  (8 x 2048 x D in bf16, the
// forward and the gradient: D = 1024 31 + 65 us; 1026 39 + 84, element by element 73 + 168; 1025 55 +
// 129, with the words around a lane's elements where all of them are in the tensor.  In fp32 1024 44 + 91,
// 1025 55 + 141.)
template <class T, int W>
struct Io;
template <int W_>
struct Io<__nv_bfloat16, W_> {
    static constexpr int W = W_;
    static constexpr bool WIDE = W == 16;
    static constexpr int NP = 2;
    using Raw = uint2;
    static __device__ __forceinline__ Raw load(const char* p, int nch) {
        if constexpr (W == 16) {
            return __ldg(reinterpret_cast<const uint2*>(p));
        } else if constexpr (W == 4) {   // nch is even
            const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
            return make_uint2(__ldg(q), __ldg(q + (nch > 2 ? 1 : 0)));
        } else {
            const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
            const uint32_t x0 = __ldg(q), x1 = __ldg(q + min(1, nch - 1)), x2 = __ldg(q + min(2, nch - 1)), x3 = __ldg(q + min(3, nch - 1));
            return make_uint2(x0 | x1 << 16, x2 | x3 << 16);
        }
    }
    // W = 2, four elements with the words around them all in the tensor: two or three words, shifted.
    static __device__ __forceinline__ Raw load_words(const char* p) {
        const uint32_t odd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 2u;
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p - odd);
        const uint32_t w0 = __ldg(q), w1 = __ldg(q + 1);
        uint32_t w2 = 0u;
        if (odd) w2 = __ldg(q + 2);
        return make_uint2(__funnelshift_r(w0, w1, odd * 8), __funnelshift_r(w1, w2, odd * 8));
    }
    static __device__ __forceinline__ void get(const Raw& r, F2 (&x)[2]) {
        x[0] = pair(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u));
        x[1] = pair(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t round2(F2 a) {
        float x, y;
        split(a, x, y);
        const __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&t);
    }
    static __device__ __forceinline__ void store(char* p, const F2 (&x)[2], int nch) {
        const uint32_t a = round2(x[0]), b = round2(x[1]);
        if constexpr (W == 16) {
            *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
        } else if constexpr (W == 4) {
            uint32_t* q = reinterpret_cast<uint32_t*>(p);
            q[0] = a;
            if (nch > 2) q[1] = b;
        } else {
            unsigned short* q = reinterpret_cast<unsigned short*>(p);
            if (nch < 4) {
                q[0] = static_cast<unsigned short>(a);
                if (nch > 1) q[1] = static_cast<unsigned short>(a >> 16);
                if (nch > 2) q[2] = static_cast<unsigned short>(b);
            } else if (reinterpret_cast<uintptr_t>(p) & 2) {
                q[0] = static_cast<unsigned short>(a);
                *reinterpret_cast<uint32_t*>(q + 1) = __funnelshift_r(a, b, 16);
                q[3] = static_cast<unsigned short>(b >> 16);
            } else {
                reinterpret_cast<uint32_t*>(p)[0] = a;
                reinterpret_cast<uint32_t*>(p)[1] = b;
            }
        }
    }
};
template <int W_>
struct Io<float, W_> {
    static constexpr int W = W_;
    static constexpr bool WIDE = W == 16;
    static constexpr int NP = 1;
    using Raw = float2;
    static __device__ __forceinline__ Raw load(const char* p, int nch) {
        if constexpr (WIDE) return __ldg(reinterpret_cast<const float2*>(p));
        const float* q = reinterpret_cast<const float*>(p);
        return make_float2(__ldg(q), __ldg(q + min(1, nch - 1)));
    }
    static __device__ __forceinline__ void get(const Raw& r, F2 (&x)[1]) { x[0] = pair(r.x, r.y); }
    static __device__ __forceinline__ void store(char* p, const F2 (&x)[1], int nch) {
        float a, b;
        split(x[0], a, b);
        if constexpr (WIDE) {
            *reinterpret_cast<float2*>(p) = make_float2(a, b);
        } else {
            reinterpret_cast<float*>(p)[0] = a;
            if (nch > 1) reinterpret_cast<float*>(p)[1] = b;
        }
    }
};
// fp32 values of a lane's channels in arrays [..][D] (bias, states); nch as above.
template <int NP>
__device__ __forceinline__ void load_f32(const float* p, int nch, F2 (&x)[NP], float none) {
#pragma unroll
    for (int j = 0; j < NP; ++j)
        x[j] = p == nullptr ? both(none) : pair(p[min(2 * j, nch - 1)], p[min(2 * j + 1, nch - 1)]);
}
template <int NP>
__device__ __forceinline__ void store_f32(float* p, int nch, const F2 (&x)[NP]) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        float a, b;
        split(x[j], a, b);
        if (2 * j < nch) p[2 * j] = a;
        if (2 * j + 1 < nch) p[2 * j + 1] = b;
    }
}

// s = sigmoid(x + bias) and n = 1 - s = sigmoid(-x - bias), to about 4 + |x + bias| units of 2^-24 relative
// for the smaller of the two (the exponent is rounded once: 6 units up to 4, 17 up to 16, 65 at the cap, with
// an exact exponential), a few for the larger; the approximate exponential and reciprocal add two or three.
// n is not formed as 1 - s, which loses it where s is near 1.  `lb` is -bias * log2(e).
// e = exp(-(x + bias)) is capped at 2^125 so that s and e*s stay normal numbers: for arguments
// below -86 (-inf included) s is 2^-125 and n is 1.  A NaN stays one.  The approximate
// exponential and reciprocal are taken without their subnormal paths, which the cap rules out
// and which flush an s or n below 2^-126 to 0.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ F2 exp2_capped(F2 t) {
    float x, y;
    split(t, x, y);
    asm("min.NaN.f32 %0, %1, 0f42FA0000;" : "=f"(x) : "f"(x));
    asm("min.NaN.f32 %0, %1, 0f42FA0000;" : "=f"(y) : "f"(y));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(y));
    return pair(x, y);
}
__device__ __forceinline__ F2 rcp_neg(F2 u) {   // -1 / u
    float x, y;
    split(u, x, y);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(-x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-y));
    return pair(x, y);
}
__device__ __forceinline__ F2 gate(F2 x) {   // s alone: an infinite e gives 0
    float a, b;
    split(mul2(x, both(-kLog2e)), a, b);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(a));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(b));
    return rcp_neg(fma2(pair(a, b), both(-1.0f), both(-1.0f)));
}
__device__ __forceinline__ void gate(F2 x, F2& s, F2& n) {
    const F2 e = exp2_capped(mul2(x, both(-kLog2e)));
    s = rcp_neg(fma2(e, both(-1.0f), both(-1.0f)));
    n = mul2(e, s);
}
// The same for the gate whose products run over thousands of rows, with one step of Newton's
// method on the reciprocal: near 1 its last place is twice what rounding leaves.
__device__ __forceinline__ void decay(F2 x, F2 lb, F2& s, F2& n) {
    const F2 e = exp2_capped(fma2(x, both(-kLog2e), lb));
    const F2 u = fma2(e, both(-1.0f), both(-1.0f));   // -(1 + e)
    s = rcp_neg(u);
    s = fma2(s, fma2(u, s, both(1.0f)), s);
    n = mul2(e, s);
}

// A row map whose A carries the sign bit ignores the state before it (a document start lies in
// its rows): -0 keeps its sign through products with the a >= 0 of later rows, and no value of
// an earlier document, NaN included, passes.  docs: whether there are any.
__device__ __forceinline__ F2 where_cut(F2 A, F2 yes, F2 no) {
    float a, b, x, y, z, w;
    split(A, a, b);
    split(yes, x, y);
    split(no, z, w);
    return pair((__float_as_uint(a) >> 31) != 0 ? x : z, (__float_as_uint(b) >> 31) != 0 ? y : w);
}
__device__ __forceinline__ F2 apply(F2 A, F2 H, F2 h, bool docs) {
    const F2 x = fma2(A, h, H);
    return docs ? where_cut(A, H, x) : x;
}
// (A, H) := the map (A2, H2) after (A, H).  A NaN in A2 takes the sign that A carries; the gradient, whose
// maps run backwards to the documents before, keeps NaN out of A for that (without_nan).
__device__ __forceinline__ void compose(F2 A2, F2 H2, F2& A, F2& H, bool docs) {
    H = apply(A2, H2, H, docs);
    A = docs ? where_cut(A2, A2, mul2(A, A2)) : mul2(A, A2);
}

// A >= 0 with 0 in the place of a NaN.  A row whose gate is NaN has NaN in H and in G too, so A need not
// carry it; as a factor it would undo the mark of a document start on an earlier row.
__device__ __forceinline__ F2 without_nan(F2 A) {
    float x, y;
    split(A, x, y);
    return pair(fmaxf(x, 0.0f), fmaxf(y, 0.0f));
}

struct Strided {
    char* p;
    int64_t sb, st;   // bytes between sequences and between rows
    char* end;        // past the last row's last element
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
    CUtensorMap maps[4];  // WIDE: f, v, r and dy
};
struct GradArgs {
    ScanArgs s;
    Strided df, dv, dr;
    float* partial;       // [B*S][D] sums of df, or null
};

// How a block cuts its rows and channels: LPR lanes make a row of CH channels, a lane's segment
// has RPT rows, a warp SEGS segments.
template <class T_, int W, int LPR_, int RPT_, int WARPS_, int MINB_, int STAGES_>
struct Shape {
    using T = T_;
    using X = Io<T_, W>;
    static constexpr int NP = X::NP, LPR = LPR_, RPT = RPT_;
    static constexpr int WARPS = WARPS_, MINB = MINB_, STAGES = STAGES_, SEGS = 32 / LPR, CH = LPR * NP * 2, WROWS = SEGS * RPT, ROWS = WARPS * WROWS;
};

// Totals of the S blocks of a cluster, pushed by each block into every block's shared memory
// (st.async) and counted there on an mbarrier: two of each in turn.  One warp sends, waits and folds
// (all of them reading the same totals would take the shared memory's bandwidth) and hands the state
// before the block's rows to the others.  It sends the totals of iteration i+1 only after it has read
// those of i, and i+2 needs everyone's i+1, so a buffer is read before it is written again.
template <class C>
struct Exchange {
    alignas(16) float A[2][kMaxCluster][C::CH], H[2][kMaxCluster][C::CH];
    uint64_t bar[2];
};
// A block may leave once its last wait has succeeded: all that its peers send has arrived, and
// what it sent is what they wait for.  After a wait that gave up nothing is known, and the thread
// stays until the peers' threads have left or come here too.
template <class E>
__device__ __forceinline__ void open_exchange(E& ex) {
    if (threadIdx.x == 0) {
        ptx::mbar_init(ptx::smem_u32(&ex.bar[0]), 1);
        ptx::mbar_init(ptx::smem_u32(&ex.bar[1]), 1);
        ptx::fence_mbar_init();
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_leave() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
template <int NP>
__device__ __forceinline__ void push_pairs(const float* mine, const F2 (&x)[NP], const uint64_t* bar, uint32_t rank) {
    const uint32_t at = ptx::mapa_shared(ptx::smem_u32(mine), rank), b = ptx::mapa_shared(ptx::smem_u32(bar), rank);
    if constexpr (NP == 2) {
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(at),
                     "l"(x[0].v), "l"(x[1].v), "r"(b) : "memory");
    } else {
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(at), "l"(x[0].v), "r"(b)
                     : "memory");
    }
}
// Waits for a phase of the exchange or of a copy, at most about two seconds: a peer block is
// resident, a copy on its way, and a healthy wait takes microseconds.  On expiry the status word is
// set; the thread waits no more and runs its steps to the end, so that the block's barriers still
// match (its results are void).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
    const uint32_t b = ptx::smem_u32(bar);
    uint64_t last = 0, waited = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(b), "r"(parity) : "memory");
        if (ok) return true;
        if ((it & 63u) == 63u) {
            const uint64_t now = ptx::globaltimer();
            // forward steps of the timer, each counted up to 1 ms, as in the GEMMs' waits
            const int64_t step = last == 0 ? 0 : static_cast<int64_t>(now - last);
            last = now;
            if (step > 0) waited += static_cast<uint64_t>(step < 1000000 ? step : 1000000);
            if (waited > 2000000000ull || it >= (1u << 30)) {
                atomicExch(&g_scan_status, 1);
                return false;
            }
        }
    }
}
// The last of a thread whose wait gave up (none of the block's barriers follows: the others do not come
// here).  Copies that are still on their way get time to land before the block leaves its shared memory.
template <bool CL>
__device__ __forceinline__ void leave_late() {
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t i = 0; i < (1u << 24) && ptx::globaltimer() - t0 < 100000ull; ++i) {
    }
    if constexpr (CL) cluster_leave();
}

__device__ __forceinline__ int rows_live(const ScanArgs& a, int b) {
    return a.lengths != nullptr ? min(max(a.lengths[b], 0), a.T) : a.T;
}
// bit i: row i of this lane's segment (live) starts a document; a lane of the warp reads each row's
// byte, or two of them.
template <class C>
__device__ __forceinline__ uint32_t start_bits(const ScanArgs& a, int64_t b, int warp_row0, int len, int seg, int lane) {
    static_assert(C::WROWS == 16 || C::WROWS == 32 || C::WROWS == 64, "whole bytes of rows per lane");
    if (a.starts == nullptr) return 0;
    const uint8_t* p = a.starts + b * a.T + warp_row0;
    auto vote = [&](int r) { return __ballot_sync(0xffffffffu, r < C::WROWS && warp_row0 + r < len && p[r] != 0); };
    const uint32_t lo = vote(lane), hi = C::WROWS > 32 ? vote(lane + 32) : 0u;
    const int at = seg * C::RPT;
    return ((at < 32 ? lo : hi) >> (at & 31)) & ((1u << C::RPT) - 1u);
}
// A step's inputs: NT tensors of ROWS rows by CH channels.  WIDE: copied by TMA into a ring of
// STAGES tiles in shared memory, ahead of their use, where a lane reads its eight bytes of a row at
// constant offsets; otherwise loaded into registers by the lanes that use them.
template <class C, int NT>
struct Inputs {
    static constexpr bool WIDE = C::X::WIDE;
    static constexpr int ROW_BYTES = C::CH * static_cast<int>(sizeof(typename C::T)), TILE_BYTES = C::ROWS * ROW_BYTES;
    static constexpr int SMEM = WIDE ? C::STAGES * NT * TILE_BYTES + 128 : 0;
    using Raw = typename C::X::Raw;
    Raw raw[WIDE ? 1 : NT][WIDE ? 1 : C::RPT];
    const char* at;   // WIDE: this lane's bytes of its segment's first row, in the current stage's first tensor

    __device__ __forceinline__ Raw get(int t, int i) const {
        if constexpr (WIDE) return *reinterpret_cast<const Raw*>(at + t * TILE_BYTES + i * ROW_BYTES);
        else return raw[t][i];
    }
    // The rows of tensor t; those that are not live stay zero.
    __device__ __forceinline__ void load(int t, const Strided& x, const char* p, int nl, int nch, bool full) {
        if constexpr (!WIDE) {
            const int64_t st = x.st;
            if constexpr (C::X::W == 2) {   // but for the tensor's first and last row the words around a lane's elements are its own
                if (__all_sync(0xffffffffu, full && nch == 2 * C::NP && p - 2 >= x.p && p + (C::RPT - 1) * st + 10 <= x.end)) {
#pragma unroll
                    for (int i = 0; i < C::RPT; ++i) raw[t][i] = C::X::load_words(p + i * st);
                    return;
                }
            }
            if (full && nch == 2 * C::NP) {   // all there: offsets known to the compiler
#pragma unroll
                for (int i = 0; i < C::RPT; ++i) raw[t][i] = C::X::load(p + i * st, 2 * C::NP);
            } else {
#pragma unroll
                for (int i = 0; i < C::RPT; ++i) {
                    raw[t][i] = Raw{};
                    if (i < nl) raw[t][i] = C::X::load(p + i * st, nch);
                }
            }
        }
    }
};
// One step's tiles: rows from step * ROWS on of sequence b, channels from ch0 on (one thread).
// What lies past the last row or channel arrives as zeros.
template <class C, int NT>
__device__ __forceinline__ void copy_step(const CUtensorMap* maps, uint32_t stage, uint32_t bar, int ch0, int64_t step, int b) {
    using I = Inputs<C, NT>;
    ptx::mbar_arrive_expect_tx(bar, NT * I::TILE_BYTES);
#pragma unroll
    for (int t = 0; t < NT; ++t)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(stage + t * I::TILE_BYTES),
            "l"(reinterpret_cast<uint64_t>(maps + t)), "r"(ch0), "r"(static_cast<int>(step * C::ROWS)), "r"(b), "r"(bar)
            : "memory");
}
// Within a warp, in log2(SEGS) exchanges: (PA, PH) = the map of the segments before this one, (A, H) that
// of all of them; and for the gradient (QA, QG) = the map, run backwards, of the segments after it, (A, G)
// that of all of them.  A, H and G come as the segment's own.
template <class C, bool GRAD>
__device__ __forceinline__ void warp_prefix(F2 (&A)[C::NP], F2 (&H)[C::NP], F2 (&G)[C::NP], F2 (&PA)[C::NP], F2 (&PH)[C::NP],
                                            F2 (&QA)[C::NP], F2 (&QG)[C::NP], int seg, int lane, bool docs) {
#pragma unroll
    for (int j = 0; j < C::NP; ++j) {
        PA[j] = both(1.0f), PH[j] = both(0.0f);
        if constexpr (GRAD) QA[j] = both(1.0f), QG[j] = both(0.0f);
#pragma unroll
        for (int d = 1; d < C::SEGS; d <<= 1) {
            const bool later = (seg & d) != 0;
            const int from = lane ^ (d * C::LPR);
            const F2 A2 = shfl2(A[j], from), H2 = shfl2(H[j], from);
            if constexpr (GRAD) {
                const F2 G2 = shfl2(G[j], from);
                if (later) {
                    F2 a = A[j], g = G[j];
                    compose(A2, G2, a, g, docs);   // backwards this half runs first
                    G[j] = g;
                } else {
                    F2 a = A2, g = G2;
                    compose(QA[j], QG[j], a, g, docs);
                    QA[j] = a, QG[j] = g;
                    a = A2, g = G2;
                    compose(A[j], G[j], a, g, docs);
                    G[j] = g;
                }
            }
            if (later) {
                F2 a = A2, h = H2;
                compose(PA[j], PH[j], a, h, docs);
                PA[j] = a, PH[j] = h;
                a = A2, h = H2;
                compose(A[j], H[j], a, h, docs);
                A[j] = a, H[j] = h;
            } else {
                compose(A2, H2, A[j], H[j], docs);
            }
        }
    }
}
// Pairs in shared memory: a lane's channels of one row of an [..][CH] array.
template <int NP>
__device__ __forceinline__ void get_s(const float* p, F2 (&x)[NP]) {
    if constexpr (NP == 2) {
        const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p);
        x[0].v = t.x, x[1].v = t.y;
    } else {
        x[0].v = *reinterpret_cast<const unsigned long long*>(p);
    }
}
template <int NP>
__device__ __forceinline__ void put_s(float* p, const F2 (&x)[NP]) {
    if constexpr (NP == 2) *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x[0].v, x[1].v);
    else *reinterpret_cast<unsigned long long*>(p) = x[0].v;
}
// h := the maps at A, H (rows `stride` floats apart) k0, k0 + dk, ... up to but without k1, after h
template <int NP>
__device__ __forceinline__ void fold(const float* A, const float* H, int stride, int k0, int k1, int dk, F2 (&h)[NP], bool docs) {
#pragma unroll 4
    for (int k = k0; k != k1; k += dk) {
        F2 Ak[NP], Hk[NP];
        get_s(A + k * stride, Ak);
        get_s(H + k * stride, Hk);
#pragma unroll
        for (int j = 0; j < NP; ++j) h[j] = apply(Ak[j], Hk[j], h[j], docs);
    }
}
// The same as one map: (PA, PH) := the maps at A, H after (PA, PH)
template <int NP>
__device__ __forceinline__ void fold_map(const float* A, const float* H, int stride, int k0, int k1, int dk, F2 (&PA)[NP],
                                         F2 (&PH)[NP], bool docs) {
#pragma unroll
    for (int k = k0; k != k1; k += dk) {
        F2 Ak[NP], Hk[NP];
        get_s(A + k * stride, Ak);
        get_s(H + k * stride, Hk);
#pragma unroll
        for (int j = 0; j < NP; ++j) compose(Ak[j], Hk[j], PA[j], PH[j], docs);
    }
}

// The parts of a step that run over a segment's rows.  PLAIN: all rows of the warp are live and
// none starts a document, which leaves out the selects.
template <class C, bool PLAIN>
__device__ __forceinline__ void fwd_rows(const Inputs<C, 3>& in, const F2 (&lb)[C::NP], int nl, uint32_t cut, F2 (&ga)[C::RPT][C::NP],
                                         F2 (&gb)[C::RPT][C::NP], F2 (&A)[C::NP], F2 (&H)[C::NP]) {
#pragma unroll
    for (int i = 0; i < C::RPT; ++i) {
        F2 f[C::NP], v[C::NP], n;
        C::X::get(in.get(0, i), f);
        C::X::get(in.get(1, i), v);
#pragma unroll
        for (int j = 0; j < C::NP; ++j) {
            decay(f[j], lb[j], ga[i][j], n);
            gb[i][j] = mul2(n, v[j]);
            if constexpr (!PLAIN) {
                if (i >= nl) ga[i][j] = both(1.0f), gb[i][j] = both(0.0f);
                if ((cut >> i) & 1u) ga[i][j] = both(-0.0f);
            }
            if (i == 0) A[j] = ga[i][j], H[j] = gb[i][j];
            else compose(ga[i][j], gb[i][j], A[j], H[j], !PLAIN);
        }
    }
}
// gb becomes the states; h the state after the rows.
template <class C, bool PLAIN>
__device__ __forceinline__ void fwd_again(const F2 (&ga)[C::RPT][C::NP], F2 (&gb)[C::RPT][C::NP], F2 (&h)[C::NP]) {
#pragma unroll
    for (int i = 0; i < C::RPT; ++i)
#pragma unroll
        for (int j = 0; j < C::NP; ++j) gb[i][j] = h[j] = apply(ga[i][j], gb[i][j], h[j], !PLAIN);
}
template <class C, bool PLAIN>
__device__ __forceinline__ void fwd_store(const Inputs<C, 3>& in, const F2 (&hs)[C::RPT][C::NP], char* y, int64_t st,
                                          int nl, int nr, int nch) {
#pragma unroll
    for (int i = 0; i < C::RPT; ++i) {
        F2 r[C::NP], o[C::NP];
        C::X::get(in.get(2, i), r);
#pragma unroll
        for (int j = 0; j < C::NP; ++j) {
            o[j] = mul2(gate(r[j]), hs[i][j]);
            if (!PLAIN && i >= nl) o[j] = both(0.0f);
        }
        if (PLAIN ? nr > 0 : i < nr) C::X::store(y + i * st, o, nch);
    }
}
// Per row: s = a, n = 1 - a, o = sigmoid(r) dy, x = sigmoid(-r); and the segment's folds.
template <class C, bool PLAIN>
__device__ __forceinline__ void bwd_rows(const Inputs<C, 4>& in, const F2 (&lb)[C::NP], int nl, uint32_t cut, F2 (&s)[C::RPT][C::NP],
                                         F2 (&n)[C::RPT][C::NP], F2 (&o)[C::RPT][C::NP], F2 (&x)[C::RPT][C::NP],
                                         F2 (&A)[C::NP], F2 (&H)[C::NP], F2 (&G)[C::NP]) {
#pragma unroll
    for (int i = 0; i < C::RPT; ++i) {
        F2 f[C::NP], v[C::NP], r[C::NP], dy[C::NP], so;
        C::X::get(in.get(0, i), f);
        C::X::get(in.get(1, i), v);
        C::X::get(in.get(2, i), r);
        C::X::get(in.get(3, i), dy);
#pragma unroll
        for (int j = 0; j < C::NP; ++j) {
            decay(f[j], lb[j], s[i][j], n[i][j]);
            gate(r[j], so, x[i][j]);
            o[i][j] = mul2(so, dy[j]);
            if (!PLAIN && i >= nl) s[i][j] = both(1.0f), n[i][j] = both(0.0f), o[i][j] = both(0.0f);
            const F2 b = mul2(n[i][j], v[j]);
            F2 m = s[i][j];
            if constexpr (!PLAIN) m = (cut >> i) & 1u ? both(-0.0f) : without_nan(m);
            if (i == 0) A[j] = m, H[j] = b;
            else compose(m, b, A[j], H[j], !PLAIN);
        }
    }
    if constexpr (PLAIN) {
#pragma unroll
        for (int j = 0; j < C::NP; ++j) A[j] = without_nan(A[j]);
    }
#pragma unroll
    for (int i = C::RPT - 1; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < C::NP; ++j) {
            G[j] = mul2(s[i][j], i == C::RPT - 1 ? o[i][j] : add2(o[i][j], G[j]));
            if (!PLAIN && ((cut >> i) & 1u)) G[j] = both(0.0f);
        }
}
// From h before the rows and e after them: the gradients, written; e before the rows.
template <class C, bool PLAIN>
__device__ __forceinline__ void bwd_store(const Inputs<C, 4>& in, const F2 (&s)[C::RPT][C::NP],
                                          const F2 (&n)[C::RPT][C::NP], const F2 (&o)[C::RPT][C::NP], F2 (&x)[C::RPT][C::NP],
                                          int nl, uint32_t cut, int nr, int nch, F2 (&h)[C::NP], F2 (&e)[C::NP],
                                          F2 (&dbias)[C::NP], char* df_p, int64_t df_st, char* dv_p, int64_t dv_st, char* dr_p,
                                          int64_t dr_st) {
    F2 hv[C::RPT][C::NP];   // n (h_{t-1} - v); x becomes dr = g h (1 - sigmoid(r))
#pragma unroll
    for (int i = 0; i < C::RPT; ++i) {
        F2 v[C::NP];
        C::X::get(in.get(1, i), v);
#pragma unroll
        for (int j = 0; j < C::NP; ++j) {
            if (!PLAIN && ((cut >> i) & 1u)) h[j] = both(0.0f);
            hv[i][j] = mul2(n[i][j], fma2(v[j], both(-1.0f), h[j]));
            h[j] = fma2(s[i][j], h[j], mul2(n[i][j], v[j]));
            x[i][j] = mul2(mul2(o[i][j], h[j]), x[i][j]);
        }
    }
#pragma unroll
    for (int i = C::RPT - 1; i >= 0; --i) {
        F2 df[C::NP], dv[C::NP];
#pragma unroll
        for (int j = 0; j < C::NP; ++j) {
            const F2 dh = add2(o[i][j], e[j]);
            e[j] = mul2(s[i][j], dh);
            dv[j] = mul2(n[i][j], dh);
            df[j] = mul2(e[j], hv[i][j]);
            if (!PLAIN && i >= nl) dv[j] = df[j] = x[i][j] = both(0.0f);
            dbias[j] = add2(dbias[j], df[j]);
            if (!PLAIN && ((cut >> i) & 1u)) e[j] = both(0.0f);
        }
        if (PLAIN ? nr > 0 : i < nr) {
            C::X::store(df_p + i * df_st, df, nch);
            C::X::store(dv_p + i * dv_st, dv, nch);
            C::X::store(dr_p + i * dr_st, x[i], nch);
        }
    }
}
// The block barrier after which `agg` holds; whether a document starts in any of its rows.
__device__ __forceinline__ bool sync_cuts(bool docs, uint32_t cut) {
    if (docs) return __syncthreads_or(cut != 0) != 0;
    __syncthreads();
    return false;
}

// What every block of the two kernels starts from.
template <class C>
struct Place {
    int w, lane, seg, c, ch, rank, d0, d, nch;
    int64_t b;
    bool on;      // this lane has channels; the others repeat the row's last and store nothing
    __device__ __forceinline__ explicit Place(const ScanArgs& a) {
        w = threadIdx.x >> 5, lane = threadIdx.x & 31;
        seg = lane / C::LPR, c = lane % C::LPR, ch = c * C::NP * 2;
        const int cl = blockIdx.x / a.S;
        rank = blockIdx.x - cl * a.S;
        b = cl / a.tiles;
        d0 = (cl - static_cast<int>(b) * a.tiles) * C::CH + ch;
        on = d0 < a.D;
        d = on ? d0 : max(a.D - C::NP * 2, 0);
        nch = C::X::WIDE ? C::NP * 2 : min(a.D - d, C::NP * 2);
    }
    __device__ __forceinline__ char* at(const Strided& x) const {
        return x.p + b * x.sb + static_cast<int64_t>(d) * static_cast<int64_t>(sizeof(typename C::T));
    }
};

}  // namespace

// ------------------------------------------------------------------------------ forward
// CL: the S blocks of a cluster take S consecutive steps at a time; otherwise S is 1.
template <class C, bool CL>
__global__ void __launch_bounds__(C::WARPS * 32, C::MINB) tern_scan_fwd_kernel(const __grid_constant__ ScanArgs a) {
    using X = typename C::X;
    constexpr int NP = C::NP, RPT = C::RPT, WARPS = C::WARPS, ROWS = C::ROWS;
    constexpr int LEAD = WARPS - 1;   // the warp that exchanges totals with the cluster's other blocks
    static_assert(kSaveRows % RPT == 0, "saved states fall on segment boundaries");
    extern __shared__ __align__(128) char smem[];
    __shared__ uint64_t full[C::STAGES];
    __shared__ alignas(16) float aggA[2][WARPS][C::CH], aggH[2][WARPS][C::CH];
    __shared__ alignas(16) float carry_s[2][C::CH];                // the state after a step (CL: before the block's)
    __shared__ typename std::conditional<CL, Exchange<C>, int>::type ex;
    const Place<C> q(a);
    if constexpr (C::X::WIDE) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < C::STAGES; ++i) ptx::mbar_init(ptx::smem_u32(&full[i]), 1);
            ptx::fence_mbar_init();
        }
    }
    if constexpr (CL) open_exchange(ex);
    ptx::pdl_wait();
    const bool docs = a.starts != nullptr;
    const int len = rows_live(a, static_cast<int>(q.b));
    const int64_t nsaved = (static_cast<int64_t>(a.T) + kSaveRows - 1) / kSaveRows;
    const char *fp = q.at(a.f), *vp = q.at(a.v), *rp = q.at(a.r);
    char* yp = q.at(a.y);

    const int steps = (a.T + ROWS - 1) / ROWS;
    const int iters = (steps + a.S - 1) / a.S;
    using In = Inputs<C, 3>;
    const uint32_t ring = (ptx::smem_u32(smem) + 127u) & ~127u;
    [[maybe_unused]] const char* lane_at = smem + (ring - ptx::smem_u32(smem)) + (q.w * C::WROWS + q.seg * RPT) * In::ROW_BYTES + q.c * 8;
    auto step_of = [&](int it) { return static_cast<int64_t>(it) * a.S + q.rank; };
    auto has_rows = [&](int it) { return it < iters && step_of(it) * ROWS < len; };   // live rows to copy
    auto copy = [&](int it) {
        if (has_rows(it))
            copy_step<C, 3>(a.maps, ring + it % C::STAGES * (3 * In::TILE_BYTES), ptx::smem_u32(&full[it % C::STAGES]),
                            q.d0 - q.ch, step_of(it), static_cast<int>(q.b));
    };
    if constexpr (C::X::WIDE) {
        if (threadIdx.x == 0)
            for (int i = 0; i < C::STAGES; ++i) copy(i);
        __syncthreads();   // the barriers are set up before anyone waits
    }
    F2 lb[NP], carry[NP];
    load_f32(a.f_bias == nullptr ? nullptr : a.f_bias + q.d, q.nch, lb, 0.0f);
    load_f32(a.h_in == nullptr ? nullptr : a.h_in + q.b * a.D + q.d, q.nch, carry, 0.0f);
#pragma unroll
    for (int j = 0; j < NP; ++j) lb[j] = mul2(lb[j], both(-kLog2e));
    [[maybe_unused]] bool ok = true;
    for (int it = 0; it < iters; ++it) {
        const int p = it & 1;
        // not at entry: blocks of the next kernel that wait in the free slots meanwhile would be its
        // share of some SMs and not of others
        if (!CL && it + 1 == iters) ptx::pdl_trigger();
        const int64_t first = step_of(it) * ROWS + q.w * C::WROWS + q.seg * RPT;
        const int row0 = first < a.T ? static_cast<int>(first) : a.T;
        const int nl = min(max(len - row0, 0), RPT);   // live rows of this segment
        if constexpr (CL) {
            if (threadIdx.x == 0)
                ptx::mbar_arrive_expect_tx(ptx::smem_u32(&ex.bar[p]), static_cast<uint32_t>(a.S * C::CH * 2 * sizeof(float)));
        }
        const bool all_live = __all_sync(0xffffffffu, nl == RPT);
        In in;
        if constexpr (C::X::WIDE) {
            in.at = lane_at + it % C::STAGES * (3 * In::TILE_BYTES);
            if (has_rows(it)) ok = ok && wait_phase(&full[it % C::STAGES], (it / C::STAGES) & 1);
        }
        in.load(0, a.f, fp + row0 * a.f.st, nl, q.nch, all_live);
        in.load(1, a.v, vp + row0 * a.v.st, nl, q.nch, all_live);
        in.load(2, a.r, rp + row0 * a.r.st, nl, q.nch, all_live);
        const uint32_t cut = start_bits<C>(a, q.b, static_cast<int>(min(first - q.seg * RPT, static_cast<int64_t>(a.T))), len, q.seg, q.lane);
        const bool plain = all_live && (!docs || __all_sync(0xffffffffu, cut == 0));
        // (A, H) of this lane's rows
        F2 ga[RPT][NP], gb[RPT][NP], A[NP], H[NP];
        if (plain) fwd_rows<C, true>(in, lb, nl, cut, ga, gb, A, H);
        else fwd_rows<C, false>(in, lb, nl, cut, ga, gb, A, H);
        F2 PA[NP], PH[NP];
        warp_prefix<C, false>(A, H, H, PA, PH, PA, PH, q.seg, q.lane, !plain);
        if (q.seg == C::SEGS - 1) {
            put_s(&aggA[p][q.w][q.ch], A);
            put_s(&aggH[p][q.w][q.ch], H);
        }
        const bool cuts_here = sync_cuts(docs, cut);
        if constexpr (C::X::WIDE) {   // everyone has left the step before: its stage takes the step STAGES later
            if (threadIdx.x == 0 && it > 0) copy(it - 1 + C::STAGES);
        }
        // the state before this block's rows
        F2 h[NP];
        if constexpr (CL) {
            if (it == 0) cluster_wait();   // every peer has set up its barriers
            if (q.w == LEAD) {   // the block's total, to every block: a segment's lanes each serve S / SEGS of them
#pragma unroll
                for (int j = 0; j < NP; ++j) A[j] = both(1.0f), H[j] = both(0.0f);
                fold_map(&aggA[p][0][q.ch], &aggH[p][0][q.ch], C::CH, 0, WARPS, 1, A, H, cuts_here);
                for (int k = q.seg; k < a.S; k += C::SEGS) {
                    push_pairs(&ex.A[p][q.rank][q.ch], A, &ex.bar[p], k);
                    push_pairs(&ex.H[p][q.rank][q.ch], H, &ex.bar[p], k);
                }
                ok = ok && wait_phase(&ex.bar[p], (it >> 1) & 1);
                fold(&ex.A[p][0][q.ch], &ex.H[p][0][q.ch], C::CH, 0, q.rank, 1, carry, docs);
                if (q.seg == 0) put_s(&carry_s[p][q.ch], carry);
            }
            __syncthreads();
            if (q.w == LEAD) fold(&ex.A[p][0][q.ch], &ex.H[p][0][q.ch], C::CH, q.rank, a.S, 1, carry, docs);
            get_s(&carry_s[p][q.ch], h);
        } else {
#pragma unroll
            for (int j = 0; j < NP; ++j) h[j] = carry[j];
            if (it > 0) get_s(&carry_s[p ^ 1][q.ch], h);
        }
        fold(&aggA[p][0][q.ch], &aggH[p][0][q.ch], C::CH, 0, q.w, 1, h, cuts_here);
#pragma unroll
        for (int j = 0; j < NP; ++j) h[j] = apply(PA[j], PH[j], h[j], !plain);
        if (a.saved != nullptr && q.on && row0 < a.T && row0 % kSaveRows == 0)
            store_f32(a.saved + (q.b * nsaved + row0 / kSaveRows) * a.D + q.d, q.nch, h);
        // the rows again, from the state before them
        if (plain) fwd_again<C, true>(ga, gb, h);
        else fwd_again<C, false>(ga, gb, h);
        if constexpr (!CL) {
            if (q.w == WARPS - 1 && q.seg == C::SEGS - 1) put_s(&carry_s[p][q.ch], h);
        }
        const int nr = q.on ? min(a.T - row0, RPT) : 0;   // rows to write
        if (plain) fwd_store<C, true>(in, gb, yp + row0 * a.y.st, a.y.st, nl, nr, q.nch);
        else fwd_store<C, false>(in, gb, yp + row0 * a.y.st, a.y.st, nl, nr, q.nch);
    }
    if constexpr (!CL) {
        __syncthreads();
        if (iters > 0) get_s(&carry_s[(iters - 1) & 1][q.ch], carry);
    }
    if (a.h_out != nullptr && q.on && q.rank == 0 && q.w == (CL ? LEAD : 0) && q.seg == 0)
        store_f32(a.h_out + q.b * a.D + q.d, q.nch, carry);
    if (!ok) leave_late<CL>();
}

// ------------------------------------------------------------------------------ backward
template <class C, bool CL>
__global__ void __launch_bounds__(C::WARPS * 32, C::MINB) tern_scan_bwd_kernel(const __grid_constant__ GradArgs g) {
    using X = typename C::X;
    constexpr int NP = C::NP, RPT = C::RPT, WARPS = C::WARPS, ROWS = C::ROWS;
    constexpr int GROUP = kSaveRows / C::WROWS;   // warps from one saved state to the next
    constexpr int LEAD = 0;   // the warp that exchanges totals with the cluster's other blocks
    static_assert(ROWS % kSaveRows == 0 && kSaveRows % C::WROWS == 0, "steps start from saved states");
    const ScanArgs& a = g.s;
    extern __shared__ __align__(128) char smem[];
    __shared__ uint64_t full[C::STAGES];
    __shared__ alignas(16) float aggA[2][WARPS][C::CH], aggH[2][WARPS][C::CH], aggG[2][WARPS][C::CH];
    __shared__ alignas(16) float carry_s[2][C::CH];
    __shared__ typename std::conditional<CL, Exchange<C>, int>::type ex;
    const Place<C> q(a);
    if constexpr (C::X::WIDE) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < C::STAGES; ++i) ptx::mbar_init(ptx::smem_u32(&full[i]), 1);
            ptx::fence_mbar_init();
        }
    }
    if constexpr (CL) open_exchange(ex);
    ptx::pdl_wait();
    const bool docs = a.starts != nullptr;
    const int len = rows_live(a, static_cast<int>(q.b));
    const int64_t nsaved = (static_cast<int64_t>(a.T) + kSaveRows - 1) / kSaveRows;
    const int steps = (a.T + ROWS - 1) / ROWS;
    const int iters = (steps + a.S - 1) / a.S;
    const char *fp = q.at(a.f), *vp = q.at(a.v), *rp = q.at(a.r), *yp = q.at(a.y);
    char *dfp = q.at(g.df), *dvp = q.at(g.dv), *drp = q.at(g.dr);

    using In = Inputs<C, 4>;
    const uint32_t ring = (ptx::smem_u32(smem) + 127u) & ~127u;
    [[maybe_unused]] const char* lane_at = smem + (ring - ptx::smem_u32(smem)) + (q.w * C::WROWS + q.seg * RPT) * In::ROW_BYTES + q.c * 8;
    auto step_of = [&](int it) { return static_cast<int64_t>(steps - 1) - (static_cast<int64_t>(it) * a.S + q.rank); };
    auto has_rows = [&](int it) { return it < iters && step_of(it) >= 0 && step_of(it) * ROWS < len; };
    // the first step with live rows: the stages' phases count from there
    [[maybe_unused]] const int it0 = (max(steps - 1 - q.rank - max(len - 1, 0) / ROWS, 0) + a.S - 1) / a.S;
    auto copy = [&](int it) {
        if (has_rows(it))
            copy_step<C, 4>(a.maps, ring + it % C::STAGES * (4 * In::TILE_BYTES), ptx::smem_u32(&full[it % C::STAGES]),
                            q.d0 - q.ch, step_of(it), static_cast<int>(q.b));
    };
    if constexpr (C::X::WIDE) {
        if (threadIdx.x == 0)
            for (int i = 0; i < C::STAGES; ++i) copy(i);
        __syncthreads();   // the barriers are set up before anyone waits
    }
    [[maybe_unused]] bool ok = true;
    F2 lb[NP], carry[NP], dbias[NP];
    load_f32(a.f_bias == nullptr ? nullptr : a.f_bias + q.d, q.nch, lb, 0.0f);
    load_f32(a.h_in == nullptr ? nullptr : a.h_in + q.b * a.D + q.d, q.nch, carry, 0.0f);
#pragma unroll
    for (int j = 0; j < NP; ++j) lb[j] = mul2(lb[j], both(-kLog2e)), dbias[j] = both(0.0f);
    for (int it = 0; it < iters; ++it) {
        const int p = it & 1;
        if (!CL && it + 1 == iters) ptx::pdl_trigger();
        const int64_t step = step_of(it);   // below 0: nothing left for this block
        const int64_t first = step * ROWS + q.w * C::WROWS + q.seg * RPT;
        const int row0 = step >= 0 && first < a.T ? static_cast<int>(first) : a.T;
        const int nl = min(max(len - row0, 0), RPT);
        if constexpr (CL) {
            if (threadIdx.x == 0)
                ptx::mbar_arrive_expect_tx(ptx::smem_u32(&ex.bar[p]), static_cast<uint32_t>(a.S * C::CH * 2 * sizeof(float)));
        }
        const bool all_live = __all_sync(0xffffffffu, nl == RPT);
        In in;
        if constexpr (C::X::WIDE) in.at = lane_at + it % C::STAGES * (4 * In::TILE_BYTES);
        in.load(0, a.f, fp + row0 * a.f.st, nl, q.nch, all_live);
        in.load(1, a.v, vp + row0 * a.v.st, nl, q.nch, all_live);
        in.load(2, a.r, rp + row0 * a.r.st, nl, q.nch, all_live);
        in.load(3, a.y, yp + row0 * a.y.st, nl, q.nch, all_live);
        const uint32_t cut = start_bits<C>(a, q.b, step >= 0 ? static_cast<int>(min(first - q.seg * RPT, static_cast<int64_t>(a.T))) : a.T,
                                           len, q.seg, q.lane);
        const bool plain = all_live && (!docs || __all_sync(0xffffffffu, cut == 0));
        F2 h[NP];
        load_f32(row0 < a.T ? a.saved + (q.b * nsaved + row0 / kSaveRows) * a.D + q.d : nullptr, q.nch, h, 0.0f);
        if constexpr (C::X::WIDE) {
            if (has_rows(it)) ok = ok && wait_phase(&full[it % C::STAGES], ((it - it0) / C::STAGES) & 1);
        }
        F2 s[RPT][NP], n[RPT][NP], o[RPT][NP], x[RPT][NP], A[NP], H[NP], G[NP];
        if (plain) bwd_rows<C, true>(in, lb, nl, cut, s, n, o, x, A, H, G);
        else bwd_rows<C, false>(in, lb, nl, cut, s, n, o, x, A, H, G);
        F2 PA[NP], PH[NP], QA[NP], QG[NP];
        warp_prefix<C, true>(A, H, G, PA, PH, QA, QG, q.seg, q.lane, !plain);
        if (q.seg == 0) {
            put_s(&aggA[p][q.w][q.ch], A);
            put_s(&aggH[p][q.w][q.ch], H);
            put_s(&aggG[p][q.w][q.ch], G);
        }
        const bool cuts_here = sync_cuts(docs, cut);
        if constexpr (C::X::WIDE) {   // everyone has left the step before: its stage takes the step STAGES later
            if (threadIdx.x == (WARPS - 1) * 32 && it > 0) copy(it - 1 + C::STAGES);   // warp 0 has the totals to send
        }
        F2 e[NP];   // e after this segment's rows
        if constexpr (CL) {
            if (it == 0) cluster_wait();   // every peer has set up its barriers
            if (q.w == LEAD) {
#pragma unroll
                for (int j = 0; j < NP; ++j) A[j] = both(1.0f), G[j] = both(0.0f);
                fold_map(&aggA[p][0][q.ch], &aggG[p][0][q.ch], C::CH, WARPS - 1, -1, -1, A, G, cuts_here);
                for (int k = q.seg; k < a.S; k += C::SEGS) {
                    push_pairs(&ex.A[p][q.rank][q.ch], A, &ex.bar[p], k);
                    push_pairs(&ex.H[p][q.rank][q.ch], G, &ex.bar[p], k);
                }
                ok = ok && wait_phase(&ex.bar[p], (it >> 1) & 1);
                fold(&ex.A[p][0][q.ch], &ex.H[p][0][q.ch], C::CH, 0, q.rank, 1, carry, docs);
                if (q.seg == 0) put_s(&carry_s[p][q.ch], carry);
            }
            __syncthreads();
            if (q.w == LEAD) fold(&ex.A[p][0][q.ch], &ex.H[p][0][q.ch], C::CH, q.rank, a.S, 1, carry, docs);
            get_s(&carry_s[p][q.ch], e);
        } else {
#pragma unroll
            for (int j = 0; j < NP; ++j) e[j] = carry[j];
            if (it > 0) get_s(&carry_s[p ^ 1][q.ch], e);
        }
        fold(&aggA[p][0][q.ch], &aggG[p][0][q.ch], C::CH, WARPS - 1, q.w, -1, e, cuts_here);
        fold(&aggA[p][0][q.ch], &aggH[p][0][q.ch], C::CH, q.w / GROUP * GROUP, q.w, 1, h, cuts_here);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            e[j] = apply(QA[j], QG[j], e[j], !plain);
            h[j] = apply(PA[j], PH[j], h[j], !plain);
        }
        const int nr = q.on ? min(a.T - row0, RPT) : 0;   // rows to write
        char *dfr = dfp + row0 * g.df.st, *dvr = dvp + row0 * g.dv.st, *drr = drp + row0 * g.dr.st;
        if (plain) bwd_store<C, true>(in, s, n, o, x, nl, cut, nr, q.nch, h, e, dbias, dfr, g.df.st, dvr, g.dv.st, drr, g.dr.st);
        else bwd_store<C, false>(in, s, n, o, x, nl, cut, nr, q.nch, h, e, dbias, dfr, g.df.st, dvr, g.dv.st, drr, g.dr.st);
        if constexpr (!CL) {
            if (q.w == 0 && q.seg == 0) put_s(&carry_s[p][q.ch], e);
        }
    }
    __syncthreads();
    if constexpr (!CL) {
        if (iters > 0) get_s(&carry_s[(iters - 1) & 1][q.ch], carry);
    }
    if (a.h_out != nullptr && q.on && q.rank == 0 && q.w == 0 && q.seg == 0)
        store_f32(a.h_out + q.b * a.D + q.d, q.nch, carry);
    if (g.partial != nullptr) {   // this block's sum of df: a warp's segments, then the warps, in order
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int k = 1; k < C::SEGS; ++k) {
                const F2 other = shfl2(dbias[j], (k * C::LPR + q.c) & 31);
                if (q.seg == 0) dbias[j] = add2(dbias[j], other);
            }
        if (q.seg == 0) put_s(&aggH[0][q.w][q.ch], dbias);
        __syncthreads();
        if (q.w == 0 && q.seg == 0 && q.on) {
            F2 sum[NP];
            get_s(&aggH[0][0][q.ch], sum);
            for (int k = 1; k < WARPS; ++k) {
                F2 part[NP];
                get_s(&aggH[0][k][q.ch], part);
#pragma unroll
                for (int j = 0; j < NP; ++j) sum[j] = add2(sum[j], part[j]);
            }
            store_f32(g.partial + (q.b * a.S + q.rank) * a.D + q.d, q.nch, sum);
        }
    }
    if (!ok) leave_late<CL>();
}

// dbias[d] = sum of the blocks' partial sums: 8 warps take every eighth partial, then in order.
__global__ void __launch_bounds__(256) tern_scan_dbias_kernel(const float* __restrict__ partial, int64_t parts, int D,
                                                              float* __restrict__ dbias) {
    __shared__ float red[8][32];
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
    const char *f, *v, *r;
    char* y;
    const float* f_bias;
    const float* h_in;
    float* h_out;
    int64_t rows, f_sb, v_sb, r_sb, y_sb;   // strides in bytes
    int D;
};

template <class T, int W>
__global__ void __launch_bounds__(128) tern_scan_step_kernel(const __grid_constant__ StepArgs a) {
    using X = Io<T, W>;
    constexpr int NP = X::NP;
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int per_row = (a.D + 2 * NP - 1) / (2 * NP);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    const int64_t b = i / per_row;
    if (b >= a.rows) return;
    const int d = static_cast<int>(i - b * per_row) * 2 * NP, nch = min(a.D - d, 2 * NP);
    const int64_t at = static_cast<int64_t>(d) * static_cast<int64_t>(sizeof(T)), hd = b * a.D + d;
    F2 f[NP], v[NP], r[NP], h[NP], lb[NP], y[NP];
    X::get(X::load(a.f + b * a.f_sb + at, nch), f);
    X::get(X::load(a.v + b * a.v_sb + at, nch), v);
    X::get(X::load(a.r + b * a.r_sb + at, nch), r);
    load_f32(a.h_in + hd, nch, h, 0.0f);
    load_f32(a.f_bias == nullptr ? nullptr : a.f_bias + d, nch, lb, 0.0f);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        F2 s, n;
        decay(f[j], mul2(lb[j], both(-kLog2e)), s, n);
        h[j] = fma2(s, h[j], mul2(n, v[j]));
        y[j] = mul2(gate(r[j]), h[j]);
    }
    store_f32(a.h_out + hd, nch, h);
    X::store(a.y + b * a.y_sb + at, y, nch);
}

// ------------------------------------------------------------------------------ host side
namespace {

size_t elem(int dtype) { return dtype == TERN_F32 ? 4 : 2; }

// TERN_OK when x can be read or written as rows of elements, else the error; `align` becomes the
// largest of 16, 4 and an element's bytes that its rows' addresses allow as well (16 for TMA copies).
int check_act(const tern_act& x, const tern_scan* s, int& align) {
    const int64_t es = static_cast<int64_t>(elem(s->dtype));
    if (x.p == nullptr || x.stride_b < 0 || x.stride_t < 0) return TERN_ERR_ARG;
    if (x.stride_b > INT64_MAX / 4 / es || x.stride_t > INT64_MAX / 4 / es) return TERN_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(x.p) % es != 0) return TERN_ERR_ALIGN;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x.p) | static_cast<uintptr_t>(x.stride_b * es) | static_cast<uintptr_t>(x.stride_t * es);
    if (bits % 16 != 0) align = std::min(align, 4);
    if (bits % 4 != 0) align = 2;
    if ((s->T > 1 && x.stride_t < s->D) || (s->B > 1 && x.stride_b == 0)) align = std::min(align, 4);   // overlapping rows
    return TERN_OK;
}
// Whether two rows of x share an element: blocks would write them in any order.
bool rows_overlap(const tern_act& x, const tern_scan* s) {
    int64_t n0 = s->B, s0 = x.stride_b, n1 = s->T, s1 = x.stride_t;
    if (n0 == 1) n0 = n1, s0 = s1, n1 = 1;   // the stride of a size of one is not used
    if (n1 > 1 && s0 > s1) std::swap(n0, n1), std::swap(s0, s1);
    if (n0 > 1 && s0 < s->D) return true;
    if (n0 <= 1 || n1 <= 1) return false;
    const __int128 d = s->D, inner = static_cast<__int128>(n0 - 1) * s0;
    if (s1 >= inner + d) return false;       // one sequence (or row of all sequences) after the other
    // interleaved: some j s1 within a row of some i s0
    for (int64_t j = 1; j < n1 && static_cast<__int128>(j) * s1 < inner + d; ++j) {
        const __int128 at = static_cast<__int128>(j) * s1, i = at / s0;
        if ((i < n0 && at - i * s0 < d) || (i + 1 < n0 && (i + 1) * s0 - at < d)) return true;
    }
    return false;
}
Strided strided(const tern_act& x, const tern_scan* s) {
    const int64_t es = static_cast<int64_t>(elem(s->dtype)), sb = x.stride_b * es, st = x.stride_t * es;
    char* p = static_cast<char*>(x.p);
    return Strided{p, sb, st, p + (s->B - 1) * sb + (s->T - 1) * st + s->D * es};
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_scan(const tern_scan* s, int& align) {
    if (s == nullptr || (s->dtype != TERN_BF16 && s->dtype != TERN_F32)) return TERN_ERR_ARG;
    if (s->B < 0 || s->T < 0 || s->D < 0 || s->T > INT32_MAX - 256 || s->D > INT32_MAX - 256 || s->B > INT32_MAX - 256) return TERN_ERR_ARG;
    const int64_t row = s->D * static_cast<int64_t>(elem(s->dtype));
    align = row % 16 == 0 ? 16 : row % 4 == 0 ? 4 : 2;
    if (s->B == 0 || s->D == 0) return TERN_OK;
    if (s->T > 0) {
        for (const tern_act* x : {&s->f, &s->v, &s->r})
            if (int st = check_act(*x, s, align)) return st;
    }
    if (!aligned4(s->f_bias) || !aligned4(s->lengths)) return TERN_ERR_ALIGN;
    return TERN_OK;
}

// Clusters of 16 that are resident at once: a part of the GPU with an odd block over holds none more.
template <class C>
constexpr int fit16() { return C::WARPS == 8 ? 14 : 33; }

// Blocks per cluster: the largest power of two, at most kMaxCluster and less than twice the steps,
// with which the blocks are all resident at once.
template <class C>
int cluster_size(int64_t blocks, int64_t steps, int num_sms) {
    int S = 1;
    while (S < kMaxCluster && S < steps && 2 * S * blocks <= static_cast<int64_t>(C::MINB) * num_sms &&
           (2 * S < kMaxCluster || blocks <= fit16<C>()))
        S *= 2;
    return S;
}

int64_t steps_of(int64_t T, int64_t rows) { return (T + rows - 1) / rows; }

// The tensor map of an input: [B][T][D] in boxes of ROWS rows by CH channels.
template <class C>
int input_map(CUtensorMap* m, const Strided& x, int64_t B, int64_t T, int64_t D) {
    const CUtensorMapDataType type = sizeof(typename C::T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    // a stride that no second row or sequence uses may be anything that the encoding takes
    const int64_t least = D * static_cast<int64_t>(sizeof(typename C::T));
    return tensor_map_3d(m, x.p, type, D, T, B, T > 1 ? x.st : least, B > 1 ? x.sb : least, C::CH, C::ROWS);
}

// Clusters of more than two steps each are launched once the kernels before them have ended, and none let
// the next kernel in before their own end: clusters that take the slots which happen to be free until then
// leave the others an uneven share of the SMs for all of their run (the gradient of 1 x 65536 x 512 306 us
// behind a small kernel that let it in early, 205 us so).  A short run would lose more by the later launch
// (the gradient of 1 x 512 x 512: 8.0 us, 10.7 us).
bool short_run(int64_t steps, int S) { return steps <= 2 * S; }

template <class C, bool CL>
int launch_fwd(const ScanArgs& a0, int64_t B, int num_sms, cudaStream_t s) {
    ScanArgs a = a0;
    a.tiles = (a.D + C::CH - 1) / C::CH;
    const int64_t blocks = B * a.tiles;
    a.S = CL ? cluster_size<C>(blocks, steps_of(a.T, C::ROWS), num_sms) : 1;
    if (blocks * a.S > INT32_MAX) return TERN_ERR_ARG;
    const unsigned grid = static_cast<unsigned>(blocks * a.S);
    if (C::X::WIDE && a.T > 0) {
        const Strided* in[3] = {&a.f, &a.v, &a.r};
        for (int i = 0; i < 3; ++i)
            if (int st = input_map<C>(&a.maps[i], *in[i], B, a.T, a.D)) return st;
    }
    constexpr size_t smem = Inputs<C, 3>::SMEM;
    if constexpr (CL) {
        if (a.S > 1) return launch_cluster(tern_scan_fwd_kernel<C, true>, grid, C::WARPS * 32, smem, a.S, short_run(steps_of(a.T, C::ROWS), a.S), s, a);
    }
    return launch_cluster(tern_scan_fwd_kernel<C, false>, grid, C::WARPS * 32, smem, 1, true, s, a);
}

template <class C, bool CL>
int launch_bwd(const GradArgs& g0, int64_t B, int num_sms, float* dbias, cudaStream_t s) {
    GradArgs g = g0;
    g.s.tiles = (g.s.D + C::CH - 1) / C::CH;
    const int64_t blocks = B * g.s.tiles;
    g.s.S = CL ? cluster_size<C>(blocks, steps_of(g.s.T, C::ROWS), num_sms) : 1;
    if (blocks * g.s.S > INT32_MAX) return TERN_ERR_ARG;
    const unsigned grid = static_cast<unsigned>(blocks * g.s.S);
    if (C::X::WIDE && g.s.T > 0) {
        const Strided* in[4] = {&g.s.f, &g.s.v, &g.s.r, &g.s.y};
        for (int i = 0; i < 4; ++i)
            if (int st = input_map<C>(&g.s.maps[i], *in[i], B, g.s.T, g.s.D)) return st;
    }
    constexpr size_t smem = Inputs<C, 4>::SMEM;
    int st = TERN_OK;
    if constexpr (CL) {
        st = g.s.S > 1 ? launch_cluster(tern_scan_bwd_kernel<C, true>, grid, C::WARPS * 32, smem, g.s.S,
                                        short_run(steps_of(g.s.T, C::ROWS), g.s.S), s, g)
                       : launch_cluster(tern_scan_bwd_kernel<C, false>, grid, C::WARPS * 32, smem, 1, true, s, g);
    } else {
        st = launch_cluster(tern_scan_bwd_kernel<C, false>, grid, C::WARPS * 32, smem, 1, true, s, g);
    }
    if (st != TERN_OK) return st;
    if (dbias == nullptr) return TERN_OK;
    return launch_pdl(tern_scan_dbias_kernel, dim3(static_cast<unsigned>((g.s.D + 31) / 32)), dim3(256), 0, s,
                      static_cast<const float*>(g.partial), B * g.s.S, g.s.D, dbias);
}

// The shape of the blocks, by how many there are of 64 bytes of channels by a whole sequence: enough
// for more than two of four warps on each SM; else blocks of eight warps, in clusters where even
// those leave SMs free; and tiles of half the channels where clusters of 16 such blocks are enough.
// (Forward and gradient of 16 x 512 x 512: 15.5 + 24.8 us as clusters of four-warp blocks, 8.8 + 18.1 us
// as eight-warp blocks; of 8 x 2048 x 2048: 53 + 118 us with four warps, 58 + 124 us with eight; of 1 x
// 65536 x 512: 82 + 186 us in the narrow tiles, 134 + 295 us in wide ones.)
template <class T, int W, int RPT, class F>
int with_shape(int64_t B, int64_t D, int64_t T_, int num_sms, F run) {
    using Four = Shape<T, W, 8, RPT, 4, 4, 2>;
    using Eight = Shape<T, W, 8, RPT, 8, 2, 2>;
    using Narrow = Shape<T, W, 4, RPT, 4, 4, 2>;
    const int64_t blocks = B * ((D + Four::CH - 1) / Four::CH);
    if (blocks > 2 * num_sms) return run(Four{}, std::false_type{});
    if (2 * blocks <= fit16<Narrow>() && steps_of(T_, Eight::ROWS) > kMaxCluster / 2) return run(Narrow{}, std::true_type{});
    return run(Eight{}, std::true_type{});
}

ScanArgs scan_args(const tern_scan* s) {
    ScanArgs a{};
    a.f = strided(s->f, s), a.v = strided(s->v, s), a.r = strided(s->r, s);
    a.f_bias = s->f_bias, a.lengths = s->lengths, a.starts = s->starts;
    a.T = static_cast<int>(s->T), a.D = static_cast<int>(s->D);
    return a;
}

}  // namespace

int scan_status_read(int clear) {
    int v = 0;
    TERN_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_scan_status, sizeof(v)));
    const int zero = 0;
    if (v != 0 && clear) TERN_CUDA_TRY(cudaMemcpyToSymbol(g_scan_status, &zero, sizeof(zero)));
    return v != 0 ? TERN_ERR_TIMEOUT : TERN_OK;
}

}  // namespace tern

using namespace tern;

extern "C" size_t tern_scan_saved(int64_t B, int64_t T, int64_t D) {
    if (B < 0 || T < 0 || D < 0) return 0;
    return static_cast<size_t>(B * steps_of(T, kSaveRows) * D) * sizeof(float);
}

extern "C" int tern_scan_fwd(const tern_scan* s, const float* h0, const tern_act* y, float* hT, float* saved,
                             size_t saved_bytes, void* stream) {
    int align;
    if (int st = check_scan(s, align)) return st;
    if (s->B == 0 || s->D == 0) return TERN_OK;
    if (s->T > 0) {
        if (y == nullptr) return TERN_ERR_ARG;
        if (int st = check_act(*y, s, align)) return st;
        if (rows_overlap(*y, s)) return TERN_ERR_ARG;
    }
    if (!aligned4(h0) || !aligned4(hT) || !aligned4(saved)) return TERN_ERR_ALIGN;
    if (saved != nullptr && saved_bytes < tern_scan_saved(s->B, s->T, s->D)) return TERN_ERR_WORKSPACE;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    ScanArgs a = scan_args(s);
    if (s->T > 0) a.y = strided(*y, s);
    a.saved = saved, a.h_in = h0, a.h_out = hT;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    auto run = [&](auto shape, auto cl) { return launch_fwd<decltype(shape), decltype(cl)::value>(a, s->B, num_sms, cs); };
    if (s->dtype == TERN_BF16)
        return align == 16  ? with_shape<__nv_bfloat16, 16, 8>(s->B, s->D, s->T, num_sms, run)
               : align == 4 ? with_shape<__nv_bfloat16, 4, 8>(s->B, s->D, s->T, num_sms, run)
                            : with_shape<__nv_bfloat16, 2, 8>(s->B, s->D, s->T, num_sms, run);
    return align == 16 ? with_shape<float, 16, 8>(s->B, s->D, s->T, num_sms, run) : with_shape<float, 4, 8>(s->B, s->D, s->T, num_sms, run);
}

extern "C" size_t tern_scan_bwd_workspace(int64_t B, int64_t T, int64_t D) {
    if (B < 0 || T < 0 || D < 0) return 0;
    return static_cast<size_t>(B * kMaxCluster * D) * sizeof(float);   // the blocks' sums of df
}

extern "C" int tern_scan_bwd(const tern_scan* s, const float* saved, const tern_act* dy, const float* dhT,
                             const tern_act* df, const tern_act* dv, const tern_act* dr, float* dbias, float* dh0,
                             void* workspace, size_t ws_bytes, void* stream) {
    int align;
    if (int st = check_scan(s, align)) return st;
    if (s->B == 0 || s->D == 0) return s->D == 0 || dbias == nullptr ? TERN_OK : TERN_ERR_ARG;
    if (s->T > 0) {
        if (saved == nullptr) return TERN_ERR_ARG;
        for (const tern_act* x : {dy, df, dv, dr}) {
            if (x == nullptr) return TERN_ERR_ARG;
            if (int st = check_act(*x, s, align)) return st;
            if (x != dy && rows_overlap(*x, s)) return TERN_ERR_ARG;
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
    if (s->T > 0) {
        g.s.y = strided(*dy, s);
        g.df = strided(*df, s), g.dv = strided(*dv, s), g.dr = strided(*dr, s);
    }
    g.partial = dbias != nullptr ? static_cast<float*>(workspace) : nullptr;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    auto run = [&](auto shape, auto cl) { return launch_bwd<decltype(shape), decltype(cl)::value>(g, s->B, num_sms, dbias, cs); };
    if (s->dtype == TERN_BF16)
        return align == 16  ? with_shape<__nv_bfloat16, 16, 4>(s->B, s->D, s->T, num_sms, run)
               : align == 4 ? with_shape<__nv_bfloat16, 4, 4>(s->B, s->D, s->T, num_sms, run)
                            : with_shape<__nv_bfloat16, 2, 4>(s->B, s->D, s->T, num_sms, run);
    return align == 16 ? with_shape<float, 16, 4>(s->B, s->D, s->T, num_sms, run) : with_shape<float, 4, 4>(s->B, s->D, s->T, num_sms, run);
}

namespace {
template <class T, int W>
int launch_step(const StepArgs& a, cudaStream_t s) {
    constexpr int VEC = 2 * Io<T, W>::NP;
    const int64_t blocks = (a.rows * ((a.D + VEC - 1) / VEC) + 127) / 128;
    if (blocks > INT32_MAX) return TERN_ERR_ARG;
    return launch_pdl(tern_scan_step_kernel<T, W>, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, s, a);
}
}  // namespace

extern "C" int tern_scan_step(const tern_scan* s, const float* h_in, float* h_out, const tern_act* y, void* stream) {
    int align;
    if (int st = check_scan(s, align)) return st;
    if (s->T != 1 || s->lengths != nullptr || s->starts != nullptr) return TERN_ERR_ARG;
    if (s->B == 0 || s->D == 0) return TERN_OK;
    if (h_in == nullptr || h_out == nullptr || y == nullptr) return TERN_ERR_ARG;
    if (int st = check_act(*y, s, align)) return st;
    if (rows_overlap(*y, s)) return TERN_ERR_ARG;
    if (!aligned4(h_in) || !aligned4(h_out)) return TERN_ERR_ALIGN;
    if (int st = check_device(nullptr)) return st;
    StepArgs a{};
    const int64_t es = static_cast<int64_t>(elem(s->dtype));
    a.f = static_cast<char*>(s->f.p), a.v = static_cast<char*>(s->v.p), a.r = static_cast<char*>(s->r.p);
    a.y = static_cast<char*>(y->p);
    a.f_sb = s->f.stride_b * es, a.v_sb = s->v.stride_b * es, a.r_sb = s->r.stride_b * es, a.y_sb = y->stride_b * es;
    a.f_bias = s->f_bias, a.h_in = h_in, a.h_out = h_out;
    a.rows = s->B, a.D = static_cast<int>(s->D);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (s->dtype == TERN_BF16) return align == 16 ? launch_step<__nv_bfloat16, 16>(a, cs) : launch_step<__nv_bfloat16, 2>(a, cs);
    return align == 16 ? launch_step<float, 16>(a, cs) : launch_step<float, 4>(a, cs);
}
