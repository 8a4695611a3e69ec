// What is computed from rows of logits: the log probability of a given token with the row's entropy and
// its most likely entries, and distillation from a teacher's top logits with its gradient.
//
//   m = max x, S = sum exp(x - m), lse = m + log S
//   logp = x[token] - lse,  entropy = log S - sum exp(x - m) (x - m) / S
//   loss = w T^2 sum p (log p - log q[id]),  dlogits = w T (q - p),   q = softmax(x / T)
//
// Memory bounds both: the score reads each logit once, the distillation reads it once and writes its
// gradient once.  One pass keeps a running maximum and sums relative to it; threads, blocks and the
// blocks of a cluster (which share a row where rows are few) are joined at the end.  Rows of up to
// 1024 entries belong to a warp each, which holds them in registers.
//
// Rows start at any element: whole 16-byte words of a row are its body, the few entries before and
// after them its head and tail.
#include <algorithm>
#include <cmath>

#include "rows.cuh"

namespace tern {
namespace {

constexpr int kWarpRow = 1024;    // widest row of a warp
constexpr int kMaxTop = TERN_SCORE_MAX_TOP;
constexpr int kMaxTeacher = TERN_DISTILL_MAX_TOP;
constexpr float kLog2e = 1.44269504f;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float pow2(float x) {   // 2^x to 2^-22 relative
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// A running softmax: maximum, sum of 2^(c (x - m)) and, for the entropy, the same with the factor (x - m).
// c = log2(e) / T.  The difference is taken first: it is exact near the maximum, where it counts.
template <bool ENT>
struct Stats {
    float m = kNegInf, s = 0.f, q = 0.f, c;
    __device__ __forceinline__ explicit Stats(float c_) : c(c_) {}

    // Moves to the maximum mn >= m (finite, or inf: then s becomes NaN as it should).
    __device__ __forceinline__ void rebase(float mn) {
        if (m != kNegInf) {   // of nothing but -inf s and q are 0, or s is NaN
            const float d = m - mn, f = pow2(d * c);
            if (ENT) q = (q + s * d) * f;
            s *= f;
        }
        m = mn;
    }

    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float top) {
        const float mn = fmaxf(m, top);   // drops NaN; the sums below bring it back
        if (mn == kNegInf) {              // nothing but -inf (and NaN) so far
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) t += x[i];
            if (t != t) s = t;
            return;
        }
        if (mn > m) rebase(mn);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // -inf (a masked entry) would give 0 times infinity
            const float z = ENT ? max_nan(x[i] - mn, -1e4f) : x[i] - mn;
            const float e = pow2(z * c);
            s += e;
            if (ENT) q = fmaf(e, z, q);
        }
    }

    __device__ __forceinline__ void join(float om, float os, float oq) {
        const float mn = fmaxf(m, om);
        if (mn == kNegInf) {
            s += os;
            return;
        }
        Stats o(c);
        o.m = om, o.s = os, o.q = oq;
        rebase(mn);
        o.rebase(mn);
        s += o.s;
        q += o.q;
    }

    __device__ __forceinline__ void join_warp() {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m, d), os = __shfl_xor_sync(0xffffffffu, s, d);
            const float oq = ENT ? __shfl_xor_sync(0xffffffffu, q, d) : 0.f;
            // the lower lane's first in both, so that all lanes hold the same bits
            if ((threadIdx.x & d) == 0) {
                join(om, os, oq);
            } else {
                Stats o(c);
                o.m = om, o.s = os, o.q = oq;
                o.join(m, s, q);
                *this = o;
            }
        }
    }
};

// A row's place: head entries, then nb words of VE, then tail entries.
template <class T>
struct Row {
    static constexpr int VE = 16 / kElem<T>;
    const T* p;
    int V, head, nb, tail0;   // tail0: first entry of the tail
    __device__ __forceinline__ Row(const void* base, int64_t row, int64_t ld, int V_) : p(static_cast<const T*>(base) + row * ld), V(V_) {
        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / kElem<T>;
        head = min(V, mis ? VE - mis : 0);
        nb = (V - head) / VE;
        tail0 = head + nb * VE;
    }
    __device__ __forceinline__ int edges() const { return head + V - tail0; }
    // entry of the e-th of the edges
    __device__ __forceinline__ int edge(int e) const { return e < head ? e : tail0 + e - head; }
    __device__ __forceinline__ const T* word(int i) const { return p + head + static_cast<int64_t>(i) * VE; }
    __device__ __forceinline__ float at(int e) const { return raw_at<T, 1>(load_raw<T, 1>(p + e), 0); }
};

template <class T, int V>
__device__ __forceinline__ float raw_max(const Raw<T, V>& r) {   // drops NaN
    float m = raw_at<T, V>(r, 0);
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, raw_at<T, V>(r, i));
    return m;
}

// The words that block `rank` of `size` takes of a row's body: [first, last).
__device__ __forceinline__ void slice(int nb, int rank, int size, int& first, int& last) {
    const int per = (nb + size - 1) / size;
    first = min(nb, rank * per);
    last = min(nb, first + per);
}

// One pass of a block of T threads over its words of a row (and, in block 0, the edges): thread t
// takes the words first + t, first + t + T, ...
template <class TX, int T, bool ENT>
__device__ __forceinline__ void read_row(const Row<TX>& r, int first, int last, bool edges, Stats<ENT>& st) {
    constexpr int VE = Row<TX>::VE, U = 4;
    int i = first + static_cast<int>(threadIdx.x);
    for (; i + (U - 1) * T < last; i += U * T) {
        Raw<TX, VE> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = load_raw<TX, VE>(r.word(i + u * T));
        float top = kNegInf;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, raw_max<TX, VE>(raw[u]));
        float x[U * VE];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < VE; ++e) x[u * VE + e] = raw_at<TX, VE>(raw[u], e);
        st.add(x, top);
    }
    for (; i < last; i += T) {
        const auto raw = load_raw<TX, VE>(r.word(i));
        float x[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = raw_at<TX, VE>(raw, e);
        st.add(x, raw_max<TX, VE>(raw));
    }
    if (edges && static_cast<int>(threadIdx.x) < r.edges()) {
        const float x[1] = {r.at(r.edge(threadIdx.x))};
        st.add(x, x[0]);
    }
}

// Joins the threads of a block (through s: 3 T / 32 floats), and the blocks of a cluster; every
// thread holds the result.  Uses barriers of both.
template <int T, bool ENT>
__device__ __forceinline__ void join_block(Stats<ENT>& st, float* s, uint32_t rank, uint32_t size) {
    constexpr int W = T / 32;
    st.join_warp();
    if ((threadIdx.x & 31) == 0) {
        float* at = s + 3 * (threadIdx.x >> 5);
        at[0] = st.m, at[1] = st.s, at[2] = st.q;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const bool in = lane < W;
        st.m = in ? s[3 * lane] : kNegInf, st.s = in ? s[3 * lane + 1] : 0.f, st.q = in ? s[3 * lane + 2] : 0.f;
        st.join_warp();
        __syncwarp();
        if (lane == 0) s[0] = st.m, s[1] = st.s, s[2] = st.q;
    }
    if (size > 1) ptx::cluster_sync(); else __syncthreads();
    if (size == 1) {
        st.m = s[0], st.s = s[1], st.q = s[2];
    } else {
        st = Stats<ENT>(st.c);
        for (uint32_t r = 0; r < size; ++r) {
            const uint32_t from = ptx::mapa_shared(ptx::smem_u32(s), r);
            float m, v, q;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(m) : "r"(from) : "memory");
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from + 4u) : "memory");
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q) : "r"(from + 8u) : "memory");
            st.join(m, v, q);
        }
    }
}

__device__ __forceinline__ void cluster_place(uint32_t& rank, uint32_t& size) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(size));
}

// ------------------------------------------------------------------------------ score
//
// The k largest entries, the lower index first where equal: a thread's running maximum is at hand after
// the pass, and the k-th largest of the threads' maxima is a bound that at least k entries reach.  Few
// others do (with T threads of E entries each about k + k^2 / 2T), so only the words of threads whose
// maximum reaches it are read again, from L2.  Entries are ordered by 64-bit keys, the value above
// the complement of the index, all different; each candidate's rank is the number of larger keys.
// Where more entries reach the bound than there is room for (masked rows, constant ones) the exact
// k-th value is found by bisection, and entries equal to it are taken in the order of the row.
constexpr int kCand = 1024;

__device__ __forceinline__ uint32_t order_key(float x) {   // larger for larger x; NaN above all, -0 as 0; never 0
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k == 0xFFFFFFFFu ? 0x7FFFFFFFu : k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ unsigned long long entry_key(uint32_t key, int index) {
    return (static_cast<unsigned long long>(key) << 32) | static_cast<uint32_t>(~index);
}

struct ScoreArgs {
    const void* logits;
    const void* tokens;
    float* logp;
    float* entropy;
    float* lse;
    int32_t* top_ids;
    float* top_logp;
    int64_t ld;
    int n, V, k, wide_ids;
};

template <int T>
struct TopSpace {
    unsigned long long cand[kCand];
    unsigned long long best[kMaxTop];
    uint16_t list[T];
    int rank[kMaxTop];
    int count, listed;
    int warps[T / 32];
};

// Every entry of the slice with a key of at least lo, as candidates; sp.count of them (kCand are kept).
template <class TX, int T>
__device__ __forceinline__ void collect(const Row<TX>& r, int first, int last, bool edges, uint32_t mine, uint32_t lo, TopSpace<T>& sp) {
    constexpr int VE = Row<TX>::VE;
    __syncthreads();
    if (threadIdx.x == 0) sp.count = sp.listed = 0;
    __syncthreads();
    if (mine >= lo) sp.list[atomicAdd(&sp.listed, 1)] = static_cast<uint16_t>(threadIdx.x);
    auto offer = [&](float x, int e) {
        const uint32_t key = order_key(x);
        if (key >= lo) {
            const int at = atomicAdd(&sp.count, 1);
            if (at < kCand) sp.cand[at] = entry_key(key, e);
        }
    };
    __syncthreads();
    const int listed = sp.listed, rounds = (last - first + T - 1) / T;
    for (int w = threadIdx.x; w < listed * rounds; w += T) {
        const int i = first + sp.list[w % listed] + (w / listed) * T;
        if (i < last) {
            const auto raw = load_raw<TX, VE>(r.word(i));
#pragma unroll
            for (int e = 0; e < VE; ++e) offer(raw_at<TX, VE>(raw, e), r.head + i * VE + e);
        }
    }
    if (edges && static_cast<int>(threadIdx.x) < r.edges()) {
        const int e = r.edge(threadIdx.x);
        offer(r.at(e), e);
    }
    __syncthreads();
}

// Entries of the slice with a key of at least lo, counted.
template <class TX, int T>
__device__ __forceinline__ int count_from(const Row<TX>& r, int first, int last, bool edges, uint32_t lo, TopSpace<T>& sp) {
    constexpr int VE = Row<TX>::VE;
    int c = 0;
    for (int i = first + static_cast<int>(threadIdx.x); i < last; i += T) {
        const auto raw = load_raw<TX, VE>(r.word(i));
#pragma unroll
        for (int e = 0; e < VE; ++e) c += order_key(raw_at<TX, VE>(raw, e)) >= lo;
    }
    if (edges && static_cast<int>(threadIdx.x) < r.edges()) c += order_key(r.at(r.edge(threadIdx.x))) >= lo;
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0) sp.warps[threadIdx.x >> 5] = c;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) all += sp.warps[w];
    __syncthreads();
    return all;
}

// The k largest entries of the slice into sp.best, largest first, zeros where there are fewer.
// `mine`: the largest key among the thread's entries, 0 without any.
template <class TX, int T>
__device__ __forceinline__ void block_top(const Row<TX>& r, int first, int last, bool edges, uint32_t mine, int k, TopSpace<T>& sp) {
    constexpr int VE = Row<TX>::VE;
    uint32_t lo = 0;   // the upper 16 bits of the bound: all that bf16 has
#pragma unroll 1
    for (int b = 31; b >= 16; --b)
        if (__syncthreads_count(mine >= (lo | (1u << b))) >= k) lo |= 1u << b;
    collect<TX, T>(r, first, last, edges, mine, lo, sp);
    int n = sp.count;
    if (n > kCand) {
        // the k-th largest value exactly.  A bf16's lower bits are known (ones where negative, and of
        // NaN), and nothing but -inf has its upper bits.
        if (kElem<TX> == 2 || lo == 0x007F0000u) {
            if (lo < 0x80000000u || lo == 0xFFFF0000u) lo |= 0xFFFFu;
        } else {
#pragma unroll 1
            for (int b = 15; b >= 0; --b)
                if (count_from<TX, T>(r, first, last, edges, lo | (1u << b), sp) >= k) lo |= 1u << b;
        }
        collect<TX, T>(r, first, last, edges, mine, lo + 1, sp);   // fewer than k; of NaN alone (no lo + 1) none below
        n = lo == 0xFFFFFFFFu ? 0 : sp.count;
        // the first of those equal to it: the head, the body in order, the tail
        int want = k - n, found = 0;
        auto place = [&](bool hit, int before, int e) {
            if (hit && before < want) sp.cand[n + before] = entry_key(lo, e);
        };
        if (edges)
            for (int e = 0; e < r.head; ++e) {
                const bool hit = order_key(r.at(e)) == lo;
                if (threadIdx.x == 0) place(hit, found, e);
                found += hit;
            }
        for (int i0 = first; i0 < last && found < want; i0 += T) {
            const int i = i0 + static_cast<int>(threadIdx.x);
            uint32_t hits = 0;
            if (i < last) {
                const auto raw = load_raw<TX, VE>(r.word(i));
#pragma unroll
                for (int e = 0; e < VE; ++e) hits |= static_cast<uint32_t>(order_key(raw_at<TX, VE>(raw, e)) == lo) << e;
            }
            const int lane = threadIdx.x & 31, mineN = __popc(hits);
            int incl = mineN;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
            }
            if (lane == 31) sp.warps[threadIdx.x >> 5] = incl;
            __syncthreads();
            int before = found + incl - mineN;
#pragma unroll
            for (int w = 0; w < T / 32; ++w) {
                if (w < static_cast<int>(threadIdx.x >> 5)) before += sp.warps[w];
                found += sp.warps[w];
            }
            for (int e = 0; hits; hits >>= 1, ++e)
                if (hits & 1) place(true, before++, r.head + i * VE + e);
            __syncthreads();
        }
        if (edges)
            for (int e = r.tail0; e < r.V && found < want; ++e) {
                const bool hit = order_key(r.at(e)) == lo;
                if (threadIdx.x == 0) place(hit, found, e);
                found += hit;
            }
        n += min(found, want);
        __syncthreads();
    }
    for (int c = threadIdx.x; c < k; c += T)
        if (c >= n) sp.best[c] = 0ull;
    for (int c = threadIdx.x; c < n; c += T) {
        const unsigned long long key = sp.cand[c];
        int rank = 0;
        for (int o = 0; o < n; ++o) rank += sp.cand[o] > key;
        if (rank < k) sp.best[rank] = key;
    }
    __syncthreads();
}

// What a row's statistics give: z(x) = log probability of an entry x.
struct RowLog {
    float m, log_s;
    bool dead;   // nothing but -inf
    template <bool ENT>
    __device__ __forceinline__ explicit RowLog(const Stats<ENT>& st) : m(st.m), log_s(logf(st.s)), dead(st.m == kNegInf && st.s == 0.f) {}
    __device__ __forceinline__ float logp(float x) const { return dead ? kNegInf : x - m - log_s; }
    __device__ __forceinline__ float lse() const { return dead ? kNegInf : m + log_s; }
};

__device__ __forceinline__ void write_top(const ScoreArgs& a, int64_t row, int c, unsigned long long key, const RowLog& l) {
    a.top_ids[row * a.k + c] = static_cast<int32_t>(~static_cast<uint32_t>(key));
    a.top_logp[row * a.k + c] = l.logp(key_value(static_cast<uint32_t>(key >> 32)));
}

template <class TX>
__device__ __forceinline__ void write_row(const ScoreArgs& a, int64_t row, const Row<TX>& r, const Stats<true>& st, const RowLog& l) {
    if (a.lse) a.lse[row] = l.lse();
    if (a.entropy) a.entropy[row] = l.dead ? 0.f : fmaxf(l.log_s - st.q / st.s, 0.f) + (st.s != st.s ? st.s : 0.f);
    if (a.logp) {
        const int64_t tok = a.wide_ids ? __ldg(static_cast<const long long*>(a.tokens) + row) : __ldg(static_cast<const int32_t*>(a.tokens) + row);
        a.logp[row] = tok >= 0 && tok < a.V ? l.logp(r.at(static_cast<int>(tok))) : 0.f;
    }
}

// A row a cluster (of one block, or of several where rows are few).
template <class TX, int T>
__global__ void __launch_bounds__(T) score_rows(const __grid_constant__ ScoreArgs a) {
    __shared__ float s[3 * (T / 32)];
    __shared__ TopSpace<T> sp;
    uint32_t rank, size;
    cluster_place(rank, size);
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int64_t row = blockIdx.x / size;
    const Row<TX> r(a.logits, row, a.ld, a.V);
    int first, last;
    slice(r.nb, rank, size, first, last);
    const bool edges = rank == 0;
    Stats<true> st(kLog2e);
    read_row<TX, T, true>(r, first, last, edges, st);
    uint32_t mine = 0;
    if (a.k) {
        const bool any = first + static_cast<int>(threadIdx.x) < last || (edges && static_cast<int>(threadIdx.x) < r.edges());
        mine = any ? order_key(st.m) : 0u;
        // infinities and NaN: the maximum that the sums are relative to may not be the largest entry's key
        if (__syncthreads_or(st.s != st.s)) {
            mine = 0;
            for (int i = first + static_cast<int>(threadIdx.x); i < last; i += T) {
                const auto raw = load_raw<TX, Row<TX>::VE>(r.word(i));
#pragma unroll
                for (int e = 0; e < Row<TX>::VE; ++e) mine = max(mine, order_key(raw_at<TX, Row<TX>::VE>(raw, e)));
            }
            if (edges && static_cast<int>(threadIdx.x) < r.edges()) mine = max(mine, order_key(r.at(r.edge(threadIdx.x))));
        }
    }
    join_block<T, true>(st, s, rank, size);
    const RowLog l(st);
    if (rank == 0 && threadIdx.x == 0) write_row(a, row, r, st, l);
    if (a.k == 0) {
        if (size > 1) ptx::cluster_sync();   // the peers have read this block's sums
        return;
    }
    block_top<TX, T>(r, first, last, edges, mine, a.k, sp);
    if (size == 1) {
        for (int c = threadIdx.x; c < a.k; c += T) write_top(a, row, c, sp.best[c], l);
        return;
    }
    // each block ranks its own entries among all blocks' sorted lists, copied here first
    ptx::cluster_sync();
    const int k = a.k, lists = static_cast<int>(size);
    for (int w = threadIdx.x; w < k * lists; w += T) {
        const uint32_t from = ptx::mapa_shared(ptx::smem_u32(&sp.best[w % k]), static_cast<uint32_t>(w / k));
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(sp.cand[w]) : "r"(from) : "memory");
    }
    for (int c = threadIdx.x; c < k; c += T) sp.rank[c] = 0;
    __syncthreads();
    for (int w = threadIdx.x; w < k * lists; w += T) {
        const int c = w % k, o = w / k;
        const unsigned long long key = sp.best[c];
        int lo = 0, hi = k;   // entries of list o above the key: a sorted list's first ones
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (sp.cand[o * k + mid] > key) lo = mid + 1;
            else hi = mid;
        }
        if (lo) atomicAdd(&sp.rank[c], lo);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < k; c += T)
        if (sp.best[c] && sp.rank[c] < k) write_top(a, row, sp.rank[c], sp.best[c], l);
    ptx::cluster_sync();   // the peers have read this block's list
}

// A row of up to 32 EPL entries in a warp's registers: lane l holds entries j 32 + l.
template <class TX, int EPL>
__global__ void __launch_bounds__(128) score_warps(const __grid_constant__ ScoreArgs a) {
    ptx::pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    ptx::pdl_wait();
    if (row >= a.n) return;
    const Row<TX> r(a.logits, row, a.ld, a.V);
    float x[EPL];
    float top = kNegInf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        x[j] = j * 32 + lane < a.V ? r.at(j * 32 + lane) : kNegInf;
        top = fmaxf(top, x[j]);
    }
    Stats<true> st(kLog2e);
    st.add(x, top);
    st.join_warp();
    const RowLog l(st);
    if (lane == 0) write_row(a, row, r, st, l);
    if (a.k == 0) return;
    // the largest k times, the lowest index first: each lane's best entry below the last one taken
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = j * 32 + lane < a.V ? order_key(x[j]) : 0u;
    for (int c = 0; c < a.k; ++c) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int j = EPL - 1; j >= 0; --j)
            if (key[j] >= best) best = key[j], at = j;
        const uint32_t all = __reduce_max_sync(0xffffffffu, best);
        const int e = at * 32 + lane;
        const int index = static_cast<int>(__reduce_min_sync(0xffffffffu, best == all ? static_cast<uint32_t>(e) : 0xFFFFFFFFu));
        if (index == e) {
            write_top(a, row, c, entry_key(all, index), l);
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (j == at) key[j] = 0u;
        }
    }
}

// ------------------------------------------------------------------------------ distillation
struct DistillArgs {
    const void* logits;
    const void* ids;
    const float* top;
    const float* weight;
    float* loss;
    float* lse_out;
    const float* lse_in;   // given: only the gradient is computed
    void* dlogits;         // or null
    int64_t ld, ld_d;
    int n, V, k, wide_ids;
    float T, inv_t;
};

// The teacher's entries of a row: ids (-1 where left out) and probabilities, by a warp into shared
// memory; false for a row without any, or of weight 0.
__device__ __forceinline__ bool teacher(const DistillArgs& a, int64_t row, int* ids, float* p, float w) {
    const int lane = threadIdx.x & 31;
    float m = kNegInf;
    bool any = false;
    for (int c = lane; c < a.k; c += 32) {
        const int64_t at = row * a.k + c;
        const int64_t id = a.wide_ids ? __ldg(static_cast<const long long*>(a.ids) + at) : __ldg(static_cast<const int32_t*>(a.ids) + at);
        const float t = a.top ? __ldg(a.top + at) * a.inv_t : 0.f;
        const bool in = id >= 0 && id < a.V && t != kNegInf;
        ids[c] = in ? static_cast<int>(id) : -1;
        p[c] = t;
        any |= in;
        if (in) m = fmaxf(m, t);   // drops NaN, which the sum brings back
    }
    any = __any_sync(0xffffffffu, any) && w != 0.f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float s = 0.f;
    for (int c = lane; c < a.k; c += 32)
        if (ids[c] >= 0) s += p[c] = pow2((p[c] - m) * kLog2e);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    for (int c = lane; c < a.k; c += 32) p[c] = ids[c] >= 0 ? p[c] / s : 0.f;
    __syncwarp();
    return any;
}

// The logits at the teacher's entries, by the threads t of T, for the loss and the gradient there: read
// before any of the row's gradient is written, which may lie in place of the logits.
template <class TX, class F>
__device__ __forceinline__ void at_teacher(const DistillArgs& a, const Row<TX>& r, const int* ids, float* xs, int t, int T, F mine) {
    for (int c = t; c < a.k; c += T)
        if (ids[c] >= 0 && mine(ids[c])) xs[c] = r.at(ids[c]);
}

// w T^2 sum p (log p - log q) of a row, by a warp.
__device__ __forceinline__ float row_loss(const DistillArgs& a, const int* ids, const float* p, const float* xs, float w, float m, float log_s) {
    float t = 0.f;
    for (int c = threadIdx.x & 31; c < a.k; c += 32)
        if (ids[c] >= 0 && p[c] != 0.f) t += p[c] * (logf(p[c]) - ((xs[c] - m) * a.inv_t - log_s));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    return w * (a.T * a.T) * t;
}

// coef 2^(c (x - shift) - base) = w T q
struct Gradient {
    float c, shift, base, coef;
    __device__ __forceinline__ float operator()(float x) const { return coef * pow2(fmaf(x - shift, c, -base)); }
};

// Where the teacher has probability: w T (q - p), by the first entry of each id.
template <class TX>
__device__ __forceinline__ void teacher_gradient(const DistillArgs& a, const int* ids, const float* p, int c, float x, const Gradient& g, float wt, TX* d) {
    float sum = p[c];
    for (int o = 0; o < a.k; ++o) {
        if (ids[o] == ids[c] && o != c) {
            if (o < c) return;
            sum += p[o];
        }
    }
    const float v[1] = {g(x) - wt * sum};
    store_as<TX, 1>(d + ids[c], v);
}

// A row a cluster.  The gradient reads the row again (from L2).  VEC: the gradient's rows start at the
// same place of a 16-byte word as the logits' do.
template <class TX, int T, bool VEC>
__global__ void __launch_bounds__(T) distill_rows(const __grid_constant__ DistillArgs a) {
    constexpr int VE = Row<TX>::VE;
    __shared__ float s[3 * (T / 32)];
    __shared__ int ids[kMaxTeacher];
    __shared__ float p[kMaxTeacher], xs[kMaxTeacher];
    __shared__ int alive;
    uint32_t rank, size;
    cluster_place(rank, size);
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int64_t row = blockIdx.x / size;
    const float w = a.weight ? __ldg(a.weight + row) : 1.f;
    if (threadIdx.x < 32) {
        const bool any = teacher(a, row, ids, p, w);
        if (threadIdx.x == 0) alive = any;
    }
    __syncthreads();
    const Row<TX> r(a.logits, row, a.ld, a.V);
    int first, last;
    slice(r.nb, rank, size, first, last);
    const bool live = alive, edges = rank == 0;   // live: the same in every block of the cluster
    auto own = [&](int e) { return e < r.head || e >= r.tail0 ? edges : e >= r.head + first * VE && e < r.head + last * VE; };
    Gradient g{a.inv_t * kLog2e, 0.f, 0.f, 0.f};
    if (live && a.lse_in) {
        at_teacher(a, r, ids, xs, threadIdx.x, T, own);
        g.base = __ldg(a.lse_in + row) * kLog2e;
        g.coef = w * a.T;
        __syncthreads();
    } else if (live) {
        if (edges || a.dlogits) at_teacher(a, r, ids, xs, threadIdx.x, T, [](int) { return true; });
        Stats<false> st(g.c);
        read_row<TX, T, false>(r, first, last, edges, st);
        join_block<T, false>(st, s, rank, size);
        const float log_s = logf(st.s);
        if (edges && threadIdx.x < 32) {
            const float loss = row_loss(a, ids, p, xs, w, st.m, log_s);
            if (threadIdx.x == 0) {
                a.loss[row] = loss;
                if (a.lse_out) a.lse_out[row] = fmaf(st.m, a.inv_t, log_s);
            }
        }
        g.shift = st.m;
        g.coef = w * a.T / st.s;
    } else if (edges && threadIdx.x == 0 && !a.lse_in) {
        a.loss[row] = 0.f;
        if (a.lse_out) a.lse_out[row] = 0.f;
    }
    if (a.dlogits) {
        TX* d = static_cast<TX*>(a.dlogits) + row * a.ld_d;
#pragma unroll 4
        for (int i = first + static_cast<int>(threadIdx.x); i < last; i += T) {
            float v[VE];
            if (live) {
                const auto raw = load_raw<TX, VE>(r.word(i));
#pragma unroll
                for (int e = 0; e < VE; ++e) v[e] = g(raw_at<TX, VE>(raw, e));
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) v[e] = 0.f;
            }
            TX* to = d + r.head + static_cast<int64_t>(i) * VE;
            if constexpr (VEC) {
                store_as<TX, VE>(to, v);
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float one[1] = {v[e]};
                    store_as<TX, 1>(to + e, one);
                }
            }
        }
        if (edges && static_cast<int>(threadIdx.x) < r.edges()) {
            const int e = r.edge(threadIdx.x);
            const float v[1] = {live ? g(r.at(e)) : 0.f};
            store_as<TX, 1>(d + e, v);
        }
        __syncthreads();
        if (live)
            for (int c = threadIdx.x; c < a.k; c += T)
                if (ids[c] >= 0 && own(ids[c])) teacher_gradient(a, ids, p, c, xs[c], g, w * a.T, d);
    }
    if (size > 1) ptx::cluster_sync();   // the peers have read this block's sums
}

// A row of up to 32 EPL entries in a warp's registers.
template <class TX, int EPL>
__global__ void __launch_bounds__(128) distill_warps(const __grid_constant__ DistillArgs a) {
    __shared__ int ids4[4][kMaxTeacher];
    __shared__ float p4[4][kMaxTeacher], xs4[4][kMaxTeacher];
    ptx::pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + warp;
    int* ids = ids4[warp];
    float *p = p4[warp], *xs = xs4[warp];
    ptx::pdl_wait();
    if (row >= a.n) return;
    const float w = a.weight ? __ldg(a.weight + row) : 1.f;
    const bool live = teacher(a, row, ids, p, w);
    const Row<TX> r(a.logits, row, a.ld, a.V);
    float x[EPL];
    Gradient g{a.inv_t * kLog2e, 0.f, 0.f, 0.f};
    if (live) {
        float top = kNegInf;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            x[j] = j * 32 + lane < a.V ? r.at(j * 32 + lane) : kNegInf;
            top = fmaxf(top, x[j]);
        }
        at_teacher(a, r, ids, xs, lane, 32, [](int) { return true; });
        __syncwarp();
        if (a.lse_in) {
            g.base = __ldg(a.lse_in + row) * kLog2e;
            g.coef = w * a.T;
        } else {
            Stats<false> st(g.c);
            st.add(x, top);
            st.join_warp();
            const float log_s = logf(st.s), loss = row_loss(a, ids, p, xs, w, st.m, log_s);
            if (lane == 0) {
                a.loss[row] = loss;
                if (a.lse_out) a.lse_out[row] = fmaf(st.m, a.inv_t, log_s);
            }
            g.shift = st.m;
            g.coef = w * a.T / st.s;
        }
    } else if (lane == 0 && !a.lse_in) {
        a.loss[row] = 0.f;
        if (a.lse_out) a.lse_out[row] = 0.f;
    }
    if (!a.dlogits) return;
    TX* d = static_cast<TX*>(a.dlogits) + row * a.ld_d;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        if (j * 32 + lane < a.V) {
            const float v[1] = {live ? g(x[j]) : 0.f};
            store_as<TX, 1>(d + j * 32 + lane, v);
        }
    }
    __syncwarp();
    if (live)
        for (int c = lane; c < a.k; c += 32)
            if (ids[c] >= 0) teacher_gradient(a, ids, p, c, xs[c], g, w * a.T, d);
}

// ------------------------------------------------------------------------------ host side
bool sizes_ok(int64_t n, int64_t V) { return n >= 0 && V >= 1 && n < (1ll << 27) && V < (1ll << 31) - 65536; }
bool float_type(int t) { return t == TERN_BF16 || t == TERN_F32; }
int elem(int t) { return t == TERN_BF16 ? 2 : 4; }
bool ld_ok(int64_t ld, int64_t V) { return ld >= V && ld < (1ll << 40); }
bool aligned_to(const void* p, int b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }

// Blocks that share a row: none while the rows fill the GPU twice, and each thread keeps a word.
int row_blocks(int64_t n, int64_t V, int es, int T, int num_sms) {
    int c = 1;
    while (c < 16 && n * c < 2 * num_sms && V * es / (2 * c) >= 16 * T) c *= 2;
    return c;
}
bool narrow(int64_t V, int es) { return V * es <= 16384; }   // a block of 128 threads, else 512

template <class TX>
int run_score(const ScoreArgs& a, int num_sms, cudaStream_t s) {
    if (a.V <= 256) return launch_pdl(score_warps<TX, 8>, dim3((a.n + 3) / 4), dim3(128), 0, s, a);
    if (a.V <= kWarpRow) return launch_pdl(score_warps<TX, 32>, dim3((a.n + 3) / 4), dim3(128), 0, s, a);
    const bool few = narrow(a.V, kElem<TX>);
    const int c = row_blocks(a.n, a.V, kElem<TX>, few ? 128 : 512, num_sms);
    if (few) return launch_cluster(score_rows<TX, 128>, a.n * c, 128, 0, c, true, s, a);
    return launch_cluster(score_rows<TX, 512>, a.n * c, 512, 0, c, true, s, a);
}

template <class TX, int T>
int run_distill_rows(const DistillArgs& a, int num_sms, cudaStream_t s) {
    constexpr int es = kElem<TX>;
    const int c = row_blocks(a.n, a.V, es, T, num_sms);
    const bool vec = (reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.dlogits)) % 16 == 0 &&
                     (a.n <= 1 || (a.ld - a.ld_d) * es % 16 == 0);
    if (vec) return launch_cluster(distill_rows<TX, T, true>, a.n * c, T, 0, c, true, s, a);
    return launch_cluster(distill_rows<TX, T, false>, a.n * c, T, 0, c, true, s, a);
}

template <class TX>
int run_distill(const DistillArgs& a, int num_sms, cudaStream_t s) {
    if (a.V <= 256) return launch_pdl(distill_warps<TX, 8>, dim3((a.n + 3) / 4), dim3(128), 0, s, a);
    if (a.V <= kWarpRow) return launch_pdl(distill_warps<TX, 32>, dim3((a.n + 3) / 4), dim3(128), 0, s, a);
    return narrow(a.V, kElem<TX>) ? run_distill_rows<TX, 128>(a, num_sms, s) : run_distill_rows<TX, 512>(a, num_sms, s);
}

int distill(const tern_distillation* t, const float* lse_in, float* loss, float* lse, void* dlogits, int64_t ld_d, void* stream) {
    if (!t || !sizes_ok(t->n, t->V) || !float_type(t->dtype) || (t->ids_dtype != TERN_I32 && t->ids_dtype != TERN_I64)) return TERN_ERR_ARG;
    if (!ld_ok(t->ld, t->V) || (dlogits && !ld_ok(ld_d, t->V)) || t->k < 1 || t->k > kMaxTeacher) return TERN_ERR_ARG;
    if (!(t->temperature >= 1e-6f) || !(t->temperature <= 1e6f)) return TERN_ERR_ARG;
    if (t->n == 0) return TERN_OK;
    if (!t->logits || !t->ids || (!t->top && t->k > 1)) return TERN_ERR_ARG;
    const int es = elem(t->dtype);
    if (dlogits == t->logits && ld_d != t->ld && t->n > 1) return TERN_ERR_ARG;   // in place means row by row
    if (!aligned_to(t->logits, es) || !aligned_to(dlogits, es) || !aligned_to(t->ids, t->ids_dtype == TERN_I64 ? 8 : 4) || !aligned_to(t->top, 4) ||
        !aligned_to(t->weight, 4) || !aligned_to(lse_in, 4) || !aligned_to(loss, 4) || !aligned_to(lse, 4))
        return TERN_ERR_ALIGN;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    DistillArgs a{};
    a.logits = t->logits, a.ids = t->ids, a.top = t->top, a.weight = t->weight, a.loss = loss, a.lse_out = lse, a.lse_in = lse_in;
    a.dlogits = dlogits, a.ld = t->ld, a.ld_d = ld_d, a.n = static_cast<int>(t->n), a.V = static_cast<int>(t->V), a.k = t->k;
    a.wide_ids = t->ids_dtype == TERN_I64, a.T = t->temperature, a.inv_t = static_cast<float>(1.0 / static_cast<double>(t->temperature));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return t->dtype == TERN_BF16 ? run_distill<__nv_bfloat16>(a, num_sms, s) : run_distill<float>(a, num_sms, s);
}

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" int tern_score(const void* logits, int dtype, int64_t ld, int64_t n, int64_t V, const void* tokens, int tokens_dtype, float* logp,
                          float* entropy, float* lse, int k, int32_t* top_ids, float* top_logp, void* stream) {
    if (!sizes_ok(n, V) || !float_type(dtype) || !ld_ok(ld, V) || (tokens_dtype != TERN_I32 && tokens_dtype != TERN_I64)) return TERN_ERR_ARG;
    if (k < 0 || k > kMaxTop || k > V) return TERN_ERR_ARG;
    if (n == 0) return TERN_OK;
    if (!logits || (logp && !tokens) || (k > 0 && (!top_ids || !top_logp))) return TERN_ERR_ARG;
    if (!aligned_to(logits, elem(dtype)) || !aligned_to(tokens, tokens_dtype == TERN_I64 ? 8 : 4) || !aligned_to(logp, 4) ||
        !aligned_to(entropy, 4) || !aligned_to(lse, 4) || !aligned_to(top_ids, 4) || !aligned_to(top_logp, 4))
        return TERN_ERR_ALIGN;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    ScoreArgs a{};
    a.logits = logits, a.tokens = tokens, a.logp = logp, a.entropy = entropy, a.lse = lse, a.top_ids = top_ids, a.top_logp = top_logp;
    a.ld = ld, a.n = static_cast<int>(n), a.V = static_cast<int>(V), a.k = k, a.wide_ids = tokens_dtype == TERN_I64;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == TERN_BF16 ? run_score<__nv_bfloat16>(a, num_sms, s) : run_score<float>(a, num_sms, s);
}

extern "C" int tern_distill(const tern_distillation* t, float* loss, float* lse, void* dlogits, int64_t ld_dlogits, void* stream) {
    if (!loss && !(t && t->n == 0)) return TERN_ERR_ARG;
    return distill(t, nullptr, loss, lse, dlogits, ld_dlogits, stream);
}

extern "C" int tern_distill_bwd(const tern_distillation* t, const float* lse, void* dlogits, int64_t ld_dlogits, void* stream) {
    if ((!lse || !dlogits) && !(t && t->n == 0)) return TERN_ERR_ARG;
    return distill(t, lse, nullptr, nullptr, dlogits, ld_dlogits, stream);
}
