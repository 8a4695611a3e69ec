// What is computed from rows of logits: the log probability of a given token with the row's entropy and
// its most likely entries, and distillation from a teacher's top logits with its gradient.
//
//   m = max x, S = sum exp(x - m), lse = m + log S
//   logp = x[token] - lse,  entropy = log S - sum exp(x - m) (x - m) / S
//   loss = w T^2 sum p (log p - log q[id]),  dlogits = w T (q - p),   q = softmax(x / T)
//
// Memory bounds both: the score reads each logit once, the distillation reads it once and writes its
// gradient once.  One pass keeps a running maximum and sums relative to it; threads, blocks and the
// blocks of a cluster (which share a row where rows are few) are joined at the end.  Rows of up to 256
// entries belong to a warp each, which holds them in registers.
//
// Rows start at any element: whole 16-byte words of a row are its body, the few entries before and
// after them its head and tail.
//
// 4096 x 100003 in bf16 (0.82 GB): lse and entropy 125 us, 0.97 of the measured copy rate, with five
// alternatives 150, with 64 169: finding them waits (bound, list, words again, ranks) while the block reads
// nothing, and four blocks an SM cover that in part.  An entry takes five instructions by pairs of fp32 (a
// scalar form eight: 169 us without alternatives).  Loss and gradient 330 us, 0.74: the row is read twice, and
// L2 keeps it from the first to the second only with two blocks a row, whose exchange the next rows cover in
// part.  Rows held in shared memory by persistent clusters of eight blocks read memory once but took 1464 us
// (a teacher's entries by one warp, loops of unknown length).  One row of 100003: 4.5 us, with 20 alternatives 9.1: a
// chain of reading, bound, list, words again, ranks and the cluster's exchange with nothing beside it (which of
// these it waits for was not measured).  32768 x 700, distillation 57 us, floor 14: rows of fewer words than a whole
// batch of a warp are loaded a word at a time, an SM holds 32 such warps, and the forms with 32 threads spill
// 40 to 128 bytes (a teacher of up to 256 entries in registers).
#include <algorithm>
#include <cmath>

#include "pairs.cuh"
#include "rows.cuh"

namespace tern {
namespace {

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

// A softmax's maximum, sum of 2^(c (x - m)) and, for the entropy, the same with the factor (x - m);
// c = log2(e) / T.  The difference is taken first: it is exact near the maximum, where it counts.
template <bool ENT>
struct Stats {
    float m = kNegInf, s = 0.f, q = 0.f;

    // Relative to mn >= m (finite, or inf: then s becomes NaN, as it should).
    __device__ __forceinline__ void rebase(float mn, float c) {
        if (m != kNegInf) {   // of nothing but -inf s and q are 0, or s is NaN
            const float d = ENT ? fmaxf(m - mn, -1e4f) : m - mn, f = pow2(d * c);   // s d finite, whatever the maximum was
            if (ENT) q = (q + s * d) * f;
            s *= f;
        }
        m = mn;
    }
    // The sums of a warp's 32 in every lane, in a fixed order.
    __device__ __forceinline__ void join_warp(float c) {
        float mn = m;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
        rebase(mn, c);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, d);
            if (ENT) q += __shfl_xor_sync(0xffffffffu, q, d);
        }
    }
};

template <class T, int V>
__device__ __forceinline__ void raw_pairs(const Raw<T, V>& r, F2* x) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) x[i] = pair(raw_at<T, V>(r, 2 * i), raw_at<T, V>(r, 2 * i + 1));
}

// A thread's running softmax over batches of pairs.
template <bool ENT>
struct Run {
    float m = kNegInf;
    F2 s = both(0.f), q = both(0.f);

    // To the largest of a batch (NaN dropped); false while there is nothing but -inf (and NaN).
    __device__ __forceinline__ bool raise(float top, float c) {
        if (top > m) {
            if (m != kNegInf) {
                const float d = ENT ? fmaxf(m - top, -1e4f) : m - top, f = pow2(d * c);
                if (ENT) q = mul2(fma2(s, both(d), q), both(f));
                s = mul2(s, both(f));
            }
            m = top;
        }
        return m != kNegInf;
    }
    // `masked`: a difference may be -inf, which would give 0 times infinity in the entropy's sum.
    template <int N2>
    __device__ __forceinline__ void add(const F2 (&x)[N2], float top, bool masked, float c) {
        if (raise(top, c)) {
            const F2 shift = both(-m), scale = both(c);
#pragma unroll
            for (int i = 0; i < N2; ++i) one(add2(x[i], shift), masked, scale);
        } else {
            F2 t = x[0];
#pragma unroll
            for (int i = 1; i < N2; ++i) t = add2(t, x[i]);
            nan_of(t);
        }
    }
    // The same of U words as they are in memory.
    template <class T, int V, int U>
    __device__ __forceinline__ void add_words(const Raw<T, V> (&raw)[U], float top, bool masked, float c) {
        F2 x[V / 2];
        if (raise(top, c)) {
            const F2 shift = both(-m), scale = both(c);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw_pairs<T, V>(raw[u], x);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) one(add2(x[i], shift), masked, scale);
            }
        } else {
            F2 t = both(0.f);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw_pairs<T, V>(raw[u], x);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) t = add2(t, x[i]);
            }
            nan_of(t);
        }
    }
    __device__ __forceinline__ void nan_of(F2 t) {
        float lo, hi;
        split(t, lo, hi);
        if (lo + hi != lo + hi) s = both(lo + hi);
    }
    __device__ __forceinline__ void one(F2 z, bool masked, F2 scale) {
        if (ENT && masked) {
            float z0, z1;
            split(z, z0, z1);
            z = pair(max_nan(z0, -1e4f), max_nan(z1, -1e4f));
        }
        sum(z, scale);
    }
    __device__ __forceinline__ void sum(F2 z, F2 scale) {
        float t0, t1;
        split(mul2(z, scale), t0, t1);
        const F2 e = pair(pow2(t0), pow2(t1));
        s = add2(s, e);
        if (ENT) q = fma2(e, z, q);
    }
    __device__ __forceinline__ void add1(float x, float c) {
        const F2 one[1] = {pair(x, kNegInf)};
        add(one, x, true, c);
    }
    __device__ __forceinline__ Stats<ENT> get() const {
        Stats<ENT> r;
        float a, b;
        split(s, a, b);
        r.m = m, r.s = a + b;
        split(q, a, b);
        r.q = a + b;
        return r;
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

// The largest and the smallest of U words' entries (NaN dropped).
template <class T, int V, int U>
__device__ __forceinline__ float raw_max(const Raw<T, V> (&r)[U]) {
    if constexpr (kElem<T> == 2) {
        uint32_t m = r[0].w[0];
#pragma unroll
        for (int i = 1; i < U * V / 2; ++i) asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(r[i / (V / 2)].w[i % (V / 2)]));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    } else {
        float m = raw_at<T, V>(r[0], 0);
#pragma unroll
        for (int i = 1; i < U * V; ++i) m = fmaxf(m, raw_at<T, V>(r[i / V], i % V));
        return m;
    }
}
// Whether a difference to the maximum may be -inf: masked entries, or values near the type's ends.
template <class T, int V, int U>
__device__ __forceinline__ bool raw_masked(const Raw<T, V> (&r)[U], float top) {
    if constexpr (kElem<T> == 2) {
        uint32_t m = r[0].w[0];
#pragma unroll
        for (int i = 1; i < U * V / 2; ++i) asm("min.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(r[i / (V / 2)].w[i % (V / 2)]));
        return fminf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)) < -1e30f || top > 1e30f;
    } else {
        return true;   // looking costs what the bound that it would save does
    }
}

// The words that block `rank` of `size` takes of a row's body: [first, last).
__device__ __forceinline__ void slice(int nb, int rank, int size, int& first, int& last) {
    const int per = (nb + size - 1) / size;
    first = min(nb, rank * per);
    last = min(nb, first + per);
}

// One pass of a block of T threads over its words of a row (and, in block 0, the edges): thread t
// takes the words first + t, first + t + T, ...  With `tops`, each thread leaves the largest entry of
// each segment, `seg` of its words in turn (one, or a power of two from kBatch on; NaN dropped), at
// tops[segment T + t].
constexpr int kBatch = 4;      // words a thread asks for at once
constexpr int kSegments = 8;
__device__ __forceinline__ int segment_words(int words, int T) {
    const int each = (words + T - 1) / T;
    int seg = 1;
    while (seg * kSegments < each) seg = seg < kBatch ? kBatch : 2 * seg;
    return seg;
}

template <class TX, int T, bool ENT>
__device__ __forceinline__ Stats<ENT> read_row(const Row<TX>& r, int first, int last, bool edges, float c, float* tops = nullptr, int seg = 0) {
    constexpr int VE = Row<TX>::VE, U = kBatch;
    Run<ENT> run;
    int i = first + static_cast<int>(threadIdx.x);
    float most = kNegInf;   // of the segment
    int left = seg;
    float* to = tops + threadIdx.x;
    Raw<TX, VE> raw[U], next[U];   // the next batch is on its way while one is summed
    const auto ask = [&](Raw<TX, VE>(&to)[U], int at) {
        if (at + (U - 1) * T < last) {
#pragma unroll
            for (int u = 0; u < U; ++u) to[u] = load_raw<TX, VE>(r.word(at + u * T));
        }
    };
    ask(raw, i);
    for (; i + (U - 1) * T < last; i += U * T) {
        ask(next, i + U * T);
        const float top = raw_max(raw);
        if (ENT && !raw_masked(raw, top)) run.add_words(raw, top, false, c);
        else run.add_words(raw, top, true, c);
        if (ENT && tops && seg == 1) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Raw<TX, VE> one[1] = {raw[u]};
                *to = raw_max(one);
                to += T;
            }
        } else if (ENT && tops) {
            most = fmaxf(most, top);
            if ((left -= U) == 0) *to = most, to += T, most = kNegInf, left = seg;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = next[u];
    }
    for (; i < last; i += T) {
        const Raw<TX, VE> raw[1] = {load_raw<TX, VE>(r.word(i))};
        const float top = raw_max(raw);
        run.add_words(raw, top, true, c);
        if (ENT && tops) {
            most = fmaxf(most, top);
            if (--left == 0) *to = most, to += T, most = kNegInf, left = seg;
        }
    }
    if (ENT && tops && left < seg) *to = most;
    if (edges && static_cast<int>(threadIdx.x) < r.edges()) run.add1(r.at(r.edge(threadIdx.x)), c);
    return run.get();
}

// Joins the threads of a block through s (3 T / 32 floats); every thread holds the result.
template <int T, bool ENT>
__device__ __forceinline__ void join_block(Stats<ENT>& st, float* s, float c) {
    constexpr int W = T / 32;
    const int lane = threadIdx.x & 31;
    st.join_warp(c);
    if (lane == 0) {
        float* at = s + 3 * (threadIdx.x >> 5);
        at[0] = st.m, at[1] = st.s, at[2] = st.q;
    }
    __syncthreads();
    const bool in = lane < W;
    st.m = in ? s[3 * lane] : kNegInf, st.s = in ? s[3 * lane + 1] : 0.f, st.q = in ? s[3 * lane + 2] : 0.f;
    st.join_warp(c);
}

constexpr int kMaxBlocks = 16;   // of a cluster

// The blocks of a cluster push what the others need into their shared memory, so that no block waits at
// its end for the others to read its own: arrive at the start; wait (every block has started), push,
// arrive and wait.  For whole warps.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// This block's sums to slot `rank` of every block's `all` (4 floats each), by warp 0.
template <bool ENT>
__device__ __forceinline__ void push_stats(const Stats<ENT>& st, float4* all, uint32_t rank, uint32_t size) {
    if (threadIdx.x < size) {
        const uint32_t to = ptx::mapa_shared(ptx::smem_u32(all + rank), threadIdx.x);
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(st.m), "f"(st.s), "f"(st.q), "f"(0.f) : "memory");
    }
}
template <bool ENT>
__device__ __forceinline__ void join_cluster(Stats<ENT>& st, const float4* all, uint32_t size, float c) {
    const uint32_t lane = threadIdx.x & 31;
    const float4 v = lane < size ? all[lane] : make_float4(kNegInf, 0.f, 0.f, 0.f);
    st.m = v.x, st.s = v.y, st.q = v.z;
    st.join_warp(c);
}

__device__ __forceinline__ void cluster_place(uint32_t& rank, uint32_t& size) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(size));
}

// ------------------------------------------------------------------------------ score
//
// The k largest entries, the lower index first where equal: a thread's running maximum is at hand after
// the pass, and the k-th largest of the threads' maxima is a bound that at least k entries reach.  Few
// others do (about k + k^2 / 2T of T threads' entries in no order), so only the words of threads whose
// maximum reaches it are read again, from L2.  Entries are ordered by 64-bit keys, the value above
// the complement of the index, all different; each candidate's rank is the number of larger keys.
// Where more entries reach the bound than there is room for (masked rows, constant ones, large entries
// in few threads' words) the exact k-th value is found, by bisection if it must be, and entries equal
// to it are taken in the order of the row.
template <int T>
constexpr int kCand = T == 32 ? 512 : 1024;

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
    unsigned long long cand[kCand<T>];
    unsigned long long best[kMaxTop];
    unsigned long long lists[T == 32 ? 1 : kMaxBlocks * kMaxTop];   // the cluster's
    float tops[kSegments * T];                                      // read_row's
    uint16_t list[kSegments * T];
    int rank[kMaxTop];
    int count, listed;
    int warps[T / 32];
};

// Places for n of each lane in a list whose length is *count: one atomic a warp.
__device__ __forceinline__ int append(int* count, int n) {
    const int lane = threadIdx.x & 31;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
    }
    int base = 0;
    if (lane == 31 && incl) base = atomicAdd(count, incl);
    return __shfl_sync(0xffffffffu, base, 31) + incl - n;
}

// Every entry of the slice with a key of at least lo, as candidates; sp.count of them (kCand are kept).
// Only segments whose largest entry reaches lo are read again; all of them where there is NaN (`every`).
template <class TX, int T>
__device__ __forceinline__ void collect(const Row<TX>& r, int first, int last, bool edges, bool every, uint32_t lo, TopSpace<T>& sp) {
    constexpr int VE = Row<TX>::VE, U = kBatch;
    const int t = threadIdx.x, seg = 1 << (31 - __clz(segment_words(last - first, T)));   // a power of two, said so
    __syncthreads();
    if (t == 0) sp.count = sp.listed = 0;
    __syncthreads();
    // For finite bounds the floats compare as the keys do; it is NaN, reached by all, for a lo below -inf's key
    const float bound = key_value(lo);
    uint32_t mask = 0;
    for (int g = 0; first + t + g * seg * T < last; ++g)
        if (every || !(sp.tops[g * T + t] < bound)) mask |= 1u << g;
    __syncwarp();
    for (int at = append(&sp.listed, __popc(mask)); mask; mask &= mask - 1) sp.list[at++] = static_cast<uint16_t>((__ffs(mask) - 1) * T + t);
    __syncthreads();
    const int units = sp.listed * seg;
    for (int w0 = 0; w0 < units; w0 += U * T) {
        Raw<TX, VE> raw[U];
        int at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int w = w0 + u * T + t;
            at[u] = last;
            if (w < units) {
                const int item = sp.list[w / seg];
                at[u] = first + item % T + (item / T * seg + w % seg) * T;
            }
            if (at[u] < last) raw[u] = load_raw<TX, VE>(r.word(at[u]));
        }
        mask = 0;   // of the words' entries, VE bits each
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (at[u] < last) {
                const Raw<TX, VE> one[1] = {raw[u]};
                if (every || !(raw_max(one) < bound)) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float x = raw_at<TX, VE>(raw[u], e);
                        mask |= static_cast<uint32_t>(every ? order_key(x) >= lo : !(x < bound)) << (u * VE + e);
                    }
                }
            }
        }
        __syncwarp();
        for (int to = append(&sp.count, __popc(mask)); mask; mask &= mask - 1, ++to) {
            const int bit = __ffs(mask) - 1, u = bit / VE;
            int i = at[0];
#pragma unroll
            for (int v = 1; v < U; ++v)
                if (u == v) i = at[v];
            const int e = r.head + i * VE + bit % VE;
            if (to < kCand<T>) sp.cand[to] = entry_key(order_key(r.at(e)), e);
        }
    }
    if (edges && t < r.edges()) {
        const int e = r.edge(t);
        const uint32_t key = order_key(r.at(e));
        if (key >= lo) {
            const int to = atomicAdd(&sp.count, 1);
            if (to < kCand<T>) sp.cand[to] = entry_key(key, e);
        }
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
// `mine`: the largest key among the thread's entries, 0 without any; `most_key`: one that none is above;
// `every`: there is NaN.
template <class TX, int T>
__device__ __forceinline__ void block_top(const Row<TX>& r, int first, int last, bool edges, bool every, uint32_t mine, uint32_t most_key, int k, TopSpace<T>& sp) {
    constexpr int VE = Row<TX>::VE;
    uint32_t lo = 0;   // the upper 16 bits of the bound: all that bf16 has
    if constexpr (T == 32) {   // of the segments' maxima
        const int seg = segment_words(last - first, T), segs = every ? 1 : (last - first + seg * T - 1) / (seg * T);
        uint32_t top[kSegments], most = mine;
#pragma unroll
        for (int g = 0; g < kSegments; ++g)
            top[g] = !every && first + static_cast<int>(threadIdx.x) + g * seg * T < last ? order_key(sp.tops[g * T + threadIdx.x]) : 0u;
        if (every) top[0] = mine;
        if (k <= 8) {   // the lanes' largest in turn; several at once where equal: the bound is lower, and still one
            for (int c = 0; c < k; ++c) {
                lo = __reduce_max_sync(0xffffffffu, most);
                if (most == lo) most = 0;
            }
        } else {
            most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll 1
            for (int b = 31; b >= 16; --b) {
                const uint32_t c = lo | (1u << b);
                if (c > most) continue;
                int reach = 0;
#pragma unroll
                for (int g = 0; g < kSegments; ++g)
                    if (g < segs) reach += __popc(__ballot_sync(0xffffffffu, top[g] >= c));
                if (reach >= k) {
                    lo = c;
                    if (reach <= k + k / 4 + 2) break;   // near enough
                }
            }
        }
    } else {
#pragma unroll 1
        for (int b = 31; b >= 16; --b) {
            const uint32_t c = lo | (1u << b);
            if (c > most_key) continue;
            const int reach = __syncthreads_count(mine >= c);
            if (reach >= k) {
                lo = c;
                if (reach <= k + k / 4 + 2) break;
            }
        }
    }
    collect<TX, T>(r, first, last, edges, every, lo, sp);
    int n = sp.count;
    if (n > kCand<T>) {
        // Too many.  They may all be one value: every bf16 with the bound's upper bits (the lower are
        // ones where negative, and of NaN), and -inf, which alone has its own.
        bool one = kElem<TX> == 2 || lo >> 16 == 0x007Fu;
        if (one) {
            if (lo < 0x80000000u || lo >> 16 == 0xFFFFu) lo |= 0xFFFFu;
            collect<TX, T>(r, first, last, edges, every, lo + 1, sp);
            n = lo == 0xFFFFFFFFu ? 0 : sp.count;   // nothing is above NaN
            one = n < k;
        }
        if (n > kCand<T>) {   // the k-th largest value by bisection; at least k entries reach lo
            uint32_t v = 0;
#pragma unroll 1
            for (int b = 31; b >= 0; --b) {
                const uint32_t c = v | (1u << b);
                if (c <= lo || count_from<TX, T>(r, first, last, edges, c, sp) >= k) v = c;
            }
            lo = v;
            collect<TX, T>(r, first, last, edges, every, lo + 1, sp);
            n = lo == 0xFFFFFFFFu ? 0 : sp.count;
            one = true;
        }
        if (one) {
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
    }
    if constexpr (T == 32) {
        // Rows of few segments have a poor bound: the candidates are thinned out before they are compared
        // with one another (32768 x 700 with 64 alternatives: 301 us without)
        if (n > k + 32) {
            uint32_t v = 0;
#pragma unroll 1
            for (int b = 31; b >= 8; --b) {
                const uint32_t at = v | (1u << b);
                int reach = 0;
                for (int c = threadIdx.x; c < n; c += 32) reach += static_cast<uint32_t>(sp.cand[c] >> 32) >= at;
                reach = __reduce_add_sync(0xffffffffu, reach);
                if (reach >= k) {
                    v = at;
                    if (reach <= k + 8) break;
                }
            }
            int kept = 0;
            for (int c0 = 0; c0 < n; c0 += 32) {
                const int c = c0 + static_cast<int>(threadIdx.x);
                const unsigned long long key = c < n ? sp.cand[c] : 0ull;
                const bool keep = c < n && static_cast<uint32_t>(key >> 32) >= v;
                const uint32_t all = __ballot_sync(0xffffffffu, keep);   // every lane has read its candidate
                if (keep) sp.cand[kept + __popc(all & ((1u << threadIdx.x) - 1))] = key;
                kept += __popc(all);
                __syncwarp();
            }
            n = kept;
        }
    }
    for (int c = threadIdx.x; c < k; c += T)
        if (c >= n) sp.best[c] = 0ull;
    // several threads a candidate where there are enough
    int parts = 1;
    while (parts < 8 && n * parts * 2 <= T) parts *= 2;
    for (int c = threadIdx.x / parts; c < n; c += T / parts) {
        const unsigned long long key = sp.cand[c];
        int rank = 0;
#pragma unroll 4
        for (int o = threadIdx.x % parts; o < n; o += parts) rank += sp.cand[o] > key;
        // a candidate's threads are neighbours in a warp, all of them here (parts > 1: one round of all candidates)
        const uint32_t who = ((1u << parts) - 1) << ((threadIdx.x & 31) / parts * parts);
        for (int d = parts / 2; d >= 1; d >>= 1) rank += __shfl_xor_sync(who, rank, d);
        if (rank < k && threadIdx.x % parts == 0) sp.best[rank] = key;
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

__device__ __forceinline__ int row_token(const ScoreArgs& a, int64_t row) {   // -1: none, or outside the row
    if (!a.logp) return -1;
    const int64_t tok = a.wide_ids ? __ldg(static_cast<const long long*>(a.tokens) + row) : __ldg(static_cast<const int32_t*>(a.tokens) + row);
    return tok >= 0 && tok < a.V ? static_cast<int>(tok) : -1;
}
__device__ __forceinline__ void write_row(const ScoreArgs& a, int64_t row, int tok, float x, const Stats<true>& st, const RowLog& l) {
    if (a.lse) a.lse[row] = l.lse();
    if (a.entropy) a.entropy[row] = l.dead ? 0.f : fmaxf(l.log_s - st.q / st.s, 0.f) + (st.s != st.s ? st.s : 0.f);
    if (a.logp) a.logp[row] = tok >= 0 ? l.logp(x) : 0.f;
}

// A row a cluster (of one block, or of several where rows are few).
template <class TX, int T>
__global__ void __launch_bounds__(T, T == 256 ? 4 : T == 128 ? 8 : 32) score_rows(const __grid_constant__ ScoreArgs a) {
    __shared__ float s[3 * (T / 32)];
    __shared__ float4 all[kMaxBlocks];
    __shared__ TopSpace<T> sp;
    uint32_t rank = 0, size = 1;
    if constexpr (T > 32) cluster_place(rank, size);
    if (size > 1) cluster_arrive();
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int64_t row = blockIdx.x / size;
    const bool edges = rank == 0, writes = edges && threadIdx.x == 0;
    const int tok = writes ? row_token(a, row) : -1;
    const Row<TX> r(a.logits, row, a.ld, a.V);
    int first, last;
    slice(r.nb, rank, size, first, last);
    const int k = a.k;
    Stats<true> st = read_row<TX, T, true>(r, first, last, edges, kLog2e, k ? sp.tops : nullptr, k ? segment_words(last - first, T) : 0);
    const float xtok = tok >= 0 ? r.at(tok) : 0.f;   // under way while the sums are joined
    if (k) {
        const bool any = first + static_cast<int>(threadIdx.x) < last || (edges && static_cast<int>(threadIdx.x) < r.edges());
        uint32_t mine = any ? order_key(st.m) : 0u;
        // infinities and NaN: the maximum that the sums are relative to may not be the largest entry's key
        const bool every = __syncthreads_or(st.s != st.s);
        if (every) {
            mine = 0;
            for (int i = first + static_cast<int>(threadIdx.x); i < last; i += T) {
                const auto raw = load_raw<TX, Row<TX>::VE>(r.word(i));
#pragma unroll
                for (int e = 0; e < Row<TX>::VE; ++e) mine = max(mine, order_key(raw_at<TX, Row<TX>::VE>(raw, e)));
            }
            if (edges && static_cast<int>(threadIdx.x) < r.edges()) mine = max(mine, order_key(r.at(r.edge(threadIdx.x))));
        }
        join_block<T, true>(st, s, kLog2e);
        block_top<TX, T>(r, first, last, edges, every, mine, every ? 0xFFFFFFFFu : order_key(st.m), k, sp);
    } else {
        join_block<T, true>(st, s, kLog2e);
    }
    if (size == 1) {
        const RowLog l(st);
        if (writes) write_row(a, row, tok, xtok, st, l);
        for (int c = threadIdx.x; c < k; c += T) write_top(a, row, c, sp.best[c], l);
        return;
    }
    cluster_wait();   // every block has started
    push_stats(st, all, rank, size);
    const int lists = static_cast<int>(size);
    for (int w = threadIdx.x; w < k * lists; w += T) {
        const int c = w % k;
        const uint32_t to = ptx::mapa_shared(ptx::smem_u32(&sp.lists[rank * k + c]), static_cast<uint32_t>(w / k));
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(sp.best[c]) : "memory");
    }
    for (int c = threadIdx.x; c < k; c += T) sp.rank[c] = 0;
    cluster_arrive();
    cluster_wait();
    join_cluster(st, all, size, kLog2e);
    const RowLog l(st);
    if (writes) write_row(a, row, tok, xtok, st, l);
    // each block ranks its own entries among all blocks' sorted lists
    for (int w = threadIdx.x; w < k * lists; w += T) {
        const int c = w % k, o = w / k;
        const unsigned long long key = sp.best[c];
        int lo = 0, hi = k;   // entries of list o above the key: its first ones
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (sp.lists[o * k + mid] > key) lo = mid + 1;
            else hi = mid;
        }
        if (lo) atomicAdd(&sp.rank[c], lo);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < k; c += T)
        if (sp.best[c] && sp.rank[c] < k) write_top(a, row, sp.rank[c], sp.best[c], l);
}

// ---- rows of up to 256 entries, a warp each: EPL entries a lane.  VEC: as whole 16-byte words (row
// starts and width allow it), else lane by lane.
template <class TX, int EPL, bool VEC>
struct WarpRow {
    static constexpr int VE = VEC ? Row<TX>::VE : 1;
    TX* p;
    int V, lane;
    // entry of the lane's j-th register
    __device__ __forceinline__ int index(int j) const { return (j / VE) * 32 * VE + lane * VE + j % VE; }
    __device__ __forceinline__ void load(float (&x)[EPL]) const {
#pragma unroll
        for (int j = 0; j < EPL; j += VE) {
            const bool in = index(j) < V;
            Raw<TX, VE> raw;
            if (in) raw = load_raw<TX, VE>(p + index(j));
#pragma unroll
            for (int e = 0; e < VE; ++e) x[j + e] = in ? raw_at<TX, VE>(raw, e) : kNegInf;
        }
    }
    __device__ __forceinline__ void store(const float (&x)[EPL]) const {
#pragma unroll
        for (int j = 0; j < EPL; j += VE) {
            if (index(j) < V) {
                float v[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) v[e] = x[j + e];
                store_as<TX, VE>(p + index(j), v);
            }
        }
    }
};

template <int EPL, bool ENT>
__device__ __forceinline__ Stats<ENT> warp_stats(const float (&x)[EPL], float c) {
    float top = x[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) top = fmaxf(top, x[j]);
    F2 xx[EPL / 2];
#pragma unroll
    for (int j = 0; j < EPL / 2; ++j) xx[j] = pair(x[2 * j], x[2 * j + 1]);
    Run<ENT> run;
    run.add(xx, top, true, c);
    Stats<ENT> st = run.get();
    st.join_warp(c);
    return st;
}

// The k largest of a warp's entries into best, largest first: candidates from a bound as in block_top
// (the k-th largest of the maxima of groups of registers), their ranks by comparison.
template <int EPL, class R>
__device__ __forceinline__ void warp_top(const uint32_t (&key)[EPL], const R& row, int k, unsigned long long* cand, unsigned long long* best) {
    constexpr int G = EPL < 4 ? EPL : 4;   // groups a lane
    const int lane = threadIdx.x & 31;
    uint32_t lo = 0;
    if (k <= 8) {   // the lanes' maxima, largest first
        uint32_t top = key[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j) top = max(top, key[j]);
        for (int c = 0; c < k; ++c) {
            lo = __reduce_max_sync(0xffffffffu, top);
            if (top == lo) top = 0;   // several at once where equal: the bound is lower, and still one
        }
    } else {
        uint32_t top[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            top[g] = key[g];
#pragma unroll
            for (int j = g + G; j < EPL; j += G) top[g] = max(top[g], key[j]);
        }
#pragma unroll 1
        for (int b = 31; b >= 16; --b) {
            const uint32_t c = lo | (1u << b);
            int reach = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) reach += __popc(__ballot_sync(0xffffffffu, top[g] >= c));
            if (reach >= k) {
                lo = c;
                if (reach <= k + k / 4 + 2) break;
            }
        }
    }
    auto reach_of = [&](uint32_t c) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) n += key[j] >= c;
        return static_cast<int>(__reduce_add_sync(0xffffffffu, n));
    };
    lo = max(lo, 1u);   // 0: no entry
    int n = 0, most = -1;   // most: index of the last entry equal to lo that is wanted, -1 for all above lo and at it
    if (reach_of(lo) > k + 64) {
        // many equal ones, or a poor bound: the k-th value by bisection, and the index up to which entries equal to it count
        uint32_t v = 0;
#pragma unroll 1
        for (int b = 31; b >= 0; --b) {
            const uint32_t c = v | (1u << b);
            if (c <= lo || reach_of(c) >= k) v = c;
        }
        lo = v;
        const int want = k - (lo == 0xFFFFFFFFu ? 0 : reach_of(lo + 1));
        int from = 0, to = row.V - 1;   // the smallest index with `want` equal entries up to it
        while (from < to) {
            const int mid = (from + to) / 2;
            int c = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) c += key[j] == lo && row.index(j) <= mid;
            if (static_cast<int>(__reduce_add_sync(0xffffffffu, c)) >= want) to = mid;
            else from = mid + 1;
        }
        most = from;
    }
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const bool hit = key[j] > lo || (key[j] == lo && (most < 0 || row.index(j) <= most));
        const uint32_t hits = __ballot_sync(0xffffffffu, hit);
        if (hit) cand[n + __popc(hits & below)] = entry_key(key[j], row.index(j));
        n += __popc(hits);
    }
    __syncwarp();
    for (int c = lane; c < n; c += 32) {
        const unsigned long long mine = cand[c];
        int rank = 0;
        for (int o = 0; o < n; ++o) rank += cand[o] > mine;
        if (rank < k) best[rank] = mine;
    }
    __syncwarp();
}

template <class TX, int EPL, bool VEC>
__global__ void __launch_bounds__(128) score_warps(const __grid_constant__ ScoreArgs a) {
    __shared__ unsigned long long cand4[4][kMaxTop + 64], best4[4][kMaxTop];
    ptx::pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + warp;
    ptx::pdl_wait();
    if (row >= a.n) return;
    const Row<TX> r(a.logits, row, a.ld, a.V);
    const WarpRow<TX, EPL, VEC> wr{const_cast<TX*>(r.p), a.V, lane};
    const int tok = lane == 0 ? row_token(a, row) : -1;
    float x[EPL];
    wr.load(x);
    const float xtok = tok >= 0 ? r.at(tok) : 0.f;
    const Stats<true> st = warp_stats<EPL, true>(x, kLog2e);
    const RowLog l(st);
    if (lane == 0) write_row(a, row, tok, xtok, st, l);
    if (a.k == 0) return;
    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = wr.index(j) < a.V ? order_key(x[j]) : 0u;
    warp_top<EPL>(key, wr, a.k, cand4[warp], best4[warp]);
    for (int c = lane; c < a.k; c += 32) write_top(a, row, c, best4[warp][c], l);
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
// memory; false for a row without any, or of weight 0.  An entry counts by its difference to the largest,
// taken before the division by T: divided first, large entries would be infinite.
__device__ __forceinline__ bool teacher(const DistillArgs& a, int64_t row, int* ids, float* p, float w) {
    const int lane = threadIdx.x & 31;
    float m = kNegInf;
    bool any = false;
    for (int c = lane; c < a.k; c += 32) {
        const int64_t at = row * a.k + c;
        const int64_t id = a.wide_ids ? __ldg(static_cast<const long long*>(a.ids) + at) : __ldg(static_cast<const int32_t*>(a.ids) + at);
        const float t = a.top ? __ldg(a.top + at) : 0.f;
        const bool in = id >= 0 && id < a.V && t != kNegInf;
        ids[c] = in ? static_cast<int>(id) : -1;
        p[c] = t;
        any |= in;
        if (in) m = fmaxf(m, t);   // drops NaN, which the sum brings back
    }
    if (lane < 3 && a.k + lane < (a.k + 3) / 4 * 4) ids[a.k + lane] = -1;
    any = __any_sync(0xffffffffu, any) && w != 0.f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float s = 0.f;
    for (int c = lane; c < a.k; c += 32)
        if (ids[c] >= 0) s += p[c] = pow2((p[c] - m) * (a.inv_t * kLog2e));
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

// coef 2^(c (x - shift)) = w T q, from the maximum or (the gradient alone) from T lse
struct Gradient {
    float c, shift, coef;
    __device__ __forceinline__ float operator()(float x) const { return coef * pow2((x - shift) * c); }
    __device__ __forceinline__ void operator()(F2 x, float& a, float& b) const {
        float t0, t1;
        split(mul2(add2(x, both(-shift)), both(c)), t0, t1);
        split(mul2(pair(pow2(t0), pow2(t1)), both(coef)), a, b);
    }
};

// Where the teacher has probability: w T (q - p), by the first entry of each id.  ids is 16-byte aligned
// and goes on to a multiple of four with -1.
template <class TX>
__device__ __forceinline__ void teacher_gradient(const DistillArgs& a, const int* ids, const float* p, int c, float x, const Gradient& g, float wt, TX* d) {
    const int id = ids[c];
    float sum = p[c];
    for (int o = 0; o < a.k; o += 4) {
        const int4 v = *reinterpret_cast<const int4*>(ids + o);
        if (v.x == id || v.y == id || v.z == id || v.w == id) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (ids[o + i] == id && o + i != c) {
                    if (o + i < c) return;
                    sum += p[o + i];
                }
            }
        }
    }
    const float v[1] = {g(x) - wt * sum};
    store_as<TX, 1>(d + id, v);
}

// A row a cluster of blocks.  The gradient reads the row again, from L2 as far as it holds the rows in
// work.  The teacher's entries belong to the threads, E each; they are asked for before the row and their
// logits after it, so that only the block's exchange waits for them.  VEC: the gradient's rows start at
// the same place of a 16-byte word as the logits' do.
template <class TX, int T, bool VEC>
__global__ void __launch_bounds__(T, T == 256 ? 4 : T == 128 ? 8 : 32) distill_rows(const __grid_constant__ DistillArgs a) {
    constexpr int VE = Row<TX>::VE, U = kBatch, W = T / 32, E = (kMaxTeacher + T - 1) / T;
    __shared__ float s[3 * W], parts[W];
    __shared__ float2 teach[W];   // the warps' largest entry and sum relative to it
    __shared__ float4 all[kMaxBlocks];
    __shared__ __align__(16) int ids[kMaxTeacher];
    __shared__ float p[kMaxTeacher];
    uint32_t rank = 0, size = 1;
    if constexpr (T > 32) cluster_place(rank, size);
    if (size > 1) cluster_arrive();
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / size;
    const Row<TX> r(a.logits, row, a.ld, a.V);
    int first, last;
    slice(r.nb, rank, size, first, last);
    const bool edges = rank == 0;
    const float w = a.weight ? __ldg(a.weight + row) : 1.f;
    int id[E];
    float t[E], x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = e * T + threadIdx.x;
        id[e] = -1, t[e] = kNegInf, x[e] = 0.f;
        if (c < a.k) {
            const int64_t at = row * a.k + c;
            const int64_t of = a.wide_ids ? __ldg(static_cast<const long long*>(a.ids) + at) : __ldg(static_cast<const int32_t*>(a.ids) + at);
            t[e] = a.top ? __ldg(a.top + at) : 0.f;
            if (of >= 0 && of < a.V && t[e] != kNegInf) id[e] = static_cast<int>(of);
        }
    }
    auto own = [&](int e) { return e < r.head || e >= r.tail0 ? edges : e >= r.head + first * VE && e < r.head + last * VE; };
    Gradient g{a.inv_t * kLog2e, 0.f, 0.f};
    Stats<false> st;
    if (!a.lse_in) st = read_row<TX, T, false>(r, first, last, edges, g.c);
    // The entries' logits, before any of the gradient is written, which may lie in their place: all of them
    // for the loss, this block's own for the gradient (of which alone it can be sure in a gradient alone)
    float tm = kNegInf, ts = 0.f;
    bool any = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (e * T < a.k) {
            if (id[e] >= 0) {
                if (!a.lse_in || own(id[e])) x[e] = r.at(id[e]);
                tm = fmaxf(tm, t[e]);   // drops NaN, which the sum brings back
                any = true;
            }
        }
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, d));
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e * T < a.k && id[e] >= 0) ts += pow2((t[e] - tm) * g.c);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) ts += __shfl_xor_sync(0xffffffffu, ts, d);
    if (!a.lse_in) st.join_warp(g.c);
    if (lane == 0) {
        s[3 * warp] = st.m, s[3 * warp + 1] = st.s, s[3 * warp + 2] = 0.f;
        teach[warp] = make_float2(tm, ts);
    }
    const bool live = __syncthreads_or(any) && w != 0.f;   // the same in every block of the cluster
    {
        const float2 mine = lane < W ? teach[lane] : make_float2(kNegInf, 0.f);
        float m = mine.x;
#pragma unroll
        for (int d = W / 2; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        tm = __shfl_sync(0xffffffffu, m, 0);
        ts = mine.x == kNegInf ? mine.y : mine.y * pow2((mine.x - tm) * g.c);   // without an entry 0, or NaN
#pragma unroll
        for (int d = W / 2; d >= 1; d >>= 1) ts += __shfl_xor_sync(0xffffffffu, ts, d);
        ts = __shfl_sync(0xffffffffu, ts, 0);
    }
    if (a.lse_in) {
        g.shift = __ldg(a.lse_in + row) * a.T;
        g.coef = w * a.T;
        if (size > 1) cluster_wait();   // the arrival at the start
    } else {
        if constexpr (W > 1) {
            const bool in = lane < W;
            st.m = in ? s[3 * lane] : kNegInf, st.s = in ? s[3 * lane + 1] : 0.f;
            st.join_warp(g.c);
        }
        if (size > 1) {
            cluster_wait();   // every block has started
            push_stats(st, all, rank, size);
            cluster_arrive();
            cluster_wait();
            join_cluster(st, all, size, g.c);
        }
        g.shift = st.m;
        g.coef = w * a.T / st.s;
    }
    TX* d = static_cast<TX*>(a.dlogits) + row * a.ld_d;
    if (a.dlogits) {
        auto word = [&](const Raw<TX, VE>& x, int i) {
            float v[VE];
            if (live) {
                F2 xx[VE / 2];
                raw_pairs<TX, VE>(x, xx);
#pragma unroll
                for (int e = 0; e < VE / 2; ++e) g(xx[e], v[2 * e], v[2 * e + 1]);
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
        };
        int i = first + static_cast<int>(threadIdx.x);
        Raw<TX, VE> raw[U], next[U];
        const auto ask = [&](Raw<TX, VE>(&to)[U], int at) {
            if (at + (U - 1) * T < last) {
#pragma unroll
                for (int u = 0; u < U; ++u) to[u] = load_raw<TX, VE>(r.word(at + u * T));
            }
        };
        ask(raw, i);
        for (; i + (U - 1) * T < last; i += U * T) {
            ask(next, i + U * T);
#pragma unroll
            for (int u = 0; u < U; ++u) word(raw[u], i + u * T);
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = next[u];
        }
        for (; i < last; i += T) word(load_raw<TX, VE>(r.word(i)), i);
        if (edges && static_cast<int>(threadIdx.x) < r.edges()) {
            const int e = r.edge(threadIdx.x);
            const float v[1] = {live ? g(r.at(e)) : 0.f};
            store_as<TX, 1>(d + e, v);
        }
    }
    // the teacher's share: its probabilities, the loss, and the gradient at its entries
    const float log_s = logf(st.s);
    float loss = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = e * T + threadIdx.x;
        if (e * T < a.k && c < (a.k + 3) / 4 * 4) {
            const float q = id[e] >= 0 ? pow2((t[e] - tm) * g.c) / ts : 0.f;
            ids[c] = id[e], p[c] = q, t[e] = q;
            if (id[e] >= 0 && q != 0.f) loss += q * (logf(q) - ((x[e] - st.m) * a.inv_t - log_s));
        }
    }
    if (edges && !a.lse_in) {
#pragma unroll
        for (int d2 = 16; d2 >= 1; d2 >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, d2);
        if (lane == 0) parts[warp] = loss;
    }
    __syncthreads();   // and the row is written
    if (edges && !a.lse_in && threadIdx.x == 0) {
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < W; ++v) sum += parts[v];
        a.loss[row] = live ? w * (a.T * a.T) * sum : 0.f;
        if (a.lse_out) a.lse_out[row] = live ? fmaf(st.m, a.inv_t, log_s) : 0.f;
    }
    if (a.dlogits && live) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = e * T + threadIdx.x;
            if (e * T < a.k && id[e] >= 0 && own(id[e])) teacher_gradient(a, ids, p, c, x[e], g, w * a.T, d);
        }
    }
}

template <class TX, int EPL, bool VEC>
__global__ void __launch_bounds__(128) distill_warps(const __grid_constant__ DistillArgs a) {
    __shared__ __align__(16) int ids4[4][kMaxTeacher];
    __shared__ float p4[4][kMaxTeacher], xs4[4][kMaxTeacher];
    ptx::pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + warp;
    int* ids = ids4[warp];
    float *p = p4[warp], *xs = xs4[warp];
    ptx::pdl_wait();
    if (row >= a.n) return;
    const Row<TX> r(a.logits, row, a.ld, a.V);
    const WarpRow<TX, EPL, VEC> wr{const_cast<TX*>(r.p), a.V, lane};
    float x[EPL];
    wr.load(x);   // under way while the teacher's entries are read
    const float w = a.weight ? __ldg(a.weight + row) : 1.f;
    const bool live = teacher(a, row, ids, p, w);
    Gradient g{a.inv_t * kLog2e, 0.f, 0.f};
    if (live) {
        at_teacher(a, r, ids, xs, lane, 32, [](int) { return true; });
        if (a.lse_in) {
            g.shift = __ldg(a.lse_in + row) * a.T;
            g.coef = w * a.T;
        } else {
            const Stats<false> st = warp_stats<EPL, false>(x, g.c);
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
    __syncwarp();   // the entries' logits are read before the row is written, maybe in their place
#pragma unroll
    for (int j = 0; j < EPL; j += 2) g(pair(x[j], x[j + 1]), x[j], x[j + 1]);
    if (!live)
#pragma unroll
        for (int j = 0; j < EPL; ++j) x[j] = 0.f;
    TX* d = static_cast<TX*>(a.dlogits) + row * a.ld_d;
    const WarpRow<TX, EPL, VEC> wd{d, a.V, lane};
    wd.store(x);
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

// Threads of a block.  Where rows are many, a warp up to 16 KB (no barriers, many rows at once) and 128 up to
// 56 KB; distillation of bf16 rows with 32, 128 and 256 threads: 32768 x 700 58, 134, 238 us; 4096 x 8000 36,
// 40, 52; 4096 x 12000 54, 48, 59; 4096 x 20000 86, 69, 77; 4096 x 40000 168, 159, 126.  Scores cross at the
// same sizes, but with few alternatives to find 128 do up to 128 KB (8192 x 60000 with 10: 183, 216 us).
int row_block(int64_t n, int64_t V, int es, int num_sms, int64_t most = 57344) {
    const int64_t bytes = V * es;
    if (bytes <= 16384) return n >= 16 * num_sms ? 32 : 128;
    return bytes <= most && n >= 8 * num_sms ? 128 : 256;
}

// Blocks that share a row: twice as many until the rows fill the GPU twice, as long as each thread keeps a word.
int row_blocks(int64_t n, int64_t V, int es, int T, int num_sms) {
    int c = 1;
    while (T > 32 && c < kMaxBlocks && n * c < 2 * num_sms && V * es / (2 * c) >= 16 * T) c *= 2;
    return c;
}

// Whether a warp's rows can be taken in 16-byte words.
bool warp_words(const void* p, int64_t ld, int64_t n, int64_t V, int es) { return rows_allow(p, ld, n, V, 16 / es, es); }

constexpr int kWarpRow = 256;   // widest row that a warp holds in registers

template <class TX>
int run_score(const ScoreArgs& a, int num_sms, cudaStream_t s) {
    constexpr int es = kElem<TX>;
    if (a.V <= kWarpRow) {
        const dim3 grid((a.n + 3) / 4), block(128);
        if (warp_words(a.logits, a.ld, a.n, a.V, es)) return launch_pdl(score_warps<TX, kWarpRow / 32, true>, grid, block, 0, s, a);
        return launch_pdl(score_warps<TX, kWarpRow / 32, false>, grid, block, 0, s, a);
    }
    const int T = row_block(a.n, a.V, es, num_sms, a.k > 0 && a.k <= 32 ? 131072 : 57344), c = row_blocks(a.n, a.V, es, T, num_sms);
    if (T == 32) return launch_cluster(score_rows<TX, 32>, a.n, T, 0, 1, true, s, a);
    if (T == 128) return launch_cluster(score_rows<TX, 128>, a.n * c, T, 0, c, true, s, a);
    return launch_cluster(score_rows<TX, 256>, a.n * c, T, 0, c, true, s, a);
}

template <class TX, bool VEC>
int run_distill_rows(const DistillArgs& a, int num_sms, cudaStream_t s) {
    constexpr int es = kElem<TX>;
    const int T = row_block(a.n, a.V, es, num_sms);
    int c = row_blocks(a.n, a.V, es, T, num_sms);
    // Rows that L2 would not keep until the gradient reads them again, with four blocks of 256 threads an SM each
    // on its own: two blocks a row (4096 x 100003 bf16: 368 to 331 us; four cost more than they save, 397; the
    // loss alone 132, 163 and 220).
    if (T == 256 && c == 1 && a.dlogits && !a.lse_in && 4 * num_sms * static_cast<int64_t>(a.V) * es > (80 << 20)) c = 2;
    if (T == 32) return launch_cluster(distill_rows<TX, 32, VEC>, a.n, T, 0, 1, true, s, a);
    if (T == 128) return launch_cluster(distill_rows<TX, 128, VEC>, a.n * c, T, 0, c, true, s, a);
    return launch_cluster(distill_rows<TX, 256, VEC>, a.n * c, T, 0, c, true, s, a);
}

template <class TX>
int run_distill(const DistillArgs& a, int num_sms, cudaStream_t s) {
    constexpr int es = kElem<TX>;
    if (a.V <= kWarpRow) {
        const dim3 grid((a.n + 3) / 4), block(128);
        if (warp_words(a.logits, a.ld, a.n, a.V, es) && (!a.dlogits || warp_words(a.dlogits, a.ld_d, a.n, a.V, es)))
            return launch_pdl(distill_warps<TX, kWarpRow / 32, true>, grid, block, 0, s, a);
        return launch_pdl(distill_warps<TX, kWarpRow / 32, false>, grid, block, 0, s, a);
    }
    const bool vec = (reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.dlogits)) % 16 == 0 &&
                     (a.n <= 1 || (a.ld - a.ld_d) * es % 16 == 0);
    return vec ? run_distill_rows<TX, true>(a, num_sms, s) : run_distill_rows<TX, false>(a, num_sms, s);
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
