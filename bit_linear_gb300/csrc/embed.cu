// Embedding of tokens and the gradient of its table.
//
//   out[i]    = scale * table[tok[i]]                       (ids outside the table: a row of zeros)
//   dtable[k] = scale * sum over i with tok[i] = k of dout[i]   (ids outside the table: dropped)
//
// Forward: HBM-bound gather; a thread moves eight channels of a row (16-byte loads and stores, shifted
// into place where rows start at odd addresses).
//
// Gradient: the positions are sorted by token (stable radix sort, hand-written here) and each
// token's rows are then summed in the order of their positions, so no atomic adds in floating
// point and the same bits on every run.
//   sort     digits of up to 11 bits, one pass for tables below 2048 rows and two below 4 million:
//            digit counts per tile of positions, a scan of each digit's counts over the tiles,
//            then each tile of 1024 places its positions (rank within the tile from warp match
//            masks; tiles of 2048 leave SMs without one: 131072 x 512 into 256 rows 59 us, 53 us).
//            Up to 32768 positions one cluster does it all in one launch (32768 x 512 into 256
//            rows: 21 us, 34 us with three launches a pass; 65536: 32 us both ways)
//   sum      a block takes 256 sorted positions (64 where those are too few blocks) and 256
//            channels; each warp sums runs of equal tokens over its positions in registers; the
//            block joins the runs that cross its warps.  A run inside the block is written once,
//            straight to dtable.  The block's first run, if it began before the block, and its
//            last, if it goes on, go to a partial buffer.
//   join     for each run that leaves its block: the block where it begins adds the partials of
//            the blocks that it covers, in order.
// Rows of dtable without a token are written as zeros by extra blocks of the sum launch, which look
// them up in the sorted keys (with accumulate they are left alone).  Marking the rows with a token
// in the sort's last pass instead cost it a fifth of its time in stores to the same few sectors
// (131072 x 512 into 256 rows: the gradient 74 us, 64 us without).  Writing them beside the sort
// instead, on the SMs it leaves idle, was slower: 279 against 177 us at 32768 positions, 100003 x
// 2048.
// Bounded by HBM for large tables and batches: the forward of 32768 tokens from 100003 x 4096 in
// bf16 takes 67 us (0.79 of the measured copy rate for the rows' distinct bytes), the gradient of
// 32768 x 2048 into 100003 rows 167 us (0.84), of which the sums and zeros are 137.  A few thousand
// tokens are bound by the three launches: 8192 x 512 into 256 rows takes 14 us where the bytes
// would take 1.3.
#include <cuda_bf16.h>

#include "common.cuh"

namespace tern {
namespace {

constexpr int kMaxBits = 11;         // digit bits of a sort pass
constexpr int kSortTile = 1024;      // positions per block of the sort (256 threads x 4)
constexpr int kChTile = 256;         // channels per block of the sum
// Of rows that start anywhere, 31 lanes' worth: a lane's channels straddle its 16 bytes and the next
// lane's (100000 rows of 513 into 50000: 94 us, by single elements 175).
template <bool WIDE>
__host__ __device__ constexpr int tile_channels() { return WIDE ? kChTile : kChTile - 8; }

// ------------------------------------------------------------------------------ forward
struct EmbedArgs {
    const void* tokens;
    const void* table;
    __nv_bfloat16* out;
    int64_t n, ld_out;
    int V, D;
    float scale;
};

template <class TOK>
__device__ __forceinline__ int token_row(const void* tokens, int64_t i, int V) {
    const TOK t = __ldg(static_cast<const TOK*>(tokens) + i);
    return t >= 0 && t < static_cast<TOK>(V) ? static_cast<int>(t) : -1;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}

// Eight bf16 from the sh-th on of two neighbouring 16-byte words.
__device__ __forceinline__ uint4 realign8(const uint4& a, const uint4& b, int sh) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (sh & 4) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (sh & 2) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const int bits = (sh & 1) * 16;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

// Eight elements from any address of the table that ends at `end`: the 16-byte words around them where
// those are the table's own, else one by one.
__device__ __forceinline__ void load8_any(const __nv_bfloat16* p, const void* table, const void* end, float (&x)[8]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), lo = at & ~static_cast<uintptr_t>(15);
    const int sh = static_cast<int>(at - lo) / 2;
    if (lo >= reinterpret_cast<uintptr_t>(table) && lo + 32 <= reinterpret_cast<uintptr_t>(end)) {
        const uint4* w = reinterpret_cast<const uint4*>(lo);
        unpack8(realign8(__ldg(w), __ldg(w + 1), sh), x);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __bfloat162float(p[k]);
    }
}
__device__ __forceinline__ void load8_any(const float* p, const void* table, const void* end, float (&x)[8]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), lo = at & ~static_cast<uintptr_t>(15);
    const int sh = static_cast<int>(at - lo) / 4;
    if (lo >= reinterpret_cast<uintptr_t>(table) && lo + 48 <= reinterpret_cast<uintptr_t>(end)) {
        const float4* w = reinterpret_cast<const float4*>(lo);
        const float4 a = __ldg(w), b = __ldg(w + 1), c = __ldg(w + 2);
        float v[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
        if (sh & 2) {
#pragma unroll
            for (int i = 0; i < 9; ++i) v[i] = v[i + 2];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = sh & 1 ? v[k + 1] : v[k];
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __ldg(p + k);
    }
}

// Eight channels per thread by 16-byte accesses: WIDE, rows start on such boundaries; otherwise the
// output's boundaries are taken and the table's words realigned to them (100000 rows of 513: 49 us, by
// single elements 94).  tx threads (a power of two) share a row.  MANY: a block has several rows, and
// reads a row's token before the row in hand is done.  It is for grids larger than the GPU holds, of rows
// that are one chunk per thread (65536 x 1024: 40 us, 52 us with a block for every four rows; 32768 x 4096
// in bf16, two chunks: 70 and 67 us; odd widths gain nothing; small grids lose 0.4 us).
template <class TOK, class TAB, bool WIDE, bool MANY>
__global__ void __launch_bounds__(256) tern_embed_fwd_kernel(const __grid_constant__ EmbedArgs a, int tx) {
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int x = threadIdx.x & (tx - 1), ty = threadIdx.x / tx;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (256 / tx);
    int64_t i = static_cast<int64_t>(blockIdx.x) * (256 / tx) + ty;
    if (i >= a.n) return;
    int row = token_row<TOK>(a.tokens, i, a.V);
    for (;;) {
        int next = -1;
        if (MANY && i + stride < a.n) next = token_row<TOK>(a.tokens, i + stride, a.V);
        const TAB* src = static_cast<const TAB*>(a.table) + static_cast<int64_t>(max(row, 0)) * a.D;
        __nv_bfloat16* dst = a.out + i * a.ld_out;
        // channels [head, tail) lie between the output's 16-byte boundaries, eight threads take those before
        // and eight those after, one each
        int head = 0, tail = a.D, edge = -1;
        float at_edge = 0.0f;
        if constexpr (!WIDE) {
            head = min(static_cast<int>((16 - reinterpret_cast<uintptr_t>(dst) % 16) % 16 / 2), a.D);
            tail = head + (a.D - head) / 8 * 8;
            if (x < 8 ? x < head : x < 16 && tail + x - 8 < a.D) edge = x < 8 ? x : tail + x - 8;
            if (row >= 0 && edge >= 0) at_edge = static_cast<float>(src[edge]) * a.scale;
        }
#pragma unroll 4
        for (int d = head + x * 8; d < tail; d += tx * 8) {
            float v[8] = {};
            if (row >= 0) {
                if constexpr (!WIDE) {
                    load8_any(src + d, a.table, static_cast<const TAB*>(a.table) + static_cast<int64_t>(a.V) * a.D, v);
                } else if constexpr (sizeof(TAB) == 4) {
                    const float4 p = __ldg(reinterpret_cast<const float4*>(src + d));
                    const float4 q = __ldg(reinterpret_cast<const float4*>(src + d) + 1);
                    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
                } else {
                    unpack8(__ldg(reinterpret_cast<const uint4*>(src + d)), v);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= a.scale;
            }
            *reinterpret_cast<uint4*>(dst + d) = pack8(v);
        }
        if (edge >= 0) dst[edge] = __float2bfloat16_rn(at_edge);
        i += stride;
        if (!MANY || i >= a.n) return;
        row = next;
    }
}

// ------------------------------------------------------------------------------ the sort
struct SortArgs {
    const void* tokens;        // first pass: the ids; later: null
    const int32_t* keys_in;
    const int32_t* pos_in;
    int32_t* keys_out;
    int32_t* pos_out;
    int32_t* counts;           // [digits][tiles], then (scanned) each tile's offset within the digit
    int32_t* totals;           // [digits]
    int n, V, tiles, shift, bits, tokens64;
};

// The key of position i: its token, or V for an id outside the table (sorted to the end).
__device__ __forceinline__ int sort_key(const SortArgs& a, int i) {
    if (a.tokens == nullptr) return a.keys_in[i];
    const int row = a.tokens64 ? token_row<long long>(a.tokens, i, a.V) : token_row<int>(a.tokens, i, a.V);
    return row >= 0 ? row : a.V;
}

__global__ void __launch_bounds__(256) tern_embed_count_kernel(const __grid_constant__ SortArgs a) {
    __shared__ int32_t hist[1 << kMaxBits];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int digits = 1 << a.bits;
    for (int k = threadIdx.x; k < digits; k += 256) hist[k] = 0;
    __syncthreads();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortTile;
#pragma unroll
    for (int r = 0; r < kSortTile / 256; ++r) {
        const int64_t i = base + r * 256 + threadIdx.x;
        if (i < a.n) atomicAdd(&hist[(sort_key(a, static_cast<int>(i)) >> a.shift) & (digits - 1)], 1);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < digits; k += 256) a.counts[static_cast<int64_t>(k) * a.tiles + blockIdx.x] = hist[k];
}

// Exclusive scan of each digit's counts over the tiles, one warp per digit; the sum to totals.
__global__ void __launch_bounds__(256) tern_embed_offsets_kernel(int32_t* counts, int32_t* totals, int digits, int tiles) {
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int k = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (k >= digits) return;
    int32_t* c = counts + static_cast<int64_t>(k) * tiles;
    int run = 0;
    for (int t0 = 0; t0 < tiles; t0 += 32) {
        const int t = t0 + lane;
        const int x = t < tiles ? c[t] : 0;
        int s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (t < tiles) c[t] = run + s - x;
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) totals[k] = run;
}

// Stable placement: within a tile the order is (warp, round, lane), as the positions lie.
__global__ void __launch_bounds__(256) tern_embed_place_kernel(const __grid_constant__ SortArgs a) {
    __shared__ int32_t base[1 << kMaxBits];            // where this tile's positions of a digit go
    __shared__ uint16_t cnt[8][1 << kMaxBits];         // per warp: count of a digit, then its offset in the tile
    __shared__ int32_t wsum[8];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int digits = 1 << a.bits, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int k = threadIdx.x; k < digits * 4; k += 256) reinterpret_cast<uint32_t*>(&cnt[k / (digits / 2)][0])[k % (digits / 2)] = 0;
    // exclusive scan of the digits' totals: each thread takes `per` consecutive digits
    const int per = (digits + 255) / 256;
    int own = 0;
    for (int j = 0; j < per; ++j) {
        const int k = threadIdx.x * per + j;
        own += k < digits ? a.totals[k] : 0;
    }
    int s = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    if (lane == 31) wsum[w] = s;
    __syncthreads();
    int before = s - own;
    for (int k = 0; k < w; ++k) before += wsum[k];
    for (int j = 0; j < per; ++j) {
        const int k = threadIdx.x * per + j;
        if (k < digits) {
            base[k] = before + a.counts[static_cast<int64_t>(k) * a.tiles + blockIdx.x];
            before += a.totals[k];
        }
    }
    // ranks within the warp's positions
    constexpr int R = kSortTile / 256;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortTile + w * (32 * R);
    int key[R], rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = i0 + r * 32 + lane < a.n ? sort_key(a, static_cast<int>(i0 + r * 32 + lane)) : -1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int dg = key[r] >= 0 ? (key[r] >> a.shift) & (digits - 1) : digits;
        const uint32_t same = __match_any_sync(0xffffffffu, dg);
        const uint32_t lower = same & ((1u << lane) - 1u);
        rank[r] = 0;
        if (dg < digits) rank[r] = cnt[w][dg] + __popc(lower);
        __syncwarp();
        if (dg < digits && lower == 0) cnt[w][dg] = static_cast<uint16_t>(cnt[w][dg] + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    for (int k = threadIdx.x; k < digits; k += 256) {
        int run = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = cnt[j][k];
            cnt[j][k] = static_cast<uint16_t>(run);
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (key[r] < 0) continue;
        const int i = static_cast<int>(i0) + r * 32 + lane;
        const int dg = (key[r] >> a.shift) & (digits - 1);
        const int at = base[dg] + cnt[w][dg] + rank[r];
        a.keys_out[at] = key[r];
        a.pos_out[at] = a.pos_in != nullptr ? a.pos_in[i] : i;
    }
}

// The whole sort by one cluster, for up to 16 * WARPS * 32 * R positions: every block ranks a tile of
// WARPS * 32 * R, the digits' counts are exchanged through distributed shared memory, and the passes
// follow one another in the launch (count, offsets and place take three launches a pass otherwise,
// most of the time of a sort of some thousand tokens).
struct ClusterSortArgs {
    SortArgs s;                // tokens, V, n, bits
    int32_t *keys[2], *pos[2]; // pass i reads i-1 and writes i & 1
    int passes;
};

template <int WARPS, int R>
__global__ void __launch_bounds__(WARPS * 32) tern_embed_sort_kernel(const __grid_constant__ ClusterSortArgs g) {
    constexpr int THREADS = WARPS * 32, TILE = THREADS * R;
    extern __shared__ __align__(16) char smem[];
    const int digits = 1 << g.s.bits;
    int32_t* hist = reinterpret_cast<int32_t*>(smem);                    // this tile's counts, read by the peers
    int32_t* base = hist + digits;                                      // where its positions of a digit go
    uint16_t* cnt = reinterpret_cast<uint16_t*>(base + digits);         // [WARPS][digits]
    __shared__ int32_t wsum[WARPS];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, P = gridDim.x, rank = blockIdx.x;
    const int64_t i0 = static_cast<int64_t>(rank) * TILE + w * (32 * R);
    for (int pass = 0; pass < g.passes; ++pass) {
        const int shift = pass * g.s.bits;
        int key[R], at[R], rk[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = i0 + r * 32 + lane;
            key[r] = -1, at[r] = static_cast<int>(i);
            if (i < g.s.n) {
                if (pass == 0) {
                    key[r] = sort_key(g.s, static_cast<int>(i));
                } else {
                    key[r] = __ldcg(g.keys[(pass - 1) & 1] + i);
                    at[r] = __ldcg(g.pos[(pass - 1) & 1] + i);
                }
            }
        }
        for (int k = threadIdx.x; k < WARPS * digits / 2; k += THREADS) reinterpret_cast<uint32_t*>(cnt)[k] = 0u;
        __syncthreads();
        uint16_t* mine = cnt + w * digits;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int dg = key[r] >= 0 ? (key[r] >> shift) & (digits - 1) : digits;
            const uint32_t same = __match_any_sync(0xffffffffu, dg);
            const uint32_t lower = same & ((1u << lane) - 1u);
            rk[r] = dg < digits ? mine[dg] + __popc(lower) : 0;
            __syncwarp();
            if (dg < digits && lower == 0) mine[dg] = static_cast<uint16_t>(mine[dg] + __popc(same));
            __syncwarp();
        }
        __syncthreads();
        for (int k = threadIdx.x; k < digits; k += THREADS) {
            int run = 0;
            for (int j = 0; j < WARPS; ++j) {
                const int x = cnt[j * digits + k];
                cnt[j * digits + k] = static_cast<uint16_t>(run);
                run += x;
            }
            hist[k] = run;
        }
        __syncwarp();   // the cluster's barriers are for whole warps
        ptx::cluster_sync();
        // of each digit: the counts of the tiles before this one, and of all; then a scan over the digits.
        // Two neighbouring digits a read: the exchange is bound by the number of requests.
        const int per = (digits + 2 * THREADS - 1) / (2 * THREADS) * 2;
        int own = 0;
        for (int j = 0; j < per; j += 2) {
            const int k = threadIdx.x * per + j;
            if (k >= digits) break;
            const uint32_t here = ptx::smem_u32(hist + k);
            int b0 = 0, b1 = 0, t0 = 0, t1 = 0;
            for (int q = 0; q < P; ++q) {
                int x, y;
                asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(ptx::mapa_shared(here, q)) : "memory");
                if (q < rank) b0 += x, b1 += y;
                t0 += x, t1 += y;
            }
            base[k] = own + b0;          // without the digits of lower threads, added below
            base[k + 1] = own + t0 + b1;
            own += t0 + t1;
        }
        // the last pass: after this the peers' counts are read no more
        const bool last = pass + 1 == g.passes;
        __syncwarp();
        if (last) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) wsum[w] = sum;
        __syncthreads();
        int lower_threads = sum - own;
        for (int k = 0; k < w; ++k) lower_threads += wsum[k];
        for (int j = 0; j < per; ++j) {
            const int k = threadIdx.x * per + j;
            if (k < digits) base[k] += lower_threads;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (key[r] < 0) continue;
            const int dg = (key[r] >> shift) & (digits - 1);
            const int to = base[dg] + mine[dg] + rk[r];
            g.keys[pass & 1][to] = key[r];
            g.pos[pass & 1][to] = at[r];
        }
        __syncwarp();
        if (last) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // the peers have read hist
        else ptx::cluster_sync();                                              // and the placed keys are visible to them
    }
}

// ------------------------------------------------------------------------------ the sums
struct RunArgs {
    const int32_t* keys;       // sorted
    const int32_t* pos;
    const __nv_bfloat16 *dout, *dout_end;
    float* dtable;
    float* partial;            // [run tiles][2][D]: 0 the run that began before the tile, 1 the one that goes on
    int64_t ld_dout;
    int n, V, D, run, run_tiles, ch_tiles;   // run: sorted positions per block of the sum
    int accumulate;
    float scale;
};

// Channels c0 + 8 lane onwards of a row's sum to dtable: WIDE by 16 bytes, else by way of `stage`.
template <bool WIDE>
__device__ __forceinline__ void write_row(const RunArgs& a, int key, int c0, int lane, const float (&x)[8], float* stage) {
    float* row = a.dtable + static_cast<int64_t>(key) * a.D;
    if constexpr (WIDE) {
        const int c = c0 + lane * 8;
        if (c >= a.D) return;
        float4* p = reinterpret_cast<float4*>(row + c);
        float4 u = make_float4(x[0] * a.scale, x[1] * a.scale, x[2] * a.scale, x[3] * a.scale);
        float4 v = make_float4(x[4] * a.scale, x[5] * a.scale, x[6] * a.scale, x[7] * a.scale);
        if (a.accumulate) {
            const float4 s = p[0], t = p[1];
            u = make_float4(s.x + u.x, s.y + u.y, s.z + u.z, s.w + u.w);
            v = make_float4(t.x + v.x, t.y + v.y, t.z + v.z, t.w + v.w);
        }
        p[0] = u, p[1] = v;
    } else {
        __syncwarp();
        *reinterpret_cast<float4*>(stage + 8 * lane) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(stage + 8 * lane + 4) = make_float4(x[4], x[5], x[6], x[7]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = k * 32 + lane;
            if (c < tile_channels<WIDE>() && c0 + c < a.D) row[c0 + c] = (a.accumulate ? row[c0 + c] : 0.0f) + stage[c] * a.scale;
        }
    }
}

// Zeros for the rows that have no token: warp `warp` of `warps` takes every warps-th row, whose
// lanes look 32 of them up in the sorted keys.
template <bool WIDE>
__device__ __forceinline__ void fill_rows(const RunArgs& a, int64_t warp, int64_t warps, int lane) {
    for (int64_t v0 = warp; v0 < a.V; v0 += 32 * warps) {
        const int64_t v = v0 + lane * warps;
        bool absent = v < a.V;
        if (absent) {
            int lo = 0, hi = a.n;
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                if (a.keys[mid] < v) lo = mid + 1;
                else hi = mid;
            }
            absent = lo == a.n || a.keys[lo] != v;
        }
        for (uint32_t m = __ballot_sync(0xffffffffu, absent); m != 0u; m &= m - 1u) {
            float* row = a.dtable + (v0 + (__ffs(m) - 1) * warps) * a.D;
            if constexpr (WIDE) {
                for (int c = lane * 4; c < a.D; c += 128) __stcs(reinterpret_cast<float4*>(row + c), make_float4(0.f, 0.f, 0.f, 0.f));
            } else {
                for (int c = lane; c < a.D; c += 32) __stcs(row + c, 0.0f);
            }
        }
    }
}

// PW: positions per warp.
template <bool WIDE, int PW>
__global__ void __launch_bounds__(256) tern_embed_sum_kernel(const __grid_constant__ RunArgs a) {
    constexpr int CH = tile_channels<WIDE>();
    __shared__ alignas(16) float first_s[8][kChTile], last_s[8][kChTile];
    __shared__ int first_key[8], last_key[8];   // of a warp's positions; -1 without any
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = blockIdx.x;
    if (unit >= static_cast<int64_t>(a.run_tiles) * a.ch_tiles) {
        const int64_t sums = static_cast<int64_t>(a.run_tiles) * a.ch_tiles;
        fill_rows<WIDE>(a, (unit - sums) * 8 + w, (gridDim.x - sums) * 8, lane);
        return;
    }
    const int tile = static_cast<int>(unit / a.ch_tiles), c0 = static_cast<int>(unit % a.ch_tiles) * CH;
    const int p0 = tile * (8 * PW) + w * PW;
    const int mine = lane < PW && p0 + lane < a.n ? a.keys[p0 + lane] : a.V;
    const int where = mine < a.V ? a.pos[p0 + lane] : 0;
    const int cnt = __popc(__ballot_sync(0xffffffffu, mine < a.V));   // sorted: the live ones come first
    float acc[8] = {};
    int cur = __shfl_sync(0xffffffffu, mine, 0);
    bool first = true;      // still in the warp's first run
    if (lane == 0) first_key[w] = cnt > 0 ? cur : -1;
    constexpr int U = 8;    // rows in flight
    for (int i0 = 0; i0 < cnt; i0 += U) {
        uint4 raw[U];
        uint32_t shifts = 0;     // elements between a row's 16-byte boundary and its channel c0
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int src = __shfl_sync(0xffffffffu, where, i0 + u);
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (i0 + u < cnt) {
                const __nv_bfloat16* row = a.dout + static_cast<int64_t>(src) * a.ld_dout + c0;
                if constexpr (WIDE) {
                    if (c0 + lane * 8 < a.D) raw[u] = __ldg(reinterpret_cast<const uint4*>(row + lane * 8));
                } else {
                    const uintptr_t at = reinterpret_cast<uintptr_t>(row), lo = (at & ~static_cast<uintptr_t>(15)) + 16 * lane;
                    const int sh = static_cast<int>(at & 15) / 2;
                    shifts |= static_cast<uint32_t>(sh) << (4 * u);
                    if (c0 + lane * 8 - sh >= a.D) continue;
                    if (lo >= reinterpret_cast<uintptr_t>(a.dout) && lo + 16 <= reinterpret_cast<uintptr_t>(a.dout_end)) {
                        raw[u] = __ldg(reinterpret_cast<const uint4*>(lo));
                    } else {   // the tensor's first or last bytes
                        uint32_t h[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const unsigned short* e = reinterpret_cast<const unsigned short*>(lo) + k;
                            h[k] = e >= reinterpret_cast<const unsigned short*>(a.dout) && e < reinterpret_cast<const unsigned short*>(a.dout_end) ? *e : 0u;
                        }
                        raw[u] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= cnt) break;
            const int key = __shfl_sync(0xffffffffu, mine, i0 + u);
            if (key != cur) {
                if (first) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) first_s[w][lane * 8 + k] = acc[k];
                    first = false;
                } else {
                    write_row<WIDE>(a, cur, c0, lane, acc, last_s[w]);   // not in use before the end
                }
                cur = key;
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
            }
            if constexpr (!WIDE) {
                uint4 next;
                next.x = __shfl_down_sync(0xffffffffu, raw[u].x, 1), next.y = __shfl_down_sync(0xffffffffu, raw[u].y, 1);
                next.z = __shfl_down_sync(0xffffffffu, raw[u].z, 1), next.w = __shfl_down_sync(0xffffffffu, raw[u].w, 1);
                raw[u] = realign8(raw[u], next, shifts >> (4 * u) & 7);
            }
            float x[8];
            unpack8(raw[u], x);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] += x[k];
        }
    }
    // the warp's open run: its only one (first) or its last
    if constexpr (!WIDE) __syncwarp();   // write_row's reads of last_s
#pragma unroll
    for (int k = 0; k < 8; ++k) (first ? first_s : last_s)[w][lane * 8 + k] = acc[k];
    if (lane == 0) last_key[w] = cnt == 0 ? -1 : (first ? -2 : cur);   // -2: a single run
    __syncthreads();
    // join the runs across the warps, a thread per channel
    const int c = c0 + threadIdx.x;
    if (threadIdx.x >= CH || c >= a.D || first_key[0] < 0) return;
    const int begin = tile * (8 * PW), end = min(begin + 8 * PW, a.n);
    const bool from_before = begin > 0 && a.keys[begin - 1] == first_key[0];
    float* part = a.partial + static_cast<int64_t>(tile) * 2 * a.D + c;
    int key = first_key[0];
    float sum = first_s[0][threadIdx.x];
    bool opening = true;    // the run began at the tile's first position
    auto flush = [&]() {
        if (opening && from_before) part[0] = sum;
        else {
            float* p = a.dtable + static_cast<int64_t>(key) * a.D + c;
            *p = (a.accumulate ? *p : 0.0f) + sum * a.scale;
        }
        opening = false;
    };
    for (int k = 0; k < 8; ++k) {
        if (first_key[k] < 0) break;
        if (k > 0) {
            if (first_key[k] == key) sum += first_s[k][threadIdx.x];
            else {
                flush();
                key = first_key[k], sum = first_s[k][threadIdx.x];
            }
        }
        if (last_key[k] >= 0) {
            flush();
            key = last_key[k], sum = last_s[k][threadIdx.x];
        }
    }
    const bool goes_on = end < a.n && a.keys[end] == key;
    if (goes_on && !(opening && from_before)) part[a.D] = sum;
    else flush();
}

// Runs that leave the tile they begin in: partial 1 of that tile, then partial 0 of the tiles that
// they cover.  A block takes 64 channels; its eight warps take every eighth tile, then add up in order.
__global__ void __launch_bounds__(256) tern_embed_join_kernel(const __grid_constant__ RunArgs a) {
    __shared__ float red[8][64];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int tile = blockIdx.x, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int begin = tile * a.run, end = min(begin + a.run, a.n);
    const int key = a.keys[end - 1], next = end < a.n ? a.keys[end] : -1;
    const int first = a.keys[begin], prev = begin > 0 ? a.keys[begin - 1] : -1;
    if (key >= a.V || next != key) return;           // ends with the tile
    if (first == key && prev == key) return;         // began before it
    // the tiles after this one whose first key is still `key`
    int more = 0;
    for (;;) {
        const int64_t at = static_cast<int64_t>(tile + 1 + more + lane) * a.run;
        const uint32_t same = __ballot_sync(0xffffffffu, at < a.n && a.keys[at < a.n ? at : 0] == key);
        more += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
        if (same != 0xffffffffu) break;
    }
    const float* part = a.partial + static_cast<int64_t>(tile + 1) * 2 * a.D;   // partial 0 of the next tile
    const int c0 = blockIdx.y * 64 + lane, c1 = c0 + 32;
    float x = 0.0f, y = 0.0f;
#pragma unroll 4
    for (int t = w; t < more; t += 8) {
        const float* p = part + static_cast<int64_t>(t) * 2 * a.D;
        if (c0 < a.D) x += p[c0];
        if (c1 < a.D) y += p[c1];
    }
    red[w][lane] = x, red[w][lane + 32] = y;
    __syncthreads();
    const int c = blockIdx.y * 64 + threadIdx.x;
    if (threadIdx.x >= 64 || c >= a.D) return;
    float sum = part[c - a.D];
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += red[k][threadIdx.x];
    float* p = a.dtable + static_cast<int64_t>(key) * a.D + c;
    *p = (a.accumulate ? *p : 0.0f) + sum * a.scale;
}

// ------------------------------------------------------------------------------ host side

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

struct Plan {   // the sort's passes and the workspace's parts, in bytes
    int passes = 0, bits = 0, sort_tiles = 0, run = 0, run_tiles = 0;
    int64_t keys[2], pos[2], counts, totals, partial, bytes = 0;
};

Plan make_plan(int64_t n, int64_t V, int64_t D) {
    Plan p;
    int need = 1;
    while ((static_cast<int64_t>(1) << need) <= V) ++need;   // keys 0..V
    p.passes = (need + kMaxBits - 1) / kMaxBits;
    p.bits = (need + p.passes - 1) / p.passes;
    p.sort_tiles = static_cast<int>((n + kSortTile - 1) / kSortTile);
    // 64 positions a block while 256 would leave SMs without one (8192 x 512: 20 to 15 us together with
    // the smaller tiles of the sort)
    p.run = (n + 255) / 256 * ((D + kChTile - 1) / kChTile) < 152 ? 64 : 256;
    p.run_tiles = static_cast<int>((n + p.run - 1) / p.run);
    auto take = [&](int64_t bytes) {
        const int64_t at = p.bytes;
        p.bytes += round256(bytes);
        return at;
    };
    for (int i = 0; i < 2; ++i) p.keys[i] = take(4 * n), p.pos[i] = take(4 * n);
    p.counts = take(4 * (static_cast<int64_t>(1) << p.bits) * p.sort_tiles);
    p.totals = take(4 * (static_cast<int64_t>(1) << p.bits));
    p.partial = take(8 * static_cast<int64_t>(p.run_tiles) * D);
    return p;
}

constexpr int64_t kClusterSort = 16 * 32 * 64;   // positions that one cluster sorts

template <int WARPS, int R>
int launch_sort(const ClusterSortArgs& c, int digits, cudaStream_t s) {
    const int64_t tile = WARPS * 32 * R;
    unsigned P = 1;
    while (P * tile < c.s.n) P *= 2;
    return launch_cluster(tern_embed_sort_kernel<WARPS, R>, P, WARPS * 32, digits * (8 + 2 * WARPS), P, true, s, c);
}

bool bad_sizes(int64_t n, int64_t V, int64_t D) {
    return n < 0 || V < 1 || D < 0 || n > INT32_MAX - kSortTile || V >= INT32_MAX || D > 65535 * 64;
}
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <class TOK, class TAB>
int launch_embed(const EmbedArgs& a, int num_sms, cudaStream_t s) {
    const bool wide = a.D % 8 == 0 && a.ld_out % 8 == 0 && aligned16(a.table) && aligned16(a.out);
    const int items = a.D / 8;
    int tx = wide ? 8 : 16;                       // threads per row
    while (tx < 256 && tx < items) tx *= 2;
    const int64_t blocks = (a.n + 256 / tx - 1) / (256 / tx);
    const bool many = wide && items <= 256 && blocks > 16ll * num_sms;
    void (*const kernel)(EmbedArgs, int) = many   ? tern_embed_fwd_kernel<TOK, TAB, true, true>
                                           : wide ? tern_embed_fwd_kernel<TOK, TAB, true, false>
                                                  : tern_embed_fwd_kernel<TOK, TAB, false, false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(many ? 16ll * num_sms : blocks)), dim3(256), 0, s, a, tx);
}

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" int tern_embed_fwd(const void* tokens, int tokens_dtype, const void* table, int table_dtype, int64_t n,
                              int64_t V, int64_t D, float scale, void* out, int64_t ld_out, void* stream) {
    if (bad_sizes(n, V, D) || ld_out < D) return TERN_ERR_ARG;
    if ((tokens_dtype != TERN_I32 && tokens_dtype != TERN_I64) || (table_dtype != TERN_BF16 && table_dtype != TERN_F32))
        return TERN_ERR_ARG;
    if (n == 0 || D == 0) return TERN_OK;
    if (!tokens || !table || !out) return TERN_ERR_ARG;
    if (!aligned(tokens, tokens_dtype == TERN_I64 ? 8 : 4) || !aligned(table, table_dtype == TERN_F32 ? 4 : 2) || !aligned(out, 2))
        return TERN_ERR_ALIGN;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    EmbedArgs a{tokens, table, static_cast<__nv_bfloat16*>(out), n, ld_out, static_cast<int>(V), static_cast<int>(D), scale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens_dtype == TERN_I64)
        return table_dtype == TERN_F32 ? launch_embed<long long, float>(a, num_sms, s) : launch_embed<long long, __nv_bfloat16>(a, num_sms, s);
    return table_dtype == TERN_F32 ? launch_embed<int, float>(a, num_sms, s) : launch_embed<int, __nv_bfloat16>(a, num_sms, s);
}

extern "C" size_t tern_embed_bwd_workspace(int64_t n, int64_t V, int64_t D) {
    return bad_sizes(n, V, D) ? 0 : static_cast<size_t>(make_plan(n, V, D).bytes);
}

extern "C" int tern_embed_bwd(const void* tokens, int tokens_dtype, const void* dout, int64_t ld_dout, int64_t n, int64_t V,
                              int64_t D, float scale, int accumulate, float* dtable, void* workspace, size_t ws_bytes,
                              void* stream) {
    if (bad_sizes(n, V, D) || ld_dout < D || (tokens_dtype != TERN_I32 && tokens_dtype != TERN_I64)) return TERN_ERR_ARG;
    if (D == 0 || (n == 0 && accumulate)) return TERN_OK;
    if (!dtable || (n > 0 && (!tokens || !dout))) return TERN_ERR_ARG;
    if (!aligned(tokens, tokens_dtype == TERN_I64 ? 8 : 4) || !aligned(dout, 2) || !aligned(dtable, 4)) return TERN_ERR_ALIGN;
    const Plan p = make_plan(n, V, D);
    if (!workspace || ws_bytes < static_cast<size_t>(p.bytes)) return TERN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TERN_ERR_ALIGN;
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto i32 = [&](int64_t at) { return reinterpret_cast<int32_t*>(ws + at); };

    SortArgs q{};
    q.n = static_cast<int>(n), q.V = static_cast<int>(V), q.tiles = p.sort_tiles, q.bits = p.bits;
    q.tokens64 = tokens_dtype == TERN_I64;
    q.counts = i32(p.counts), q.totals = i32(p.totals);
    if (n == 0) {   // nothing to sort: every row is without a token
        TERN_CUDA_TRY(cudaMemsetAsync(dtable, 0, static_cast<size_t>(V) * D * sizeof(float), s));
        return TERN_OK;
    }
    const int digits = 1 << p.bits;
    const bool wide = D % 8 == 0 && ld_dout % 8 == 0 && aligned16(dout) && aligned16(dtable);
    if (n <= kClusterSort) {
        ClusterSortArgs c{};
        c.s = q, c.passes = p.passes;
        c.s.tokens = tokens;
        for (int i = 0; i < 2; ++i) c.keys[i] = i32(p.keys[i]), c.pos[i] = i32(p.pos[i]);
        const int st = n <= 8192 ? launch_sort<8, 2>(c, digits, s) : launch_sort<32, 2>(c, digits, s);
        if (st != TERN_OK) return st;
        q.keys_out = c.keys[(p.passes - 1) & 1], q.pos_out = c.pos[(p.passes - 1) & 1];
    } else {
        for (int pass = 0; pass < p.passes; ++pass) {
            q.tokens = pass == 0 ? tokens : nullptr;
            q.keys_in = pass == 0 ? nullptr : i32(p.keys[(pass - 1) & 1]);
            q.pos_in = pass == 0 ? nullptr : i32(p.pos[(pass - 1) & 1]);
            q.keys_out = i32(p.keys[pass & 1]), q.pos_out = i32(p.pos[pass & 1]);
            q.shift = pass * p.bits;
            if (int st = launch_pdl(tern_embed_count_kernel, dim3(p.sort_tiles), dim3(256), 0, s, q)) return st;
            if (int st = launch_pdl(tern_embed_offsets_kernel, dim3((digits + 7) / 8), dim3(256), 0, s, q.counts, q.totals, digits, p.sort_tiles)) return st;
            if (int st = launch_pdl(tern_embed_place_kernel, dim3(p.sort_tiles), dim3(256), 0, s, q)) return st;
        }
    }
    RunArgs a{};
    a.keys = q.keys_out, a.pos = q.pos_out, a.dout = static_cast<const __nv_bfloat16*>(dout), a.dtable = dtable;
    a.partial = reinterpret_cast<float*>(ws + p.partial), a.ld_dout = ld_dout;
    a.n = q.n, a.V = q.V, a.D = static_cast<int>(D), a.run = p.run, a.run_tiles = p.run_tiles;
    a.dout_end = a.dout + (n - 1) * ld_dout + D;
    const int ch = wide ? tile_channels<true>() : tile_channels<false>();
    a.ch_tiles = static_cast<int>((D + ch - 1) / ch);
    a.accumulate = accumulate ? 1 : 0, a.scale = scale;
    const int64_t units = static_cast<int64_t>(a.run_tiles) * a.ch_tiles;
    const int64_t fill = accumulate ? 0 : (V + 7) / 8 < 8 * num_sms ? (V + 7) / 8 : 8 * num_sms;
    if (units + fill > INT32_MAX) return TERN_ERR_ARG;
    void (*const sum)(RunArgs) = p.run == 64 ? (wide ? tern_embed_sum_kernel<true, 8> : tern_embed_sum_kernel<false, 8>)
                                             : (wide ? tern_embed_sum_kernel<true, 32> : tern_embed_sum_kernel<false, 32>);
    if (int st = launch_pdl(sum, dim3(static_cast<unsigned>(units + fill)), dim3(256), 0, s, a)) return st;
    if (p.run_tiles < 2) return TERN_OK;
    const unsigned gy = static_cast<unsigned>((D + 63) / 64);
    return launch_pdl(tern_embed_join_kernel, dim3(static_cast<unsigned>(p.run_tiles), gy), dim3(256), 0, s, a);
}
