// What the tcgen05 GEMM kernels share: descriptors, the tile raster, the bounded wait, and the
// host's cached tensor maps.
#pragma once

#include "common.cuh"

namespace tern {

// Tensor map of a dense row-major matrix [outer][inner] read in boxes of box_outer x box_inner
// (gemm.cu; cached).
int tensor_map_2d(CUtensorMap* m, const void* ptr, CUtensorMapDataType type, int64_t inner, int64_t outer, int box_inner,
                  int box_outer, CUtensorMapSwizzle sw);

// Tensor map of [n2][n1][n0] elements with strides of s1 and s2 bytes, read in boxes of box1 x box0
// (gemm.cu; cached).
int tensor_map_3d(CUtensorMap* m, const void* ptr, CUtensorMapDataType type, int64_t n0, int64_t n1, int64_t n2, int64_t s1,
                  int64_t s2, int box0, int box1);

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s per wait; a healthy wait takes microseconds

enum { SW128 = 2, SW64 = 4 };   // tcgen05 descriptor layout codes

// tcgen05 instruction descriptor: fp32 D, M x N, operand majors and the A/B format code
// (kind::f16: 0 = f16, 1 = bf16; kind::f8f6f4: 0 = e4m3).
__host__ __device__ constexpr uint32_t make_idesc(int M, int N, bool a_mn, bool b_mn, uint32_t fmt = 1u) {
    return (1u << 4)                       // D format: f32
           | (fmt << 7)                    // A format
           | (fmt << 10)                   // B format
           | (static_cast<uint32_t>(a_mn) << 15)
           | (static_cast<uint32_t>(b_mn) << 16)
           | (static_cast<uint32_t>(N >> 3) << 17)
           | (static_cast<uint32_t>(M >> 4) << 24);
}

// tcgen05 shared-memory matrix descriptor.
__device__ __forceinline__ uint64_t make_sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) |
           (static_cast<uint64_t>(layout) << 61);
}

// Descriptor of the kk-th 16-deep k-slice of an operand tile at `base`.
//  K-major, BK = 64: rows of 128 B (SW128), 8-row atoms 1024 B apart; the slice
//                    starts 32 B further along the row.
//  K-major, BK = 32: rows of 64 B (SW64), 8-row atoms 512 B apart.
//  MN-major (BK 64): 64-element MN chunks of BK k-rows (128 B each, SW128);
//                    chunks LBO = 64*BK*2 B apart, 8-k-row groups SBO = 1024 B
//                    apart; the slice starts two groups (2048 B) further.
template <bool MN, int BK>
__device__ __forceinline__ uint64_t op_desc(uint32_t base, int kk) {
    if constexpr (MN) {
        return make_sdesc(base + kk * 2048u, 64u * BK * 2u, 1024u, SW128);
    } else if constexpr (BK == 64) {
        return make_sdesc(base + kk * 32u, 16u, 1024u, SW128);
    } else {
        return make_sdesc(base + kk * 32u, 16u, 512u, SW64);
    }
}

// Grouped raster: runs of GM m-tiles share an n-tile, so neighbouring CTAs reuse
// the same B panel and A panels stay resident in L2.
template <int GM>
__host__ __device__ __forceinline__ void tile_coords(int tile, int tiles_m, int tiles_n, int& mt, int& nt) {
    const int group = tile / (GM * tiles_n);
    const int first_m = group * GM;
    const int gm = min(GM, tiles_m - first_m);
    const int local = tile - group * GM * tiles_n;
    mt = first_m + local % gm;
    nt = local / gm;
}

// Bounded wait on an mbarrier phase.  Returns false when the limit is reached (after raising the
// abort flag and calling on_expiry) or, when `watch_abort`, once another role has raised it.
template <class F>
__device__ __forceinline__ bool wait_limited(uint32_t bar, uint32_t parity, volatile int* abort_flag, bool watch_abort,
                                             uint64_t limit_ns, F on_expiry) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    // The time waited is the sum of the timer's forward steps between polls, each
    // counted up to 1 ms: a timer that steps backwards, or jumps forward once, cannot
    // end a healthy wait.  A poll count backs the bound should the timer stall.
    uint64_t last = ptx::globaltimer(), waited = 0;
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (watch_abort && *abort_flag) return false;
            const uint64_t now = ptx::globaltimer();
            const int64_t step = static_cast<int64_t>(now - last);
            last = now;
            if (step > 0) waited += static_cast<uint64_t>(step < 1000000 ? step : 1000000);
            if (waited > limit_ns || it >= (1u << 30)) {
                *abort_flag = 1;
                on_expiry();
                return false;
            }
        }
    }
}

}  // namespace
}  // namespace tern
