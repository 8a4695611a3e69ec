// What the kernels over rows of activations share: loads and stores of V neighbouring elements of
// bf16 or fp32 as fp32, and sums over warps and blocks in a fixed order.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace tern {
namespace {

template <class T>
constexpr int kElem = static_cast<int>(sizeof(T));

// Words of up to 16 bytes that hold V elements of T.
template <class T, int V>
struct Raw {
    static constexpr int BYTES = V * kElem<T>;
    static constexpr int WORDS = (BYTES + 3) / 4;
    uint32_t w[WORDS];
};

// V elements at p, which is aligned to min(16, V * sizeof(T)) bytes.
template <class T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
    Raw<T, V> r;
    constexpr int B = Raw<T, V>::BYTES;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) {
            const uint4 u = reinterpret_cast<const uint4*>(p)[i];
            r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
        }
    } else if constexpr (B == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        r.w[0] = u.x, r.w[1] = u.y;
    } else if constexpr (B == 4) {
        r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        r.w[0] = *reinterpret_cast<const unsigned short*>(p);
    }
    return r;
}

template <class T, int V>
__device__ __forceinline__ float raw_at(const Raw<T, V>& r, int i) {
    if constexpr (kElem<T> == 4) return __uint_as_float(r.w[i]);
    // a bf16 is the upper half of the fp32 with the same value
    return __uint_as_float((i & 1) ? r.w[i >> 1] & 0xFFFF0000u : r.w[i >> 1] << 16);
}

template <class T, int V>
__device__ __forceinline__ void set_raw(Raw<T, V>& r, const float (&v)[V]) {
    if constexpr (kElem<T> == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(v[i]);
    } else if constexpr (V == 1) {
        r.w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            r.w[i] = *reinterpret_cast<const uint32_t*>(&t);
        }
    }
}

template <class T, int V>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, V>& r) {
    constexpr int B = Raw<T, V>::BYTES;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
    } else if constexpr (B == 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    } else if constexpr (B == 4) {
        *reinterpret_cast<uint32_t*>(p) = r.w[0];
    } else {
        *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>(r.w[0]);
    }
}

// Rounded to nearest even (bf16) or as it is (fp32).
template <class T, int V>
__device__ __forceinline__ void store_as(T* p, const float (&v)[V]) {
    Raw<T, V> r;
    set_raw<T, V>(r, v);
    store_raw<T, V>(p, r);
}

// Sums of N values over the threads that share a row: T neighbours of a warp (T <= 32, all of the warp
// calling), or the whole block of T threads through `s` (N * T / 32 floats; the caller keeps it from being reused too early by
// alternating two of them).  Every thread gets the sums; the order is fixed.
template <int T, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* s) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int d = T < 32 ? T / 2 : 16; d >= 1; d >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    if constexpr (T > 32) {
        constexpr int W = T / 32;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) s[i * W + (threadIdx.x >> 5)] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) t += s[i * W + w];
            v[i] = t;
        }
    }
}

// Elements per access that every row of a matrix allows: V of them are `V * es` aligned bytes at the
// first row, from row to row and at the row's end.
inline bool rows_allow(const void* p, int64_t ld, int64_t n, int64_t D, int V, int es) {
    const int64_t b = V * es < 16 ? V * es : 16;
    return D % V == 0 && reinterpret_cast<uintptr_t>(p) % b == 0 && (n <= 1 || ld * es % b == 0);
}

}  // namespace
}  // namespace tern
