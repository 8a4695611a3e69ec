// Layer norm over rows of D channels and its gradient.
//
//   mean = sum x / D, var = sum (x - mean)^2 / D, rstd = 1 / sqrt(var + eps)
//   xhat = (x - mean) rstd,  y = xhat weight + bias
//   g = dy weight
//   dx = rstd (g - sum g / D - xhat sum (g xhat) / D)
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy
//
// What bounds it is memory: a row is read once into registers, and everything that needs the whole
// row (two passes of sums in the forward, three sums at once in the gradient) works there.  A row
// belongs to a warp or to a block, whichever holds it at EPT elements a thread; rows wider than a
// block of 1024 threads holds are read again for each pass (from L2 as a rule).
//
// The mean of a row far from zero rounds by up to half a unit of its own size, which may be large
// beside the row's spread.  So what the rounded mean leaves, delta = sum (x - mean) / D, is summed in
// the pass that needs x - mean anyway and taken out of xhat: in the forward, and again in the
// gradient, where sum g xhat = rstd (sum g d - delta sum g) with d = x - mean.
//
// The gradient's blocks stay for many rows and keep the sums of their columns in registers; each
// block stores its sums once, and a second launch adds the blocks' in a fixed order.
#include <algorithm>
#include <cmath>

#include "rows.cuh"

namespace tern {
namespace {

constexpr int kPartMax = 608;   // blocks of the gradient: four for each of 152 SMs

struct NormArgs {
    const void* x;
    const void* dy;
    void* y;          // the forward's y, the gradient's dx
    const float* weight;
    const float* bias;
    float* mean;
    float* rstd;
    float* part;      // [2][blocks][D] sums of the columns, or null
    int64_t ld_x, ld_dy, ld_y;
    int n, D;
    float eps, inv_d;
};

// EPT elements of a row in registers: thread t holds V neighbouring elements at (j T + t) V.
// T threads a row, R rows a block side by side (R > 1 with T = 32 only).
template <class TX, class TY, int T, int R, int EPT, int V>
__global__ void __launch_bounds__(T * R, 1) norm_fwd(const __grid_constant__ NormArgs a) {
    constexpr int NV = EPT / V;
    __shared__ float sums[2][2 * (T / 32)];
    ptx::pdl_trigger();
    const int t = threadIdx.x % T;
    const int row = static_cast<int>(blockIdx.x) * R + static_cast<int>(threadIdx.x) / T;
    ptx::pdl_wait();
    if (row >= a.n) return;   // whole warps, and with T > 32 whole blocks
    const TX* x = static_cast<const TX*>(a.x) + row * a.ld_x;
    Raw<TX, V> raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * T + t) * V;
        if (c < a.D) {
            raw[j] = load_raw<TX, V>(x + c);
        } else {
#pragma unroll
            for (int i = 0; i < Raw<TX, V>::WORDS; ++i) raw[j].w[i] = 0u;
        }
    }
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += raw_at<TX, V>(raw[j], i);
    row_sums<T, 1>(s, sums[0]);
    const float mean = s[0] * a.inv_d;
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if ((j * T + t) * V < a.D) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = raw_at<TX, V>(raw[j], i) - mean;
                q[0] += d;
                q[1] = fmaf(d, d, q[1]);
            }
        }
    }
    row_sums<T, 2>(q, sums[1]);
    const float delta = q[0] * a.inv_d;
    const float rstd = 1.0f / sqrtf(fmaxf(fmaf(-delta, delta, q[1] * a.inv_d), 0.f) + a.eps);
    // fmaxf drops a NaN: the row's own comes back through x - mean
    if (t == 0) {
        if (a.mean) a.mean[row] = mean + delta;
        if (a.rstd) a.rstd[row] = q[1] == q[1] ? rstd : q[1];
    }
    TY* y = static_cast<TY*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * T + t) * V;
        if (c < a.D) {
            float v[V];
            Raw<float, V> w, b;
            if (a.weight) w = load_raw<float, V>(a.weight + c);
            if (a.bias) b = load_raw<float, V>(a.bias + c);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = (raw_at<TX, V>(raw[j], i) - mean - delta) * rstd;
                if (a.weight) v[i] *= raw_at<float, V>(w, i);
                if (a.bias) v[i] += raw_at<float, V>(b, i);
            }
            store_as<TY, V>(y + c, v);
        }
    }
}

// Rows of any width: three passes over the row by a block.
template <class TX, class TY>
__global__ void __launch_bounds__(1024) norm_fwd_wide(const __grid_constant__ NormArgs a) {
    __shared__ float sums[2][64];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int64_t row = blockIdx.x;
    const TX* x = static_cast<const TX*>(a.x) + row * a.ld_x;
    TY* y = static_cast<TY*>(a.y) + row * a.ld_y;
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < a.D; c += 1024) s[0] += raw_at<TX, 1>(load_raw<TX, 1>(x + c), 0);
    row_sums<1024, 1>(s, sums[0]);
    const float mean = s[0] * a.inv_d;
    float q[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float d = raw_at<TX, 1>(load_raw<TX, 1>(x + c), 0) - mean;
        q[0] += d;
        q[1] = fmaf(d, d, q[1]);
    }
    row_sums<1024, 2>(q, sums[1]);
    const float delta = q[0] * a.inv_d;
    const float rstd = 1.0f / sqrtf(fmaxf(fmaf(-delta, delta, q[1] * a.inv_d), 0.f) + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean + delta;
        if (a.rstd) a.rstd[row] = q[1] == q[1] ? rstd : q[1];
    }
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        float v[1] = {(raw_at<TX, 1>(load_raw<TX, 1>(x + c), 0) - mean - delta) * rstd};
        if (a.weight) v[0] *= __ldg(a.weight + c);
        if (a.bias) v[0] += __ldg(a.bias + c);
        store_as<TY, 1>(y + c, v);
    }
}

// The gradient's blocks take rows blockIdx.x R + r, then gridDim.x R further, and so on.
template <class TX, class TY, int T, int R, int EPT, int V>
__global__ void __launch_bounds__(T * R, 1) norm_bwd(const __grid_constant__ NormArgs a) {
    constexpr int NV = EPT / V;
    __shared__ float sums[2][3 * (T / 32)];
    ptx::pdl_trigger();
    const int t = threadIdx.x % T, r = static_cast<int>(threadIdx.x) / T;
    const int step = static_cast<int>(gridDim.x) * R;
    float w[EPT], dw[EPT], db[EPT];
    ptx::pdl_wait();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * T + t) * V;
        Raw<float, V> raw;
        if (a.weight && c < a.D) raw = load_raw<float, V>(a.weight + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[j * V + i] = a.weight && c < a.D ? raw_at<float, V>(raw, i) : 1.0f;
            dw[j * V + i] = db[j * V + i] = 0.f;
        }
    }
    Raw<TX, V> rx[NV], nx[NV];
    Raw<TY, V> rd[NV], nd[NV];
    float mean = 0.f, rstd = 0.f, nmean = 0.f, nrstd = 0.f;
    auto fetch = [&](int64_t row, Raw<TX, V>(&fx)[NV], Raw<TY, V>(&fd)[NV], float& m, float& s) {
        const TX* x = static_cast<const TX*>(a.x) + row * a.ld_x;
        const TY* dy = static_cast<const TY*>(a.dy) + row * a.ld_dy;
        m = __ldg(a.mean + row);
        s = __ldg(a.rstd + row);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * T + t) * V;
            if (c < a.D) {
                fx[j] = load_raw<TX, V>(x + c);
                fd[j] = load_raw<TY, V>(dy + c);
            }
        }
    };
    int64_t row = static_cast<int64_t>(blockIdx.x) * R + r;
    if (row < a.n) fetch(row, rx, rd, mean, rstd);
    for (int flip = 0; row < a.n; row += step, flip ^= 1) {
        if (row + step < a.n) fetch(row + step, nx, nd, nmean, nrstd);   // in flight while this row is summed
        float s[3] = {0.f, 0.f, 0.f};   // sums of g, g d, d
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if ((j * T + t) * V < a.D) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = raw_at<TX, V>(rx[j], i) - mean;
                    const float g = raw_at<TY, V>(rd[j], i) * w[j * V + i];
                    s[0] += g;
                    s[1] = fmaf(g, d, s[1]);
                    s[2] += d;
                }
            }
        }
        row_sums<T, 3>(s, sums[flip]);
        const float delta = s[2] * a.inv_d;
        const float along = rstd * rstd * fmaf(-delta, s[0], s[1]) * a.inv_d;   // rstd sum (g xhat) / D
        const float base = s[0] * a.inv_d;
        TX* dx = static_cast<TX*>(a.y) + row * a.ld_y;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * T + t) * V;
            if (c < a.D) {
                float v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = j * V + i;
                    const float d = raw_at<TX, V>(rx[j], i) - mean - delta;
                    const float dy = raw_at<TY, V>(rd[j], i);
                    v[i] = rstd * (fmaf(dy, w[e], -base) - d * along);
                    dw[e] = fmaf(dy, d * rstd, dw[e]);
                    db[e] += dy;
                }
                store_as<TX, V>(dx + c, v);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) rx[j] = nx[j], rd[j] = nd[j];
        mean = nmean, rstd = nrstd;
    }
    if (!a.part) return;
    if constexpr (R > 1) {   // the block's rows side by side: added in order, one row of warps at a time
        extern __shared__ float cols[];   // [2][EPT * 32]
        for (int k = 0; k < R; ++k) {
            if (r == k) {
#pragma unroll
                for (int e = 0; e < EPT; ++e) {
                    const int at = e * T + t;
                    if (k > 0) dw[e] += cols[at], db[e] += cols[EPT * T + at];
                    cols[at] = dw[e], cols[EPT * T + at] = db[e];
                }
            }
            __syncthreads();
        }
        if (r != R - 1) return;
    }
    float* pw = a.part + static_cast<int64_t>(blockIdx.x) * a.D;
    float* pb = pw + static_cast<int64_t>(gridDim.x) * a.D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * T + t) * V;
        if (c < a.D) {
            float v[V], u[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = dw[j * V + i], u[i] = db[j * V + i];
            if constexpr (V >= 4) {   // D % V == 0 and the workspace is 16-byte aligned
                store_as<float, V>(pw + c, v);
                store_as<float, V>(pb + c, u);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) pw[c + i] = v[i], pb[c + i] = u[i];
            }
        }
    }
}

// dx of rows of any width: two passes over the row by a block.
template <class TX, class TY>
__global__ void __launch_bounds__(1024) norm_bwd_wide(const __grid_constant__ NormArgs a) {
    __shared__ float sums[96];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int64_t row = blockIdx.x;
    const TX* x = static_cast<const TX*>(a.x) + row * a.ld_x;
    const TY* dy = static_cast<const TY*>(a.dy) + row * a.ld_dy;
    TX* dx = static_cast<TX*>(a.y) + row * a.ld_y;
    const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    float s[3] = {0.f, 0.f, 0.f};
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float d = raw_at<TX, 1>(load_raw<TX, 1>(x + c), 0) - mean;
        const float g = raw_at<TY, 1>(load_raw<TY, 1>(dy + c), 0) * (a.weight ? __ldg(a.weight + c) : 1.0f);
        s[0] += g;
        s[1] = fmaf(g, d, s[1]);
        s[2] += d;
    }
    row_sums<1024, 3>(s, sums);
    const float delta = s[2] * a.inv_d;
    const float along = rstd * rstd * fmaf(-delta, s[0], s[1]) * a.inv_d;
    const float base = s[0] * a.inv_d;
    if (a.part && threadIdx.x == 0) a.part[row] = delta;   // for the columns' sums
    for (int c = threadIdx.x; c < a.D; c += 1024) {
        const float d = raw_at<TX, 1>(load_raw<TX, 1>(x + c), 0) - mean - delta;
        const float g = raw_at<TY, 1>(load_raw<TY, 1>(dy + c), 0) * (a.weight ? __ldg(a.weight + c) : 1.0f);
        float v[1] = {rstd * (g - base - d * along)};
        store_as<TX, 1>(dx + c, v);
    }
}

// The columns' sums of such rows: a thread adds one column over all rows, in order.  (Rows of more
// than 16384 channels are few, and the columns many.)
template <class TX, class TY>
__global__ void __launch_bounds__(256) norm_cols_wide(const __grid_constant__ NormArgs a, float* dweight, float* dbias) {
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int c = static_cast<int>(blockIdx.x) * 256 + static_cast<int>(threadIdx.x);
    if (c >= a.D) return;
    float w = 0.f, b = 0.f;
#pragma unroll 4
    for (int64_t row = 0; row < a.n; ++row) {
        const float d = raw_at<TX, 1>(load_raw<TX, 1>(static_cast<const TX*>(a.x) + row * a.ld_x + c), 0) - __ldg(a.mean + row) - a.part[row];
        const float dy = raw_at<TY, 1>(load_raw<TY, 1>(static_cast<const TY*>(a.dy) + row * a.ld_dy + c), 0);
        w = fmaf(dy, d * __ldg(a.rstd + row), w);
        b += dy;
    }
    if (dweight) dweight[c] = w;
    if (dbias) dbias[c] = b;
}

// Sums of the blocks' columns: a block takes 32 columns, warp w adds the parts w, w + 16, ... and the
// warps' sums are added in order.  grid.y = 2: the weight's, the bias's.
__global__ void __launch_bounds__(512) norm_cols(const float* __restrict__ part, int parts, int D, float* dweight, float* dbias) {
    __shared__ float s[16][33];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    float* out = blockIdx.y == 0 ? dweight : dbias;
    if (!out) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = static_cast<int>(blockIdx.x) * 32 + lane;
    float v = 0.f;
    if (c < D) {
        const float* p = part + static_cast<int64_t>(blockIdx.y) * parts * D + c;
#pragma unroll 8
        for (int k = warp; k < parts; k += 16) v += __ldcg(p + static_cast<int64_t>(k) * D);
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < D) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) t += s[w][lane];
        out[c] = t;
    }
}

constexpr int kFwdEpt = 16, kBwdEpt = 16;
constexpr int kWidest = 16384;   // channels that a block of 1024 threads holds

// Threads a row takes at 16 elements each: a warp, or a block of 128 to 1024.
int row_threads(int64_t D) {
    int t = 32;
    while (static_cast<int64_t>(t) * 16 < D) t = t == 32 ? 128 : 2 * t;
    return t;
}

constexpr int kWarpRows = 4;   // rows a block side by side, of a warp each

int bwd_parts(int64_t n, int64_t D) {
    if (D > kWidest) return 0;
    const int R = row_threads(D) == 32 ? kWarpRows : 1;
    return static_cast<int>(std::min<int64_t>(kPartMax, (n + R - 1) / R));
}

template <bool BWD, class TX, class TY, int T, int R, int V>
int launch_rows(const NormArgs& a, int grid, cudaStream_t s) {
    if constexpr (BWD)
        return launch_pdl(norm_bwd<TX, TY, T, R, kBwdEpt, V>, dim3(grid), dim3(T * R), R > 1 ? 2 * kBwdEpt * 32 * sizeof(float) : 0, s, a);
    else
        return launch_pdl(norm_fwd<TX, TY, T, R, kFwdEpt, V>, dim3(grid), dim3(T * R), 0, s, a);
}

template <bool BWD, class TX, class TY, int V>
int pick_rows(const NormArgs& a, cudaStream_t s) {
    const int T = row_threads(a.D);
    const int R = T == 32 ? kWarpRows : 1;
    const int grid = BWD ? bwd_parts(a.n, a.D) : (a.n + R - 1) / R;
    switch (T) {
    case 32: return launch_rows<BWD, TX, TY, 32, kWarpRows, V>(a, grid, s);
    case 128: return launch_rows<BWD, TX, TY, 128, 1, V>(a, grid, s);
    case 256: return launch_rows<BWD, TX, TY, 256, 1, V>(a, grid, s);
    case 512: return launch_rows<BWD, TX, TY, 512, 1, V>(a, grid, s);
    default: return launch_rows<BWD, TX, TY, 1024, 1, V>(a, grid, s);
    }
}

bool all_allow(const NormArgs& a, bool bwd, int V, int ex, int ey) {
    const uintptr_t b = static_cast<uintptr_t>(V * 4 < 16 ? V * 4 : 16) - 1;
    auto params = [&](const float* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & b) == 0; };
    return rows_allow(a.x, a.ld_x, a.n, a.D, V, ex) && rows_allow(a.y, a.ld_y, a.n, a.D, V, bwd ? ex : ey) &&
           (!bwd || rows_allow(a.dy, a.ld_dy, a.n, a.D, V, ey)) && params(a.weight) && params(a.bias);
}

template <bool BWD, class TX, class TY>
int run_norm(const NormArgs& a, float* dweight, float* dbias, cudaStream_t s) {
    if (a.D > kWidest) {
        if constexpr (BWD) {
            if (a.n > 0)
                if (int st = launch_pdl(norm_bwd_wide<TX, TY>, dim3(a.n), dim3(1024), 0, s, a)) return st;
            if (dweight || dbias) return launch_pdl(norm_cols_wide<TX, TY>, dim3((a.D + 255) / 256), dim3(256), 0, s, a, dweight, dbias);
            return TERN_OK;
        } else {
            return launch_pdl(norm_fwd_wide<TX, TY>, dim3(a.n), dim3(1024), 0, s, a);
        }
    }
    if (a.n > 0) {
        constexpr int ex = kElem<TX>, ey = kElem<TY>;
        int st;
        if (all_allow(a, BWD, 8, ex, ey)) st = pick_rows<BWD, TX, TY, 8>(a, s);
        else if (all_allow(a, BWD, 2, ex, ey)) st = pick_rows<BWD, TX, TY, 2>(a, s);
        else st = pick_rows<BWD, TX, TY, 1>(a, s);
        if (st) return st;
    }
    if (BWD && (dweight || dbias))   // of no rows: zeros
        return launch_pdl(norm_cols, dim3((a.D + 31) / 32, 2), dim3(512), 0, s, static_cast<const float*>(a.part), bwd_parts(a.n, a.D), a.D,
                          dweight, dbias);
    return TERN_OK;
}

template <bool BWD>
int run_types(const NormArgs& a, int tx, int ty, float* dweight, float* dbias, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (tx == TERN_BF16)
        return ty == TERN_BF16 ? run_norm<BWD, B, B>(a, dweight, dbias, s) : run_norm<BWD, B, float>(a, dweight, dbias, s);
    return ty == TERN_BF16 ? run_norm<BWD, float, B>(a, dweight, dbias, s) : run_norm<BWD, float, float>(a, dweight, dbias, s);
}

bool sizes_ok(int64_t n, int64_t D) { return n >= 0 && D >= 0 && n < (1ll << 31) - 2048 && D <= (1ll << 22); }
bool float_type(int t) { return t == TERN_BF16 || t == TERN_F32; }
int elem(int t) { return t == TERN_BF16 ? 2 : 4; }
bool ld_ok(int64_t ld, int64_t D) { return ld >= D && ld < (1ll << 40); }
bool aligned_to(const void* p, int b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" int tern_norm_fwd(const void* x, int x_dtype, int64_t ld_x, const float* weight, const float* bias, int64_t n,
                             int64_t D, float eps, void* y, int y_dtype, int64_t ld_y, float* mean, float* rstd, void* stream) {
    if (!sizes_ok(n, D) || !float_type(x_dtype) || !float_type(y_dtype) || !ld_ok(ld_x, D) || !ld_ok(ld_y, D)) return TERN_ERR_ARG;
    if (!(eps > 0.f) || std::isinf(eps)) return TERN_ERR_ARG;
    if (n == 0 || D == 0) return TERN_OK;
    if (!x || !y) return TERN_ERR_ARG;
    if (!aligned_to(x, elem(x_dtype)) || !aligned_to(y, elem(y_dtype)) || !aligned_to(weight, 4) || !aligned_to(bias, 4) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return TERN_ERR_ALIGN;
    if (int st = check_device(nullptr)) return st;
    NormArgs a{};
    a.x = x, a.y = y, a.weight = weight, a.bias = bias, a.mean = mean, a.rstd = rstd;
    a.ld_x = ld_x, a.ld_y = ld_y, a.n = static_cast<int>(n), a.D = static_cast<int>(D), a.eps = eps;
    a.inv_d = static_cast<float>(1.0 / static_cast<double>(D));
    return run_types<false>(a, x_dtype, y_dtype, nullptr, nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" size_t tern_norm_bwd_workspace(int64_t n, int64_t D) {
    if (!sizes_ok(n, D)) return 0;
    // the blocks' column sums, or, for rows wider than a block holds, one value a row
    const int64_t floats = D > kWidest ? n : 2 * static_cast<int64_t>(bwd_parts(n, D)) * D;
    return static_cast<size_t>(floats) * sizeof(float);
}

extern "C" int tern_norm_bwd(const void* x, int x_dtype, int64_t ld_x, const float* weight, const float* mean, const float* rstd,
                             const void* dy, int y_dtype, int64_t ld_dy, int64_t n, int64_t D, void* dx, int64_t ld_dx,
                             float* dweight, float* dbias, void* workspace, size_t ws_bytes, void* stream) {
    if (!sizes_ok(n, D) || !float_type(x_dtype) || !float_type(y_dtype) || !ld_ok(ld_x, D) || !ld_ok(ld_dy, D) || !ld_ok(ld_dx, D))
        return TERN_ERR_ARG;
    if (D == 0) return TERN_OK;
    if (n > 0 && (!x || !dy || !dx || !mean || !rstd)) return TERN_ERR_ARG;
    const bool sums = dweight || dbias;
    if (sums && n > 0 && (!workspace || ws_bytes < tern_norm_bwd_workspace(n, D))) return TERN_ERR_WORKSPACE;
    if (!aligned_to(x, elem(x_dtype)) || !aligned_to(dx, elem(x_dtype)) || !aligned_to(dy, elem(y_dtype)) || !aligned_to(weight, 4) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4) || (sums && !aligned16(workspace)))
        return TERN_ERR_ALIGN;
    if (int st = check_device(nullptr)) return st;
    NormArgs a{};
    a.x = x, a.dy = dy, a.y = dx, a.weight = weight, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.ld_x = ld_x, a.ld_dy = ld_dy, a.ld_y = ld_dx, a.n = static_cast<int>(n), a.D = static_cast<int>(D);
    a.inv_d = static_cast<float>(1.0 / static_cast<double>(D));
    return run_types<true>(a, x_dtype, y_dtype, dweight, dbias, static_cast<cudaStream_t>(stream));
}
