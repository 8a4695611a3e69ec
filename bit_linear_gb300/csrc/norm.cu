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
// belongs to part of a warp, a warp or a block, whichever holds it at 16 or 32 elements a thread; rows of more
// than 16384 channels are read again for each pass (from L2 as a rule).
//
// The mean of a row far from zero rounds by up to half a unit of its own size, which may be large
// beside the row's spread.  So what the rounded mean leaves, delta = sum (x - mean) / D, is summed in
// the pass that needs x - mean anyway and taken out of xhat: in the forward, and again in the
// gradient, where sum g xhat = rstd (sum g d - delta sum g) with d = x - mean.
//
// The mean that is kept has delta in it only where delta is more than its own rounding (2^-20 of the
// deviation): around zero the first sum is the better one, of bf16 often exact.
//
// The gradient's blocks stay for many rows and keep the sums of their columns in registers; each
// block stores its sums once, and a second launch adds the blocks' in a fixed order.  Rows of more than 16384
// channels have a kernel of their own for the columns' sums, by parts of the rows.
//
// 32768 x 4096 in bf16: forward 99 us, 0.80 of the measured copy rate, gradient 137 us, 0.87; 65536 x 1024 46 and
// 65 us (0.86, 0.91); from fp32 to bf16 117 and 237 us (1.01, 0.83), in fp32 alone 245 (0.97) for the gradient.
// Row by row, each block waiting for its one row: 124 and 308 in bf16, 124 and 367 from fp32.  The forward in
// bf16 uses two thirds of the issue slots: three passes over a row's words; with them in registers the
// barriers stand alone.  8192 x 512 from fp32: 4.6 and 13.3 us, of which two launches in turn and two rounds of
// rows; floors 3.7 and 6.2.  Odd widths go element by element: 32768 x 4095 in bf16 136 and 266 us (runs of
// aligned words, of which a row's first and last are in part others', took as long or longer).  More than 8192
// channels: the gradient with 1024 threads has 64 registers a thread and spills 268 to 576 bytes (16384 x 12288 from
// fp32 873 us, floor 297; 8192 x 16384 in bf16 376, 119); more than 16384, rows read three times in the
// forward and x and dy three times in the gradient: 8192 x 16385 in bf16 228 and 556 us (floors 79, 119), 8192 x 20000
// 298 and 670 (97, 145).
#include <algorithm>
#include <cmath>

#include "pairs.cuh"
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

__device__ __forceinline__ float kept_mean(float mean, float delta, float rstd) {
    return fabsf(delta) * rstd > 9.5367432e-7f ? mean + delta : mean;
}

// EPT elements of a row in registers: thread t holds V neighbouring elements at (j T + t) V.
// T threads a row, R rows a block side by side (R > 1 with T <= 32 only).
template <class TX, class TY, int T, int R, int EPT, int V>
__global__ void __launch_bounds__(T * R, EPT > 16 ? 1024 / (T * R) : 1) norm_fwd(const __grid_constant__ NormArgs a) {
    constexpr int NV = EPT / V;
    __shared__ float sums[2][2 * ((T + 31) / 32)];
    ptx::pdl_trigger();
    const int t = threadIdx.x % T;
    const int64_t mine = static_cast<int64_t>(blockIdx.x) * R + static_cast<int>(threadIdx.x) / T;
    ptx::pdl_wait();
    const bool in = mine < a.n;   // a last block's other rows do the last one again, unwritten
    const int64_t row = in ? mine : a.n - 1;
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
    if (!in) return;
    if (t == 0) {
        if (a.mean) a.mean[row] = kept_mean(mean, delta, rstd);
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

// The same for many rows off 16-byte words: blocks stay, with weight and bias in registers (element by
// element they take as many loads as the rows) and the next row under way.
constexpr int loop_blocks(int threads) { return threads >= 512 ? 1 : 640 / threads; }   // of an SM

template <class TX, class TY, int T, int R, int EPT, int V>
__global__ void __launch_bounds__(T * R, loop_blocks(T * R)) norm_fwd_loop(const __grid_constant__ NormArgs a) {
    constexpr int NV = EPT / V;
    __shared__ float sums[2][2 * ((T + 31) / 32)];
    ptx::pdl_trigger();
    const int t = threadIdx.x % T;
    const int64_t step = static_cast<int64_t>(gridDim.x) * R;
    int64_t row = static_cast<int64_t>(blockIdx.x) * R + static_cast<int>(threadIdx.x) / T;
    Raw<TX, V> raw[NV], next[NV];
    auto fetch = [&](int64_t of, Raw<TX, V>(&to)[NV]) {
        const TX* x = static_cast<const TX*>(a.x) + of * a.ld_x;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * T + t) * V;
            if (c < a.D) to[j] = load_raw<TX, V>(x + c);
        }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < Raw<TX, V>::WORDS; ++i) raw[j].w[i] = next[j].w[i] = 0u;   // behind the row: always
    ptx::pdl_wait();
    if (row < a.n) fetch(row, raw);
    float w[EPT], b[EPT];
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
        const int c = (e / V * T + t) * V + e % V;
        w[e] = a.weight && c < a.D ? __ldg(a.weight + c) : 1.f;
        b[e] = a.bias && c < a.D ? __ldg(a.bias + c) : 0.f;
    }
    for (; row < a.n; row += step) {
        if (row + step < a.n) fetch(row + step, next);
        float s[1] = {0.f};
#pragma unroll
        for (int e = 0; e < EPT; ++e) s[0] += raw_at<TX, V>(raw[e / V], e % V);
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
        if (t == 0) {
            if (a.mean) a.mean[row] = kept_mean(mean, delta, rstd);
            if (a.rstd) a.rstd[row] = q[1] == q[1] ? rstd : q[1];   // fmaxf drops a NaN
        }
        TY* y = static_cast<TY*>(a.y) + row * a.ld_y;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * T + t) * V;
            if (c < a.D) {
                float v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = fmaf((raw_at<TX, V>(raw[j], i) - mean - delta) * rstd, w[j * V + i], b[j * V + i]);
                store_as<TY, V>(y + c, v);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) raw[j] = next[j];
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
        if (a.mean) a.mean[row] = kept_mean(mean, delta, rstd);
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

// The columns' sums of such rows: a thread adds one column over a part of the rows, in order and in runs of
// kWideRun, so that what a sum rounds away does not grow with the rows (one thread over all of them: off by
// up to half a step of the sum for each row, and 4.5 ms of the 4.8 of 8192 x 16385 in bf16, for 0.28 of 0.56).
// Parts of no rows are zeros.
constexpr int kWideRun = 128;

// Parts of the rows: one up to kWideRun rows, which writes the sums itself; else for norm_cols.
int wide_parts(int64_t n) { return static_cast<int>(std::min<int64_t>(kPartMax, std::max<int64_t>(1, (n + kWideRun - 1) / kWideRun))); }

template <class TX, class TY>
__global__ void __launch_bounds__(256) norm_cols_wide(const __grid_constant__ NormArgs a, float* dweight, float* dbias) {
    ptx::pdl_trigger();
    ptx::pdl_wait();
    const int c = static_cast<int>(blockIdx.x) * 256 + static_cast<int>(threadIdx.x);
    if (c >= a.D) return;
    const int parts = static_cast<int>(gridDim.y), part = static_cast<int>(blockIdx.y);
    const int64_t rows = (static_cast<int64_t>(a.n) + parts - 1) / parts;
    const int64_t last = min(static_cast<int64_t>(a.n), (part + 1) * rows);
    float w = 0.f, b = 0.f;
    for (int64_t first = part * rows; first < last; first += kWideRun) {
        const int64_t end = min(last, first + kWideRun);
        float rw = 0.f, rb = 0.f;
#pragma unroll 8
        for (int64_t row = first; row < end; ++row) {
            const float d = raw_at<TX, 1>(load_raw<TX, 1>(static_cast<const TX*>(a.x) + row * a.ld_x + c), 0) - __ldg(a.mean + row) - a.part[row];
            const float dy = raw_at<TY, 1>(load_raw<TY, 1>(static_cast<const TY*>(a.dy) + row * a.ld_dy + c), 0);
            rw = fmaf(dy, d * __ldg(a.rstd + row), rw);
            rb += dy;
        }
        w += rw;
        b += rb;
    }
    if (parts > 1) {   // behind the rows' deltas
        float* to = a.part + a.n + static_cast<int64_t>(part) * a.D + c;
        to[0] = w;
        to[static_cast<int64_t>(parts) * a.D] = b;
        return;
    }
    if (dweight) dweight[c] = w;
    if (dbias) dbias[c] = b;
}

// Sums of the blocks' columns: a block takes C columns, a warp's lanes 32 / C parts of each, further
// parts in turn (ten asked for at once); lanes and warps are added in a fixed order.  grid.y = 2: the weight's,
// the bias's.  Eight columns a block where that makes too few blocks otherwise.
template <int C>
__global__ void __launch_bounds__(1024) norm_cols(const float* __restrict__ part, int parts, int D, float* dweight, float* dbias) {
    constexpr int BESIDE = 32 / C, STEP = 32 * BESIDE, EACH = 10;
    __shared__ float s[32][C + 1];
    ptx::pdl_trigger();
    ptx::pdl_wait();
    float* out = blockIdx.y == 0 ? dweight : dbias;
    if (!out) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = static_cast<int>(blockIdx.x) * C + lane % C, first = warp * BESIDE + lane / C;
    const float* p = part + (static_cast<int64_t>(blockIdx.y) * parts + first) * D + c;
    float t = 0.f;
    for (int k0 = 0; k0 * STEP < parts; k0 += EACH) {
        float v[EACH];
#pragma unroll
        for (int k = 0; k < EACH; ++k) v[k] = c < D && first + (k0 + k) * STEP < parts ? __ldcg(p + static_cast<int64_t>((k0 + k) * STEP) * D) : 0.f;
#pragma unroll
        for (int k = 0; k < EACH; ++k) t += v[k];
    }
#pragma unroll
    for (int d = 16; d >= C; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    if (lane < C) s[warp][lane] = t;
    __syncthreads();
    if (warp < C) {
        t = s[lane][warp];   // column `warp`, the warps' sums side by side
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
        const int mine = static_cast<int>(blockIdx.x) * C + warp;
        if (lane == 0 && mine < D) out[mine] = t;
    }
}

// ---- rows of pairs of elements (even widths): the same sums, with rows on their way while others are
// worked on.  A block takes two rows at a time, whose sums share their exchanges and barriers, and copies
// the two after next into shared memory as it leaves their places; a thread reads only the words that
// it copied itself.  Arithmetic on pairs of neighbours (an element takes 8 instructions in the forward
// and 11 in the gradient; twice as many without).
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait_all_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// A thread takes 16 elements of a row, in runs of a 16-byte word: eight of bf16; four where there is fp32
// (neighbouring threads' words are neighbours then; with runs of eight, each of two words, a 32-byte piece came
// over in halves: 32768 x 4096 from fp32 to bf16, gradient 297 us for 237, forward, row by row, 187 for 124 and, with 32 elements a thread, 117).
// The forward's blocks that an SM holds:
constexpr int pair_blocks(int T) { return T == 64 ? 10 : T <= 128 ? 6 : T == 256 ? 3 : 1; }   // 65536 x 1024 with 8, 9, 10: 56, 50, 46 us
constexpr int kPairWidest = 8192;          // channels of a row that 512 threads take
constexpr size_t kPairSpace = 216 << 10;   // shared memory for it
template <class TX, class TY>
constexpr int kRun = kElem<TX> + kElem<TY> == 4 ? 8 : 4;

template <int B>
__device__ __forceinline__ void copy_small(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(B) : "memory");
}

// A thread's run of RUN elements, one word in shared memory.  WHOLE: copied and stored as such; else two
// elements at a time, `pairs` of which there are.
template <class T, int RUN, bool WHOLE>
struct Run {
    static constexpr int BYTES = RUN * kElem<T>, PAIRS = RUN / 2;
    static_assert(BYTES == 8 || BYTES == 16, "a word");
    static __device__ __forceinline__ void ask(const uint8_t* to, const T* from, int pairs) {
        const uint32_t at = ptx::smem_u32(to);
        if constexpr (WHOLE && BYTES == 16) {
            copy16(at, from);
        } else if constexpr (WHOLE) {
            copy_small<8>(at, from);
        } else {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i)
                if (i < pairs) copy_small<2 * kElem<T>>(at + i * 2 * kElem<T>, from + 2 * i);
        }
    }
    static __device__ __forceinline__ void get(const uint8_t* from, F2 (&x)[PAIRS]) {
        uint32_t w[BYTES / 4];
        if constexpr (BYTES == 16) {
            const uint4 u = *reinterpret_cast<const uint4*>(from);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(from);
            w[0] = u.x, w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            if constexpr (kElem<T> == 2) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            else x[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
    static __device__ __forceinline__ void put(T* to, const F2 (&x)[PAIRS], int pairs) {
        float v[RUN];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) split(x[i], v[2 * i], v[2 * i + 1]);
        if constexpr (WHOLE) {
            store_as<T, RUN>(to, v);
        } else {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                const float two[2] = {v[2 * i], v[2 * i + 1]};
                if (i < pairs) store_as<T, 2>(to + 2 * i, two);
            }
        }
    }
};

__device__ __forceinline__ float sum_of(F2 x) {
    float a, b;
    split(x, a, b);
    return a + b;
}
// A run's parameters, columns from c of which `pairs` pairs there are, or a value in place of them.
template <int RUN, bool WHOLE>
__device__ __forceinline__ void params(const float* p, int c, int pairs, float other, F2 (&x)[RUN / 2]) {
#pragma unroll
    for (int i = 0; i < RUN / 2; ++i) x[i] = both(other);
    if (!p) return;
    if constexpr (WHOLE) {
        if (pairs > 0) {
            const auto raw = load_raw<float, RUN>(p + c);
#pragma unroll
            for (int i = 0; i < RUN / 2; ++i) x[i] = pair(raw_at<float, RUN>(raw, 2 * i), raw_at<float, RUN>(raw, 2 * i + 1));
        }
    } else {
#pragma unroll
        for (int i = 0; i < RUN / 2; ++i)
            if (i < pairs) x[i] = pair(__ldg(p + c + 2 * i), __ldg(p + c + 2 * i + 1));
    }
}

template <class TX, class TY, int T, int R>
__global__ void __launch_bounds__(T * R, pair_blocks(T)) norm_fwd_pairs(const __grid_constant__ NormArgs a) {
    constexpr int RUN = kRun<TX, TY>, RUNS = 16 / RUN, PAIRS = RUN / 2;
    using X = Run<TX, RUN, true>;
    extern __shared__ __align__(16) uint8_t ring[];   // [2 turns][2 rows][RUNS][T R] words
    __shared__ float sums[2][4 * ((T + 31) / 32)];
    ptx::pdl_trigger();
    const int t = threadIdx.x % T;
    const int64_t step = 2 * static_cast<int64_t>(gridDim.x) * R;
    int64_t row = 2 * (static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / T);
    const int ahead = T < 32 ? 2 * (threadIdx.x % 32 / T) : 0;   // of the warp's first row: a warp stays together
    auto place = [&](int turn, int which, int j) { return ring + (((turn * 2 + which) * RUNS + j) * T * R + threadIdx.x) * X::BYTES; };
    auto ask = [&](int64_t of, int turn) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int j = 0; j < RUNS; ++j) {
                const int c = (j * T + t) * RUN;
                if (of + which < a.n && c < a.D) X::ask(place(turn, which, j), static_cast<const TX*>(a.x) + (of + which) * a.ld_x + c, PAIRS);
            }
        copies_close();
    };
    ptx::pdl_wait();
    ask(row, 0);
    ask(row + step, 1);
    F2 w[RUNS][PAIRS], b[RUNS][PAIRS];
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
        const int c = (j * T + t) * RUN;
        params<RUN, true>(a.weight, c, c < a.D ? PAIRS : 0, 1.f, w[j]);
        params<RUN, true>(a.bias, c, c < a.D ? PAIRS : 0, 0.f, b[j]);
    }
    for (int turn = 0; row - ahead < a.n; row += step, turn ^= 1) {
        copies_wait_all_but_one();
        F2 x[PAIRS];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            F2 u = both(0.f);
#pragma unroll
            for (int j = 0; j < RUNS; ++j) {
                if ((j * T + t) * RUN < a.D) {
                    X::get(place(turn, which, j), x);
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) u = add2(u, x[i]);
                }
            }
            s[which] = sum_of(u);
        }
        row_sums<T, 2>(s, sums[0]);
        const float mean[2] = {s[0] * a.inv_d, s[1] * a.inv_d};
        float q[4];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            F2 u = both(0.f), v = both(0.f);
            const F2 shift = both(-mean[which]);
#pragma unroll
            for (int j = 0; j < RUNS; ++j) {
                if ((j * T + t) * RUN < a.D) {
                    X::get(place(turn, which, j), x);
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        const F2 d = add2(x[i], shift);
                        u = add2(u, d);
                        v = fma2(d, d, v);
                    }
                }
            }
            q[2 * which] = sum_of(u), q[2 * which + 1] = sum_of(v);
        }
        row_sums<T, 4>(q, sums[1]);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (row + which >= a.n) break;
            const float delta = q[2 * which] * a.inv_d, sq = q[2 * which + 1];
            const float rstd = 1.0f / sqrtf(fmaxf(fmaf(-delta, delta, sq * a.inv_d), 0.f) + a.eps);
            if (t == 0) {
                if (a.mean) a.mean[row + which] = kept_mean(mean[which], delta, rstd);
                if (a.rstd) a.rstd[row + which] = sq == sq ? rstd : sq;   // fmaxf drops a NaN
            }
            TY* y = static_cast<TY*>(a.y) + (row + which) * a.ld_y;
            const F2 shift = both(-mean[which]), rest = both(-delta), scale = both(rstd);
#pragma unroll
            for (int j = 0; j < RUNS; ++j) {
                const int c = (j * T + t) * RUN;
                if (c < a.D) {
                    X::get(place(turn, which, j), x);
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) x[i] = fma2(mul2(add2(add2(x[i], shift), rest), scale), w[j][i], b[j][i]);
                    Run<TY, RUN, true>::put(y + c, x, PAIRS);
                }
            }
        }
        ask(row + 2 * step, turn);
    }
}

// As row_sums, for T neighbours of a block of T R threads; r: which of the R.
template <int T, int R, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float* s, int r) {
    if constexpr (T <= 32 || R == 1) {
        row_sums<T, N>(v, s);
    } else {
        constexpr int W = T / 32;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
        s += r * N * W;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) s[i * W + threadIdx.x % T / 32] = v[i];
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + r), "n"(T) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) t += s[i * W + w];
            v[i] = t;
        }
    }
}

// The gradient: one block an SM, of R rows' threads that go their own ways (barriers of T threads), so that
// there are as few sums of columns to store as SMs (2048 x 2048 bf16 11.6 us, with four blocks an SM 12.4; 4096 x
// 512 7.3, 8.3).
template <class TX, class TY, int T, int R, bool WHOLE>
__global__ void __launch_bounds__(T * R, 1) norm_bwd_pairs(const __grid_constant__ NormArgs a) {
    constexpr int RUN = kRun<TX, TY>, RUNS = 16 / RUN, PAIRS = RUN / 2;
    using X = Run<TX, RUN, WHOLE>;
    using Y = Run<TY, RUN, WHOLE>;
    constexpr int ROW = RUNS * (X::BYTES + Y::BYTES) * T * R;   // of a row of x and one of dy, each as [RUNS][T R] words
    extern __shared__ __align__(16) uint8_t ring[];             // [2 turns][2 rows] of them
    __shared__ float sums[2][6 * R * ((T + 31) / 32)];
    constexpr int SUB = T < 32 ? 32 / T : 1;                 // rows of a warp
    const int t = threadIdx.x % T, r = static_cast<int>(threadIdx.x) / T;
    const int64_t step = 2 * static_cast<int64_t>(gridDim.x) * R;
    const int ahead = 2 * (r % SUB);   // of the warp's first row: a warp stays together
    int64_t row = 2 * SUB * (static_cast<int64_t>(r / SUB) * gridDim.x + blockIdx.x) + ahead;
    auto place_x = [&](int turn, int which, int j) { return ring + (turn * 2 + which) * ROW + (j * T * R + threadIdx.x) * X::BYTES; };
    auto place_d = [&](int turn, int which, int j) { return ring + (turn * 2 + which) * ROW + (RUNS * X::BYTES + j * Y::BYTES) * T * R + threadIdx.x * Y::BYTES; };
    int pairs[RUNS];   // of each run, that lie in the row
#pragma unroll
    for (int j = 0; j < RUNS; ++j) pairs[j] = min(PAIRS, max(0, (a.D - (j * T + t) * RUN) / 2));
    const auto in_row = [&](int j, int i) { return WHOLE ? pairs[j] > 0 : i < pairs[j]; };
    float mean[2], rstd[2], mean_next[2] = {0.f, 0.f}, rstd_next[2] = {0.f, 0.f};
    auto ask = [&](int64_t of, int turn) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int j = 0; j < RUNS; ++j) {
                const int c = (j * T + t) * RUN;
                if (of + which < a.n && pairs[j] > 0) {
                    X::ask(place_x(turn, which, j), static_cast<const TX*>(a.x) + (of + which) * a.ld_x + c, pairs[j]);
                    Y::ask(place_d(turn, which, j), static_cast<const TY*>(a.dy) + (of + which) * a.ld_dy + c, pairs[j]);
                }
            }
        copies_close();
    };
    auto stats = [&](int64_t of, float (&m)[2], float (&s)[2]) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const bool in = of + which < a.n;
            m[which] = in ? __ldg(a.mean + of + which) : 0.f;
            s[which] = in ? __ldg(a.rstd + of + which) : 0.f;
        }
    };
    ptx::pdl_wait();
    ask(row, 0);
    ask(row + step, 1);
    stats(row, mean, rstd);
    F2 w[RUNS][PAIRS], dw[RUNS][PAIRS], db[RUNS][PAIRS];
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
        params<RUN, WHOLE>(a.weight, (j * T + t) * RUN, pairs[j], 1.f, w[j]);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) dw[j][i] = db[j][i] = both(0.f);
    }
    for (int turn = 0; row - ahead < a.n; row += step, turn ^= 1) {
        stats(row + step, mean_next, rstd_next);
        copies_wait_all_but_one();
        F2 x[PAIRS], d[PAIRS];
        float s[6];   // a row's sums of g, g (x - mean), x - mean
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            F2 u0 = both(0.f), u1 = u0, u2 = u0;
            const F2 shift = both(-mean[which]);
            if (row + which < a.n) {
#pragma unroll
                for (int j = 0; j < RUNS; ++j) {
                    if (pairs[j] > 0) {
                        X::get(place_x(turn, which, j), x);
                        Y::get(place_d(turn, which, j), d);
#pragma unroll
                        for (int i = 0; i < PAIRS; ++i) {
                            if (!in_row(j, i)) continue;
                            const F2 e = add2(x[i], shift), g = mul2(d[i], w[j][i]);
                            u0 = add2(u0, g);
                            u1 = fma2(g, e, u1);
                            u2 = add2(u2, e);
                        }
                    }
                }
            }
            s[3 * which] = sum_of(u0), s[3 * which + 1] = sum_of(u1), s[3 * which + 2] = sum_of(u2);
        }
        group_sums<T, R, 6>(s, sums[turn], r);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (row + which >= a.n) break;
            const float delta = s[3 * which + 2] * a.inv_d;
            const F2 along = both(-rstd[which] * fmaf(-delta, s[3 * which], s[3 * which + 1]) * a.inv_d);   // minus the sum of g xhat / D
            const F2 base = both(-rstd[which] * s[3 * which] * a.inv_d);
            const F2 shift = both(-mean[which]), rest = both(-delta), scale = both(rstd[which]);
            TX* dx = static_cast<TX*>(a.y) + (row + which) * a.ld_y;
#pragma unroll
            for (int j = 0; j < RUNS; ++j) {
                const int c = (j * T + t) * RUN;
                if (pairs[j] > 0) {
                    X::get(place_x(turn, which, j), x);
                    Y::get(place_d(turn, which, j), d);
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        if (!in_row(j, i)) continue;
                        const F2 xhat = mul2(add2(add2(x[i], shift), rest), scale);
                        dw[j][i] = fma2(d[i], xhat, dw[j][i]);
                        db[j][i] = add2(db[j][i], d[i]);
                        x[i] = fma2(mul2(xhat, scale), along, fma2(mul2(d[i], w[j][i]), scale, base));
                    }
                    X::put(dx + c, x, pairs[j]);
                }
            }
        }
        ask(row + 2 * step, turn);
#pragma unroll
        for (int which = 0; which < 2; ++which) mean[which] = mean_next[which], rstd[which] = rstd_next[which];
    }
    ptx::pdl_trigger();   // not before: blocks that wait would take registers from rows (1048576 x 64 88, 76 us)
    if (!a.part) return;
    float v[2][16];   // the weight's and the bias's
#pragma unroll
    for (int j = 0; j < RUNS; ++j)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            split(dw[j][i], v[0][RUN * j + 2 * i], v[0][RUN * j + 2 * i + 1]);
            split(db[j][i], v[1][RUN * j + 2 * i], v[1][RUN * j + 2 * i + 1]);
        }
    // Rows side by side, added in a fixed order: a warp's by lanes, the block's through the ring's place
    if constexpr (T < 32) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
                for (int d = T; d < 32; d *= 2) v[which][e] += __shfl_xor_sync(0xffffffffu, v[which][e], d);
    }
    constexpr int GROUPS = R / SUB;
    float* cols = reinterpret_cast<float*>(ring);   // [GROUPS][2][16][T]
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (r % SUB == 0) {
#pragma unroll
        for (int e = 0; e < 32; ++e) cols[((r / SUB) * 32 + e) * T + t] = v[e / 16][e % 16];
    }
    __syncthreads();
    for (int unit = threadIdx.x; unit < 8 * T; unit += T * R) {   // four columns of one of the two sums
        const int four = unit / T, of = unit % T;                // four = (which, run, part of it)
        const int c = ((four & 3) * 4 / RUN * T + of) * RUN + (four & 3) * 4 % RUN;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < GROUPS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] += cols[(k * 32 + four * 4 + i) * T + of];
        float* to = a.part + (static_cast<int64_t>(four >> 2) * gridDim.x + blockIdx.x) * a.D + c;
        if constexpr (WHOLE) {
            if (c < a.D) store_as<float, 4>(to, x);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < a.D) to[i] = x[i];
        }
    }
}

constexpr int kWidest = 16384;   // channels that a block of 1024 threads holds

// Threads a row takes at 16 elements each: part of a warp (where its elements come eight at a time), a
// warp, or a block of 64 to 1024.
int row_threads(int64_t D, int V) {
    int t = V >= 4 ? 8 : 32;
    while (static_cast<int64_t>(t) * 16 < D) t *= 2;
    return t;
}
constexpr int rows_beside(int T) { return T <= 32 ? 128 / T : 1; }   // rows of a block

int bwd_parts(int64_t n, int64_t D) {
    if (D > kWidest) return 0;
    return static_cast<int>(std::min<int64_t>(kPartMax, n));   // as few rows a block as there may be
}

template <bool BWD, class TX, class TY, int T, int R, int V, int EPT = 16>
int launch_rows(const NormArgs& a, int grid, int num_sms, cudaStream_t s) {
    if constexpr (T == 32 && V <= 2 && EPT == 16) {   // narrow rows: fewer elements a thread (1048576 x 63 361, 265 us)
        if (a.D <= 64) return launch_rows<BWD, TX, TY, T, R, V, 2>(a, grid, num_sms, s);
        if (a.D <= 128) return launch_rows<BWD, TX, TY, T, R, V, 4>(a, grid, num_sms, s);
        if (a.D <= 256) return launch_rows<BWD, TX, TY, T, R, V, 8>(a, grid, num_sms, s);
    }
    if constexpr (BWD) {
        return launch_pdl(norm_bwd<TX, TY, T, R, EPT, V>, dim3(grid), dim3(T * R), R > 1 ? 2 * EPT * 32 * sizeof(float) : 0, s, a);
    } else {
        // More than 256 channels off 16-byte words: blocks that stay (32768 x 4095 bf16 136 us, a block a row 204;
        // 500 x 4095 4.4, 5.4; 4096 x 511 4.2, 5.9; narrower 500000 x 127 167, 129; of whole words 32768 x 4096
        // from fp32 135, 124).
        if constexpr (V <= 2 && EPT == 16 && T <= 512)
            return launch_pdl(norm_fwd_loop<TX, TY, T, R, EPT, V>, dim3(std::min(grid, num_sms * loop_blocks(T * R))), dim3(T * R), 0, s, a);
        else
            return launch_pdl(norm_fwd<TX, TY, T, R, EPT, V>, dim3(grid), dim3(T * R), 0, s, a);
    }
}

template <bool BWD, class TX, class TY, int V>
int pick_rows(const NormArgs& a, int num_sms, int* parts, cudaStream_t s) {
    const int T = row_threads(a.D, BWD ? 1 : V), R = rows_beside(T);
    int grid = static_cast<int>((static_cast<int64_t>(a.n) + R - 1) / R);
    if (BWD) grid = std::min(grid, kPartMax);
    *parts = grid;
    switch (T) {
    case 8:
        if constexpr (!BWD && V >= 4) return launch_rows<BWD, TX, TY, 8, rows_beside(8), V>(a, grid, num_sms, s);
    case 16:
        if constexpr (!BWD && V >= 4) return launch_rows<BWD, TX, TY, 16, rows_beside(16), V>(a, grid, num_sms, s);
    case 32: return launch_rows<BWD, TX, TY, 32, rows_beside(32), V>(a, grid, num_sms, s);
    case 64: return launch_rows<BWD, TX, TY, 64, 1, V>(a, grid, num_sms, s);
    case 128: return launch_rows<BWD, TX, TY, 128, 1, V>(a, grid, num_sms, s);
    case 256: return launch_rows<BWD, TX, TY, 256, 1, V>(a, grid, num_sms, s);
    case 512: return launch_rows<BWD, TX, TY, 512, 1, V>(a, grid, num_sms, s);
    default:
        if constexpr (BWD) return launch_rows<BWD, TX, TY, 1024, 1, V>(a, grid, num_sms, s);
        else return launch_rows<BWD, TX, TY, 512, 1, V, 32>(a, grid, num_sms, s);   // two rows an SM
    }
}

// The forward with 32 elements a thread, half of T threads a row.
template <class TX, class TY>
int pick_tall(const NormArgs& a, int T, int num_sms, cudaStream_t s) {
    constexpr int V = kRun<TX, TY>;
    const auto blocks = [&](int R) { return static_cast<int>((static_cast<int64_t>(a.n) + R - 1) / R); };
    switch (T) {
    case 16: return launch_rows<false, TX, TY, 8, 16, V, 32>(a, blocks(16), num_sms, s);
    case 32: return launch_rows<false, TX, TY, 16, 8, V, 32>(a, blocks(8), num_sms, s);
    case 64: return launch_rows<false, TX, TY, 32, 4, V, 32>(a, blocks(4), num_sms, s);
    case 128: return launch_rows<false, TX, TY, 64, 1, V, 32>(a, a.n, num_sms, s);
    case 256: return launch_rows<false, TX, TY, 128, 1, V, 32>(a, a.n, num_sms, s);
    default: return launch_rows<false, TX, TY, 256, 1, V, 32>(a, a.n, num_sms, s);
    }
}

// Rows side by side in the gradient's blocks: whole warps, up to 512 threads and the shared memory.
template <class TX, class TY, int T>
constexpr int bwd_beside() {
    const int each = 4 * 16 * (kElem<TX> + kElem<TY>);   // bytes of a thread
    const int threads = std::min(512, static_cast<int>(kPairSpace) / each) / std::max(T, 32) * std::max(T, 32);
    return threads / T;
}

template <bool BWD, class TX, class TY, int T, bool WHOLE>
int launch_pairs(const NormArgs& a, int num_sms, int* parts, cudaStream_t s) {
    if constexpr (BWD) {
        constexpr int R = bwd_beside<TX, TY, T>(), SUB = T < 32 ? 32 / T : 1;
        if constexpr (R == 0) {
            return pick_rows<BWD, TX, TY, WHOLE ? kRun<TX, TY> : 2>(a, num_sms, parts, s);
        } else {
            constexpr int smem = 4 * 16 * T * R * (kElem<TX> + kElem<TY>);
            static_assert(smem >= R / SUB * 32 * T * 4, "the columns' sums");
            *parts = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(a.n) + 2 * SUB - 1) / (2 * SUB), num_sms));
            TERN_CUDA_TRY(cudaFuncSetAttribute(norm_bwd_pairs<TX, TY, T, R, WHOLE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
            return launch_pdl(norm_bwd_pairs<TX, TY, T, R, WHOLE>, dim3(*parts), dim3(T * R), smem, s, a);
        }
    } else {
        constexpr int R = rows_beside(T);
        constexpr size_t smem = 4u * 16 * T * R * kElem<TX>;
        const int64_t pairs = (static_cast<int64_t>(a.n) + 2 * R - 1) / (2 * R);
        const int blocks = std::min(pair_blocks(T), static_cast<int>(kPairSpace / smem));
        const int grid = static_cast<int>(std::min(pairs, static_cast<int64_t>(num_sms) * blocks));
        if (smem > 40 * 1024) TERN_CUDA_TRY(cudaFuncSetAttribute(norm_fwd_pairs<TX, TY, T, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
        return launch_pdl(norm_fwd_pairs<TX, TY, T, R>, dim3(grid), dim3(T * R), smem, s, a);
    }
}

template <bool BWD, class TX, class TY, bool WHOLE>
int pick_pairs(const NormArgs& a, int num_sms, int* parts, cudaStream_t s) {
    switch (row_threads(a.D, 8)) {
    case 8: return launch_pairs<BWD, TX, TY, 8, WHOLE>(a, num_sms, parts, s);
    case 16: return launch_pairs<BWD, TX, TY, 16, WHOLE>(a, num_sms, parts, s);
    case 32: return launch_pairs<BWD, TX, TY, 32, WHOLE>(a, num_sms, parts, s);
    case 64: return launch_pairs<BWD, TX, TY, 64, WHOLE>(a, num_sms, parts, s);
    case 128: return launch_pairs<BWD, TX, TY, 128, WHOLE>(a, num_sms, parts, s);
    case 256: return launch_pairs<BWD, TX, TY, 256, WHOLE>(a, num_sms, parts, s);
    default: return launch_pairs<BWD, TX, TY, 512, WHOLE>(a, num_sms, parts, s);
    }
}

bool all_allow(const NormArgs& a, bool bwd, int V, int ex, int ey) {
    const uintptr_t b = static_cast<uintptr_t>(V * 4 < 16 ? V * 4 : 16) - 1;
    auto params = [&](const float* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & b) == 0; };
    return rows_allow(a.x, a.ld_x, a.n, a.D, V, ex) && rows_allow(a.y, a.ld_y, a.n, a.D, V, bwd ? ex : ey) &&
           (!bwd || rows_allow(a.dy, a.ld_dy, a.n, a.D, V, ey)) && params(a.weight) && params(a.bias);
}

// The blocks' (or parts') sums [2][parts][D], in their order.
int launch_cols(const float* part, int parts, int D, float* dweight, float* dbias, cudaStream_t s) {
    if (D <= 2048) return launch_pdl(norm_cols<8>, dim3((D + 7) / 8, 2), dim3(1024), 0, s, part, parts, D, dweight, dbias);
    return launch_pdl(norm_cols<32>, dim3((D + 31) / 32, 2), dim3(1024), 0, s, part, parts, D, dweight, dbias);
}

template <bool BWD, class TX, class TY>
int run_norm(const NormArgs& a, float* dweight, float* dbias, int num_sms, cudaStream_t s) {
    if (a.D > kWidest) {
        if constexpr (BWD) {
            if (a.n > 0)
                if (int st = launch_pdl(norm_bwd_wide<TX, TY>, dim3(a.n), dim3(1024), 0, s, a)) return st;
            if (!dweight && !dbias) return TERN_OK;
            const int parts = wide_parts(a.n);
            if (int st = launch_pdl(norm_cols_wide<TX, TY>, dim3((a.D + 255) / 256, parts), dim3(256), 0, s, a, dweight, dbias)) return st;
            return parts > 1 ? launch_cols(a.part + a.n, parts, a.D, dweight, dbias, s) : TERN_OK;
        } else {
            return launch_pdl(norm_fwd_wide<TX, TY>, dim3(a.n), dim3(1024), 0, s, a);
        }
    }
    int parts = 0;
    if (a.n > 0) {
        constexpr int ex = kElem<TX>, ey = kElem<TY>;
        int st;
        // Pairs of rows where there are some for each SM: the gradient (32768 x 4096 bf16 137 us, row by row 308; 64 x
        // 4096 7.2, 5.7; 304 x 4096 7.8, 8.6; 600 x 1024 6.3, 7.6) and the forward of bf16 (32768 x 4096 99 us, 124;
        // 65536 x 1024 46, 69).  Else, and of bf16 rows that leave many of those threads idle or take 512, the forward
        // gives a thread 32 elements as soon as rows are more than fit at once with 16, from pairs or 16 to 32:
        // from fp32 32768 x 4096 124, 117 us, 65536 x 1024 71, 61, 65536 x 600 69, 39, 8192 x 512 5.1, 4.6, 65536 x 512 31,
        // 32, 600 x 4096 3.6, 4.9; bf16 32768 x 8192 227, 222, 32768 x 6000 210, 180, 262144 x 160 48, 37, 32768 x
        // 4096 99, 105.
        constexpr int V = kRun<TX, TY>;
        const int T = row_threads(a.D, 8);
        const bool many = a.D <= kPairWidest && a.n > num_sms * (BWD && T >= 256 ? 1 : 2 * rows_beside(T));
        const bool tall = a.D <= kPairWidest && static_cast<int64_t>(a.n) * T > 1536 * num_sms &&
                          (V == 4 ? T >= 32 : T == 512 || (T >= 16 && a.D * 6 < 16 * 5 * T));
        if (all_allow(a, BWD, V, ex, ey)) {
            if constexpr (BWD) {
                st = many ? pick_pairs<BWD, TX, TY, true>(a, num_sms, &parts, s) : pick_rows<BWD, TX, TY, V>(a, num_sms, &parts, s);
            } else if (tall) {
                st = pick_tall<TX, TY>(a, T, num_sms, s);
            } else {
                if constexpr (V == 8) st = many ? pick_pairs<BWD, TX, TY, true>(a, num_sms, &parts, s) : pick_rows<BWD, TX, TY, V>(a, num_sms, &parts, s);
                else st = pick_rows<BWD, TX, TY, V>(a, num_sms, &parts, s);
            }
        } else if (all_allow(a, BWD, 2, ex, ey)) {
            if constexpr (BWD) st = many ? pick_pairs<BWD, TX, TY, false>(a, num_sms, &parts, s) : pick_rows<BWD, TX, TY, 2>(a, num_sms, &parts, s);
            else st = pick_rows<BWD, TX, TY, 2>(a, num_sms, &parts, s);
        } else {
            st = pick_rows<BWD, TX, TY, 1>(a, num_sms, &parts, s);
        }
        if (st) return st;
    }
    if (BWD && (dweight || dbias)) return launch_cols(a.part, parts, a.D, dweight, dbias, s);   // of no rows: zeros
    return TERN_OK;
}

template <bool BWD>
int run_types(const NormArgs& a, int tx, int ty, float* dweight, float* dbias, int num_sms, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (tx == TERN_BF16)
        return ty == TERN_BF16 ? run_norm<BWD, B, B>(a, dweight, dbias, num_sms, s) : run_norm<BWD, B, float>(a, dweight, dbias, num_sms, s);
    return ty == TERN_BF16 ? run_norm<BWD, float, B>(a, dweight, dbias, num_sms, s) : run_norm<BWD, float, float>(a, dweight, dbias, num_sms, s);
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
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    NormArgs a{};
    a.x = x, a.y = y, a.weight = weight, a.bias = bias, a.mean = mean, a.rstd = rstd;
    a.ld_x = ld_x, a.ld_y = ld_y, a.n = static_cast<int>(n), a.D = static_cast<int>(D), a.eps = eps;
    a.inv_d = static_cast<float>(1.0 / static_cast<double>(D));
    return run_types<false>(a, x_dtype, y_dtype, nullptr, nullptr, num_sms, static_cast<cudaStream_t>(stream));
}

extern "C" size_t tern_norm_bwd_workspace(int64_t n, int64_t D) {
    if (!sizes_ok(n, D)) return 0;
    // the blocks' column sums; for rows wider than a block holds one value a row, and the parts' column sums
    const int parts = D > kWidest ? wide_parts(n) : bwd_parts(n, D);
    const int64_t floats = (D > kWidest ? n : 0) + (D > kWidest && parts == 1 ? 0 : 2 * static_cast<int64_t>(parts) * D);
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
    int num_sms = 0;
    if (int st = check_device(&num_sms)) return st;
    NormArgs a{};
    a.x = x, a.dy = dy, a.y = dx, a.weight = weight, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.ld_x = ld_x, a.ld_dy = ld_dy, a.ld_y = ld_dx, a.n = static_cast<int>(n), a.D = static_cast<int>(D);
    a.inv_d = static_cast<float>(1.0 / static_cast<double>(D));
    return run_types<true>(a, x_dtype, y_dtype, dweight, dbias, num_sms, static_cast<cudaStream_t>(stream));
}
