// ew_layernorm.hip -- the layer norm with the residual's addition, and its
// gradient, for CDNA4 (gfx950).

#include "ew_rows_vec.h"

namespace ew {

// Threads of a block: a row's waves, or four waves of short rows.
constexpr int layernorm_block(int waves) { return waves < 3 ? 256 : waves * 64; }

// Which of a block's rows a thread works on, the same in all of a wave, and its
// place among the row's threads.
template <int Threads, int Rows>
__device__ __forceinline__ uint32_t row_of_thread()
{
    if constexpr (Rows == 1) return 0;
    else return (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / Threads));
}
template <int Threads, int Rows>
__device__ __forceinline__ uint32_t place_in_row()
{
    return Rows == 1 ? threadIdx.x : threadIdx.x % Threads;
}

// A mean in two binary32 numbers: h - mean as (h - hi) - lo keeps 24 bits of
// the difference however far the row lies from 0, where one number would leave
// the mean's rounding in it (a row of equal values would not give 0).
struct Mean {
    float hi, lo;
    __device__ explicit Mean(double m) : hi((float)m), lo((float)(m - (double)(float)m)) {}
};

// Sum of one value a wave (scratch[0 .. Waves)) in all lanes: of eight or
// sixteen by lane exchanges, which hold one of them in a register, not all.
template <int Waves>
__device__ __forceinline__ double join_waves(const double *scratch)
{
    if constexpr (Waves == 8 || Waves == 16) {
        double x = scratch[threadIdx.x % Waves];
        x += dpp64<0xB1>(x);
        x += dpp64<0x4E>(x);
        x += dpp64<0x141>(x);
        if constexpr (Waves == 16) x += dpp64<0x140>(x);
        return x;
    }
    double x = scratch[0];
#pragma unroll
    for (int w = 1; w < Waves; ++w) x += scratch[w];
    return x;
}

template <int Waves>
__device__ __forceinline__ float join_waves(const float *scratch)
{
    if constexpr (Waves == 8 || Waves == 16) {
        float x = quad_reduce<Sum>(scratch[threadIdx.x % Waves]);
        x += dpp<0x141>(x);
        if constexpr (Waves == 16) x += dpp<0x140>(x);
        return x;
    }
    float x = scratch[0];
#pragma unroll
    for (int w = 1; w < Waves; ++w) x += scratch[w];
    return x;
}

// Sum over a row's Waves waves in all of them.  scratch: the row's own.
template <int Waves>
__device__ __forceinline__ double row_sum(double x, double *scratch)
{
    x = wave_sum64(x);
    if constexpr (Waves > 1) {
        if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64 % Waves] = x;
        __syncthreads();
        x = join_waves<Waves>(scratch);
    }
    return x;
}

template <int Waves>
__device__ __forceinline__ float row_sum(float x, float *scratch)
{
    x = wave_reduce<Sum>(x);
    if constexpr (Waves > 1) {
        if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64 % Waves] = x;
        __syncthreads();
        x = join_waves<Waves>(scratch);
    }
    return x;
}

// Sum of a vector's elements in binary64.
template <typename T>
__device__ __forceinline__ double sum64(u32x4 v)
{
    const typename Vec<T>::wide f = Vec<T>::widen(v);
    double a = f[0], b = f[1];
#pragma unroll
    for (int j = 2; j < Vec<T>::N; j += 2) {
        a += (double)f[j];
        b += (double)f[j + 1];
    }
    return a + b;
}

// Sum of the squares of a vector's differences from the mean, of those of its
// elements that lie in the row.
template <typename T>
__device__ __forceinline__ float squares(u32x4 v, const Mean &m, uint32_t cols, uint32_t at)
{
    constexpr uint32_t N = Vec<T>::N;
    if (at >= cols) return 0.0f;
    typename Vec<T>::wide d = (Vec<T>::widen(v) - m.hi) - m.lo;
    if (at + N > cols) {
#pragma unroll
        for (uint32_t j = 0; j < N; ++j)
            if (at + j >= cols) d[j] = 0.0f;
    }
    float sum = 0.0f;
#pragma unroll
    for (uint32_t j = 0; j < N; ++j) sum = __builtin_fmaf(d[j], d[j], sum);
    return sum;
}

template <typename T>
__device__ __forceinline__ u32x4 normed(u32x4 v, const Mean &m, float rstd,
                                        typename Vec<T>::wide w, typename Vec<T>::wide b)
{
    typename Vec<T>::wide y = (Vec<T>::widen(v) - m.hi) - m.lo;
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) y[j] = __builtin_fmaf(y[j] * rstd, w[j], b[j]);
    return Vec<T>::narrow(y);
}

// The weight's (or bias's) vector; `none` where it is absent.
template <typename T>
__device__ __forceinline__ typename Vec<T>::wide affine(const void *p, u32x4 v, float none)
{
    return p ? Vec<T>::widen(v) : typename Vec<T>::wide(none);
}

// ---------------------------------------------------------------------------
// Forward, rows that fit in registers: Waves waves a row, V vectors a lane
// ---------------------------------------------------------------------------

template <typename T, int Waves, int V>
__global__ void __launch_bounds__(layernorm_block(Waves)) ew_layernorm_row_kernel(LayerNormArgs a)
{
    constexpr uint32_t N = Vec<T>::N, kThreads = Waves * 64;
    constexpr uint32_t kRows = layernorm_block(Waves) / kThreads;
    // weight and bias are on their way with the row, unless they would not fit
    // in registers
    constexpr bool kEarly = V < 3;
    // two sets, used in turn: a wave is at most one barrier ahead of another
    __shared__ double sums[2][layernorm_block(Waves) / 64];
    __shared__ float sqs[2][layernorm_block(Waves) / 64];
    const uint32_t group = row_of_thread<kThreads, kRows>(), i = place_in_row<kThreads, kRows>();
    const T *const weight = static_cast<const T *>(a.weight), *const bias = static_cast<const T *>(a.bias);
    const auto at = [&](int k) { return (i + k * kThreads) * N; };
    int set = 0;
    // a block's rows go round together (the barriers)
    for (uint64_t r0 = (uint64_t)blockIdx.x * kRows; r0 < a.rows;
         r0 += (uint64_t)gridDim.x * kRows, set ^= 1) {
        const bool live = r0 + group < a.rows;
        const uint64_t r = live ? r0 + group : r0;
        u32x4 h[V], w[V], b[V];
        const T *const x = static_cast<const T *>(a.x) + r * a.x_stride;
#pragma unroll
        for (int k = 0; k < V; ++k) h[k] = load_vec<T, true, true>(x, a.cols, at(k));
        const auto fetch_affine = [&](int k) {
            if (weight) w[k] = load_vec<T, false, true>(weight, a.cols, at(k));
            if (bias) b[k] = load_vec<T, false, true>(bias, a.cols, at(k));
        };
        if (a.residual) {
            const T *const p = static_cast<const T *>(a.residual) + r * a.residual_stride;
            u32x4 res[V];
#pragma unroll
            for (int k = 0; k < V; ++k) res[k] = load_vec<T, true, true>(p, a.cols, at(k));
            if constexpr (kEarly)
#pragma unroll
                for (int k = 0; k < V; ++k) fetch_affine(k);
#pragma unroll
            for (int k = 0; k < V; ++k)
                h[k] = Vec<T>::narrow(Vec<T>::widen(h[k]) + Vec<T>::widen(res[k]));
        } else if constexpr (kEarly) {
#pragma unroll
            for (int k = 0; k < V; ++k) fetch_affine(k);
        }
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            h[k] = settle<T>(h[k], a.cols, at(k));
            sum += sum64<T>(h[k]);
        }
        // the outputs may be the inputs: nothing is stored before every wave
        // of the row has loaded (a row of one wave loads before it stores)
        const double m64 = row_sum<Waves>(sum, sums[set] + group * Waves) / (double)a.cols;
        const Mean m(m64);
        if (live && a.total) {
            T *const total = static_cast<T *>(a.total) + r * a.total_stride;
#pragma unroll
            for (int k = 0; k < V; ++k) store_vec<T, true>(total, a.cols, at(k), h[k]);
        }
        float sq = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) sq += squares<T>(h[k], m, a.cols, at(k));
        sq = row_sum<Waves>(sq, sqs[set] + group * Waves);
        const float rstd = 1.0f / __builtin_sqrtf(sq / (float)a.cols + a.eps);
        if (live && i == 0) {
            if (a.mean) a.mean[r] = m.hi;
            if (a.rstd) a.rstd[r] = rstd;
        }
        if (!live) continue;
        T *const y = static_cast<T *>(a.y) + r * a.y_stride;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (!kEarly) fetch_affine(k);
            const auto wide = affine<T>(weight, settle<T>(w[k], a.cols, at(k)), 1.0f);
            const auto shift = affine<T>(bias, settle<T>(b[k], a.cols, at(k)), 0.0f);
            store_vec<T, true>(y, a.cols, at(k), normed<T>(h[k], m, rstd, wide, shift));
        }
    }
}

// ---------------------------------------------------------------------------
// Forward, longer rows: a block a row, three passes over it
// ---------------------------------------------------------------------------

constexpr int kLongBlock = 1024;
constexpr int kLongWaves = kLongBlock / 64;

template <typename T>
__global__ void __launch_bounds__(kLongBlock) ew_layernorm_long_kernel(LayerNormArgs a)
{
    constexpr uint32_t N = Vec<T>::N;
    __shared__ double sums[2][kLongWaves];
    __shared__ float sqs[2][kLongWaves];
    const T *const weight = static_cast<const T *>(a.weight), *const bias = static_cast<const T *>(a.bias);
    int set = 0;
    for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x, set ^= 1) {
        const T *const x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *const res =
            a.residual ? static_cast<const T *>(a.residual) + r * a.residual_stride : nullptr;
        T *const total = a.total ? static_cast<T *>(a.total) + r * a.total_stride : nullptr;
        const auto value = [&](uint32_t at) {
            u32x4 h = settle<T>(load_vec<T, false>(x, a.cols, at), a.cols, at);
            if (res)
                h = Vec<T>::narrow(Vec<T>::widen(h) + Vec<T>::widen(settle<T>(
                                       load_vec<T, false>(res, a.cols, at), a.cols, at)));
            return h;
        };
        // (the first pass stores total where its thread reads it back: total
        // may be x or residual)
        const auto again = [&](uint32_t at) {
            return total ? settle<T>(load_vec<T, false>(total, a.cols, at), a.cols, at) : value(at);
        };
        double sum = 0.0;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
            const u32x4 h = value(at);
            sum += sum64<T>(h);
            if (total) store_vec(total, a.cols, at, h);
        }
        const double m64 = row_sum<kLongWaves>(sum, sums[set]) / (double)a.cols;
        const Mean m(m64);
        float sq = 0.0f;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N)
            sq += squares<T>(again(at), m, a.cols, at);
        sq = row_sum<kLongWaves>(sq, sqs[set]);
        const float rstd = 1.0f / __builtin_sqrtf(sq / (float)a.cols + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = m.hi;
            if (a.rstd) a.rstd[r] = rstd;
        }
        T *const y = static_cast<T *>(a.y) + r * a.y_stride;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
            u32x4 w{}, b{};
            if (weight) w = settle<T>(load_vec<T, false>(weight, a.cols, at), a.cols, at);
            if (bias) b = settle<T>(load_vec<T, false>(bias, a.cols, at), a.cols, at);
            store_vec(y, a.cols, at, normed<T>(again(at), m, rstd, affine<T>(weight, w, 1.0f),
                                               affine<T>(bias, b, 0.0f)));
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

// dweight and dbias are added up in two steps: at most this many blocks sum a
// part of the rows each, then the parts are summed.
constexpr uint32_t kParts = 256;

// Floats of one part's sums of dweight (those of dbias follow): whole vectors.
__host__ __device__ constexpr uint64_t sums_pitch(uint64_t cols) { return (cols + 7) & ~(uint64_t)7; }

// Two sums over a row's Waves waves with one barrier.
template <int Waves>
__device__ __forceinline__ void row_sum2(float &x, float &y, float *xs, float *ys)
{
    x = wave_reduce<Sum>(x);
    y = wave_reduce<Sum>(y);
    if constexpr (Waves > 1) {
        if (threadIdx.x % 64 == 0) {
            xs[threadIdx.x / 64 % Waves] = x;
            ys[threadIdx.x / 64 % Waves] = y;
        }
        __syncthreads();
        x = join_waves<Waves>(xs);
        y = join_waves<Waves>(ys);
    }
}

// Rows that fit in registers: Waves waves a row, V vectors a lane, Groups rows
// at a time in a block, which adds up dweight and dbias over its rows.
template <typename T, int Waves, int V, int Groups>
__global__ void __launch_bounds__(Waves * 64 * Groups) ew_layernorm_grad_kernel(LayerNormGradArgs a)
{
    constexpr uint32_t N = Vec<T>::N, kThreads = Waves * 64;
    using Wide = typename Vec<T>::wide;
    __shared__ float firsts[2][Waves * Groups], seconds[2][Waves * Groups];
    __shared__ float joined[Groups > 1 ? kThreads * V * N : 1];
    const uint32_t group = row_of_thread<kThreads, Groups>(), i = place_in_row<kThreads, Groups>();
    // the next row is on its way while this one is worked on, and the weight
    // stays, unless they would not fit in registers
    constexpr bool kAhead = V < 3;
    const T *const weight = static_cast<const T *>(a.weight);
    const auto at = [&](int k) { return (i + k * kThreads) * N; };
    u32x4 wv[kAhead ? V : 1];
    const auto fetch_weight = [&](int k) {
        return weight ? settle<T>(load_vec<T, false, true>(weight, a.cols, at(k)), a.cols, at(k))
                      : u32x4{};
    };
    if constexpr (kAhead)
#pragma unroll
        for (int k = 0; k < V; ++k) wv[k] = fetch_weight(k);
    const auto factor = [&](int k) {
        return affine<T>(weight, kAhead ? wv[kAhead ? k : 0] : fetch_weight(k), 1.0f);
    };
    const auto fetch = [&](u32x4 (&v)[V], const void *p, uint64_t first) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            v[k] = load_vec<T, true, true>(static_cast<const T *>(p) + first, a.cols, at(k));
    };
    Wide dw[V], db[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        dw[k] = Wide(0.0f);
        db[k] = Wide(0.0f);
    }
    u32x4 dy[V], x[V], dt[kAhead ? V : 1];
    float mean = 0.0f, rstd = 0.0f;
    const auto fetch_row = [&](uint64_t r0) {
        const uint64_t r = r0 + group < a.rows ? r0 + group : r0;
        fetch(dy, a.dy, r * a.dy_stride);
        fetch(x, a.x, r * a.x_stride);
        if constexpr (kAhead)
            if (a.dtotal) fetch(dt, a.dtotal, r * a.dtotal_stride);
        mean = a.mean[r];
        rstd = a.rstd[r];
    };
    uint64_t r0 = (uint64_t)blockIdx.x * Groups;
    const uint64_t step = (uint64_t)gridDim.x * Groups;
    if (kAhead && r0 < a.rows) fetch_row(r0);
    for (int set = 0; r0 < a.rows; r0 += step, set ^= 1) {
        const bool live = r0 + group < a.rows;
        const uint64_t r = live ? r0 + group : r0;
        if constexpr (!kAhead) fetch_row(r0);
        const float rs = rstd, mu = mean;
        u32x4 dyv[V], xv[V], dtv[kAhead ? V : 1];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dyv[k] = settle<T>(dy[k], a.cols, at(k));
            xv[k] = settle<T>(x[k], a.cols, at(k));
            if constexpr (kAhead) dtv[k] = dt[k];
        }
        if constexpr (kAhead)
            if (r0 + step < a.rows) fetch_row(r0 + step);
        float first = 0.0f, second = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            // (past the row dy is 0)
            const Wide d = Vec<T>::widen(dyv[k]), h = (Vec<T>::widen(xv[k]) - mu) * rs;
            const Wide g = d * factor(k);
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) {
                first += g[j];
                second = __builtin_fmaf(g[j], h[j], second);
            }
            if (live) {
                dw[k] += d * h;
                db[k] += d;
            }
        }
        // dx may be an input: nothing is stored before every wave of the row
        // has loaded
        row_sum2<Waves>(first, second, firsts[set] + group * Waves, seconds[set] + group * Waves);
        first /= (float)a.cols;
        second /= (float)a.cols;
        if (!live) continue;
        T *const dx = static_cast<T *>(a.dx) + r * a.dx_stride;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const Wide h = (Vec<T>::widen(xv[k]) - mu) * rs;
            Wide g = rs * ((Vec<T>::widen(dyv[k]) * factor(k) - first) - h * second);
            if (a.dtotal) {
                const u32x4 v = kAhead ? dtv[kAhead ? k : 0]
                                       : load_vec<T, true, true>(static_cast<const T *>(a.dtotal) +
                                                                    r * a.dtotal_stride,
                                                                a.cols, at(k));
                g += Vec<T>::widen(settle<T>(v, a.cols, at(k)));
            }
            store_vec<T, true>(dx, a.cols, at(k), Vec<T>::narrow(g));
        }
    }
    if (!a.dweight && !a.dbias) return;
    if constexpr (Groups > 1) {
        const auto join = [&](Wide (&v)[V]) {
            for (uint32_t from = 1; from < Groups; ++from) {
                if (group == from)
#pragma unroll
                    for (int k = 0; k < V; ++k)
#pragma unroll
                        for (uint32_t j = 0; j < N; ++j) joined[(k * N + j) * kThreads + i] = v[k][j];
                __syncthreads();
                if (group == 0)
#pragma unroll
                    for (int k = 0; k < V; ++k)
#pragma unroll
                        for (uint32_t j = 0; j < N; ++j) v[k][j] += joined[(k * N + j) * kThreads + i];
                __syncthreads();
            }
        };
        join(dw);
        join(db);
    }
    if (group != 0) return;
    const bool only = gridDim.x == 1;      // the one part is the sum
    // the workspace is 16-byte aligned, a vector of sums of 16-bit data is 32 bytes
    typedef float Sums __attribute__((ext_vector_type(N), aligned(16)));
    float *const part = static_cast<float *>(a.workspace) + blockIdx.x * (2 * sums_pitch(a.cols));
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const uint32_t c = at(k);
        if (only) {
#pragma unroll
            for (uint32_t j = 0; j < N; ++j)
                if (c + j < a.cols) {
                    if (a.dweight) a.dweight[c + j] = dw[k][j];
                    if (a.dbias) a.dbias[c + j] = db[k][j];
                }
        } else if (c < a.cols) {
            *reinterpret_cast<Sums *>(part + c) = dw[k];
            *reinterpret_cast<Sums *>(part + sums_pitch(a.cols) + c) = db[k];
        }
    }
}

// dweight (blockIdx.y 0) and dbias (1) from the parts' sums: 32 columns a
// block, 32 threads a column.
constexpr uint32_t kSumCols = 32, kSumParts = 32;

__global__ void __launch_bounds__(kSumCols * kSumParts) ew_layernorm_sums_kernel(LayerNormGradArgs a,
                                                                                uint32_t parts)
{
    __shared__ float sums[kSumParts][kSumCols];
    float *const out = blockIdx.y ? a.dbias : a.dweight;
    if (!out) return;
    const uint64_t pitch = sums_pitch(a.cols);
    const float *const in = static_cast<const float *>(a.workspace) + blockIdx.y * pitch;
    const uint32_t col = threadIdx.x % kSumCols, p0 = threadIdx.x / kSumCols;
    for (uint64_t c0 = (uint64_t)blockIdx.x * kSumCols; c0 < a.cols; c0 += (uint64_t)gridDim.x * kSumCols) {
        const uint64_t c = c0 + col;
        float sum = 0.0f;
        if (c < a.cols)
            for (uint32_t p = p0; p < parts; p += kSumParts) sum += in[p * 2 * pitch + c];
        sums[p0][col] = sum;
        __syncthreads();
        if (p0 == 0 && c < a.cols) {
#pragma unroll
            for (uint32_t p = 1; p < kSumParts; ++p) sum += sums[p][col];
            out[c] = sum;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Gradient, longer rows: the parts' sums of dweight and dbias (a thread a
// vector of columns over a part of the rows), their sum, then dx (a block a
// row, two passes over it).  dx comes last: it may be dy or x.
// ---------------------------------------------------------------------------

constexpr uint32_t kColsBlock = 256;

template <typename T>
__global__ void __launch_bounds__(kColsBlock) ew_layernorm_cols_kernel(LayerNormGradArgs a,
                                                                      uint32_t parts)
{
    constexpr uint32_t N = Vec<T>::N;
    using Wide = typename Vec<T>::wide;
    const uint32_t at = (blockIdx.x * kColsBlock + threadIdx.x) * N;
    if (at >= a.cols) return;
    Wide dw(0.0f), db(0.0f);
    for (uint64_t r = blockIdx.y; r < a.rows; r += parts) {
        const u32x4 dy = load_vec<T, true>(static_cast<const T *>(a.dy) + r * a.dy_stride, a.cols, at);
        const u32x4 x = load_vec<T, true>(static_cast<const T *>(a.x) + r * a.x_stride, a.cols, at);
        const Wide d = Vec<T>::widen(settle<T>(dy, a.cols, at));
        dw += d * ((Vec<T>::widen(settle<T>(x, a.cols, at)) - a.mean[r]) * a.rstd[r]);
        db += d;
    }
    typedef float Sums __attribute__((ext_vector_type(N), aligned(16)));
    float *const part = static_cast<float *>(a.workspace) + blockIdx.y * (2 * sums_pitch(a.cols));
    *reinterpret_cast<Sums *>(part + at) = dw;
    *reinterpret_cast<Sums *>(part + sums_pitch(a.cols) + at) = db;
}

template <typename T>
__global__ void __launch_bounds__(kLongBlock) ew_layernorm_dx_kernel(LayerNormGradArgs a)
{
    constexpr uint32_t N = Vec<T>::N;
    using Wide = typename Vec<T>::wide;
    __shared__ float firsts[2][kLongWaves], seconds[2][kLongWaves];
    const T *const weight = static_cast<const T *>(a.weight);
    int set = 0;
    for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x, set ^= 1) {
        const T *const dy = static_cast<const T *>(a.dy) + r * a.dy_stride;
        const T *const x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *const dt =
            a.dtotal ? static_cast<const T *>(a.dtotal) + r * a.dtotal_stride : nullptr;
        T *const dx = static_cast<T *>(a.dx) + r * a.dx_stride;
        const float mu = a.mean[r], rs = a.rstd[r];
        const auto wide = [&](const T *p, uint32_t at) {
            return Vec<T>::widen(settle<T>(load_vec<T, false>(p, a.cols, at), a.cols, at));
        };
        const auto slope = [&](uint32_t at) {
            const Wide d = wide(dy, at);
            return weight ? d * wide(weight, at) : d;
        };
        float first = 0.0f, second = 0.0f;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
            const Wide g = slope(at), h = (wide(x, at) - mu) * rs;
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) {
                first += g[j];
                second = __builtin_fmaf(g[j], h[j], second);
            }
        }
        row_sum2<kLongWaves>(first, second, firsts[set], seconds[set]);
        first /= (float)a.cols;
        second /= (float)a.cols;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
            const Wide h = (wide(x, at) - mu) * rs;
            Wide g = rs * ((slope(at) - first) - h * second);
            if (dt) g += wide(dt, at);
            store_vec(dx, a.cols, at, Vec<T>::narrow(g));
        }
    }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

template <typename T>
static hipError_t layernorm_rows(const LayerNormArgs &a, uint32_t vectors, hipStream_t s)
{
#define EW_LAYERNORM_ROWS(W, V)                                                                  \
    if (vectors <= W * 64 * V)                                                                   \
        return start(reinterpret_cast<const void *>(&ew_layernorm_row_kernel<T, W, V>),          \
                     dim3(row_blocks(((uint64_t)a.rows * W * 64 + layernorm_block(W) - 1) /      \
                                     layernorm_block(W))),                                       \
                     layernorm_block(W), 0, s, a);
    EW_LAYERNORM_ROWS(1, 1)
    EW_LAYERNORM_ROWS(2, 1)
    EW_LAYERNORM_ROWS(3, 1)
    EW_LAYERNORM_ROWS(4, 1)
    EW_LAYERNORM_ROWS(5, 1)
    EW_LAYERNORM_ROWS(8, 1)
    EW_LAYERNORM_ROWS(8, 2)
    EW_LAYERNORM_ROWS(12, 2)
    EW_LAYERNORM_ROWS(16, 2)
    if constexpr (sizeof(T) == 4) {
        EW_LAYERNORM_ROWS(16, 4)
    } else {
        EW_LAYERNORM_ROWS(12, 4)
    }
#undef EW_LAYERNORM_ROWS
    return hipErrorInvalidValue;
}
static uint32_t register_vectors(RowType t) { return (t == kRowF32 ? 16 : 12) * 64 * 4; }

hipError_t launch_layernorm(RowType t, const LayerNormArgs &a, hipStream_t s, const char **path)
{
    const uint32_t vectors = vectors_of(t, a.cols);
    if (vectors <= register_vectors(t)) {
        *path = "rows in registers";
        return t == kRowF32   ? layernorm_rows<float>(a, vectors, s)
               : t == kRowF16 ? layernorm_rows<_Float16>(a, vectors, s)
                              : layernorm_rows<__bf16>(a, vectors, s);
    }
    *path = "three passes";
    return start(EW_KERNEL_OF(t, ew_layernorm_long_kernel), dim3(row_blocks(a.rows)), kLongBlock, 0, s, a);
}

size_t layernorm_grad_workspace(uint64_t rows, uint64_t cols)
{
    return (rows < kParts ? rows : kParts) * 2 * sums_pitch(cols) * sizeof(float);
}

// Up to this many rounds of rows are one block's, which writes dweight and
// dbias itself and saves the second launch.
constexpr uint64_t kOnePart = 2;

template <typename T>
static hipError_t layernorm_grad_rows(const LayerNormGradArgs &a, uint32_t vectors, hipStream_t s,
                                      uint32_t *parts)
{
#define EW_LAYERNORM_GRAD_ROWS(W, V)                                                              \
    if (vectors <= W * 64 * V) {                                                                  \
        constexpr int kGroups = W < 8 ? 8 / W : 1;                                                \
        const uint64_t blocks = ((uint64_t)a.rows + kGroups - 1) / kGroups;                       \
        *parts = blocks <= kOnePart ? 1 : (uint32_t)(blocks < kParts ? blocks : kParts);          \
        return start(reinterpret_cast<const void *>(&ew_layernorm_grad_kernel<T, W, V, kGroups>), \
                     dim3(*parts), W * 64 * kGroups, 0, s, a);                                    \
    }
    EW_LAYERNORM_GRAD_ROWS(1, 1)
    EW_LAYERNORM_GRAD_ROWS(2, 1)
    EW_LAYERNORM_GRAD_ROWS(4, 1)
    EW_LAYERNORM_GRAD_ROWS(8, 1)
    EW_LAYERNORM_GRAD_ROWS(8, 2)
    EW_LAYERNORM_GRAD_ROWS(8, 4)
    if constexpr (sizeof(T) == 4) {
        EW_LAYERNORM_GRAD_ROWS(12, 4)
    }
#undef EW_LAYERNORM_GRAD_ROWS
    return hipErrorInvalidValue;
}
static uint32_t grad_vectors(RowType t) { return t == kRowF32 ? 12 * 64 * 4 : 8 * 64 * 4; }

hipError_t launch_layernorm_grad(RowType t, const LayerNormGradArgs &a, hipStream_t s, const char **path)
{
    const bool sums = a.dweight || a.dbias;
    const auto sum = [&](uint32_t parts) {
        return start(reinterpret_cast<const void *>(&ew_layernorm_sums_kernel),
                     dim3(row_blocks(((uint64_t)a.cols + kSumCols - 1) / kSumCols), 2),
                     kSumCols * kSumParts, 0, s, a, parts);
    };
    if (a.rows == 0) return sum(0);
    const uint32_t vectors = vectors_of(t, a.cols);
    uint32_t parts = 0;
    if (vectors <= grad_vectors(t)) {
        *path = "rows in registers";
        const hipError_t e = t == kRowF32   ? layernorm_grad_rows<float>(a, vectors, s, &parts)
                             : t == kRowF16 ? layernorm_grad_rows<_Float16>(a, vectors, s, &parts)
                                            : layernorm_grad_rows<__bf16>(a, vectors, s, &parts);
        return e != hipSuccess || !sums || parts == 1 ? e : sum(parts);
    }
    *path = "two passes, dweight and dbias by columns";
    if (sums) {
        parts = a.rows < kParts ? a.rows : kParts;
        hipError_t e = start(EW_KERNEL_OF(t, ew_layernorm_cols_kernel),
                             dim3((vectors + kColsBlock - 1) / kColsBlock, parts), kColsBlock, 0, s, a, parts);
        if (e == hipSuccess) e = sum(parts);
        if (e != hipSuccess) return e;
    }
    return start(EW_KERNEL_OF(t, ew_layernorm_dx_kernel), dim3(row_blocks(a.rows)), kLongBlock, 0, s, a);
}

}  // namespace ew
