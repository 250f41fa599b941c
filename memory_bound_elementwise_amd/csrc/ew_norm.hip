// ew_norm.hip -- the RMS norm with the residual's addition (plain and e4m3
// output) and its gradient for CDNA4 (gfx950).

#include "ew_rows_device.h"

namespace ew {

constexpr int kNormBlock = 256;
constexpr int kNormWaves = kNormBlock / 64;
constexpr float kE4M3Max = 448.0f;
constexpr float kScaleMin = 0x1p-126f;

// y / scale for |y| <= 448 scale (up to a rounding error), as e4m3 sees it: the
// product with the rounded reciprocal and one correction by its residual.
// Before its rounding that is within 2^-22 of a last place of the quotient, so
// it could only round otherwise where the quotient lies that close to the
// middle of two binary32 numbers, and only matter where one of them lies
// halfway between two e4m3 values; in none of the mantissas for which both
// hold does it.  (The product alone puts 0.1-1.5 % of the bytes one step off,
// at ties; a division costs 3-8 % more time.)  Small scales are worked with 2^64
// times as large, so that the residual is exact; a scale of +inf (a norm that
// overflowed) divides finite y to 0.
struct Quotient {
    float up, over, inv;
    __device__ explicit Quotient(float scale)
    {
        up = scale < 1.0f ? 0x1p64f : 1.0f;
        over = scale * up;
        inv = 1.0f / over;
        over = over == kInf ? 0.0f : over;
    }
    __device__ float of(float y) const
    {
        const float u = y * up, q = u * inv;
        return __builtin_fmaf(-__builtin_fmaf(q, over, -u), inv, q);
    }
};

// e4m3 bits of x (|x| <= 448 up to a rounding error), nearest even.
__device__ __forceinline__ uint8_t to_e4m3(float x)
{
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xff);
}

// ---------------------------------------------------------------------------
// Forward, rows that fit in registers: Waves waves a row, V vectors a lane
// ---------------------------------------------------------------------------

// A row's vectors start at its start whatever its alignment, so that groups
// of columns fall on whole lanes; the last vector may be a part (its elements
// past the row are 0).
template <typename T>
__device__ __forceinline__ u32x4 load_part(const T *p, uint32_t n)
{
    typename Vec<T>::type t{};
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j)
        if ((uint32_t)j < n) t[j] = p[j];
    return __builtin_bit_cast(u32x4, t);
}

// The row's vectors of this thread (i, i + step, ...); Nt: a stream read
// once, else data that other rows read too.
template <typename T, int V, bool Nt>
__device__ __forceinline__ void load_row(u32x4 (&v)[V], const T *row, uint32_t cols, uint32_t i,
                                         uint32_t step)
{
    constexpr uint32_t N = Vec<T>::N;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const uint32_t at = (i + k * step) * N;
        v[k] = u32x4{0, 0, 0, 0};
        if (at + N <= cols) {
            if constexpr (Nt) {
                v[k] = load16<false, sizeof(T)>(reinterpret_cast<const char *>(row + at));
            } else if constexpr (sizeof(T) == 4) {
                v[k] = *reinterpret_cast<const u32x4_a4 *>(row + at);
            } else {
                v[k] = *reinterpret_cast<const u32x4_a2 *>(row + at);
            }
        }
    }
    if (cols % N) {        // one lane holds the last, partial vector
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint32_t at = (i + k * step) * N;
            if (at < cols && at + N > cols) v[k] = load_part(row + at, cols - at);
        }
    }
}

template <typename T>
__device__ __forceinline__ void store_vec(T *row, uint32_t cols, uint32_t at, u32x4 v)
{
    constexpr uint32_t N = Vec<T>::N;
    if (at + N <= cols) {
        store16_row<T>(reinterpret_cast<char *>(row + at), v);
    } else if (at < cols) {
        const typename Vec<T>::type t = __builtin_bit_cast(typename Vec<T>::type, v);
#pragma unroll
        for (uint32_t j = 0; j < N; ++j)
            if (at + j < cols) row[at + j] = t[j];
    }
}

// R over a row's Waves waves, in all of them.  scratch: Waves floats of the
// row's own.
template <class R, int Waves>
__device__ __forceinline__ float row_reduce(float x, float *scratch)
{
    x = wave_reduce<R>(x);
    if constexpr (Waves > 1) {
        if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64 % Waves] = x;
        __syncthreads();
        x = scratch[0];
#pragma unroll
        for (int w = 1; w < Waves; ++w) x = R::f(x, scratch[w]);
    }
    return x;
}

// The largest |y| (a NaN if one is) over `lanes` neighbouring lanes, a power
// of two, in each of them.
__device__ __forceinline__ float lanes_max(float x, uint32_t lanes)
{
    if (lanes > 1) x = max_or_nan(x, dpp<0xB1>(x));
    if (lanes > 2) x = max_or_nan(x, dpp<0x4E>(x));
    if (lanes > 4) x = max_or_nan(x, dpp<0x141>(x));
    if (lanes > 8) x = max_or_nan(x, dpp<0x140>(x));
    if (lanes > 16) x = max_or_nan(x, __shfl_xor(x, 16));
    if (lanes > 32) x = max_or_nan(x, __shfl_xor(x, 32));
    return x;
}

// Eight (four) e4m3 bytes of a vector's quotients by scale.
template <typename T>
__device__ __forceinline__ void store_e4m3(uint8_t *row, uint32_t cols, uint32_t at,
                                           typename Vec<T>::wide y, const Quotient &by)
{
    constexpr uint32_t N = Vec<T>::N;
    uint32_t w[N / 4];
#pragma unroll
    for (uint32_t k = 0; k < N / 4; ++k) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(by.of(y[4 * k]), by.of(y[4 * k + 1]), 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(by.of(y[4 * k + 2]), by.of(y[4 * k + 3]), p, true);
        w[k] = (uint32_t)p;
    }
    typedef uint32_t word __attribute__((aligned(1)));
    if (at + N <= cols) {
        if constexpr (N == 8) {
            typedef uint32_t words __attribute__((ext_vector_type(2), aligned(1)));
            __builtin_nontemporal_store(words{w[0], w[1]}, reinterpret_cast<words *>(row + at));
        } else {
            __builtin_nontemporal_store(w[0], reinterpret_cast<word *>(row + at));
        }
    } else {
#pragma unroll
        for (uint32_t j = 0; j < N; ++j)
            if (at + j < cols) row[at + j] = (uint8_t)(w[j / 4] >> j % 4 * 8);
    }
}

// Threads of a block: a row's waves, or four waves of short rows.
constexpr int norm_block(int waves) { return waves < 3 ? 256 : waves * 64; }

// total = round(x + residual), y = total * rstd * weight in one pass: the row's
// vectors stay in registers between the sum of squares and the product, and
// the sum costs one barrier.  Bound by memory: 8192 x 4096 bf16 with residual
// and total 42.5 us, 6.3 TB/s (a copy of 2^28 floats: 6.64); e4m3, 4096 x 8192
// bf16 41-42 us, 5.6-5.8 TB/s (8-byte stores; the vector unit is busy 72 %).  A
// row whose columns fill no whole vectors is bound by latency: the last
// vector's elements are loaded one after another while the block waits, and
// the weight, x and the residual are waited for in turn (1021 x 5003 f32 17.8
// us, 4.6 TB/s; 8192 x 4097 bf16 65).  One row of 4096 2.4 us on the GPU.
template <typename T, int Waves, int V, bool E4M3>
__global__ void __launch_bounds__(norm_block(Waves)) ew_norm_row_kernel(NormArgs a)
{
    constexpr uint32_t N = Vec<T>::N, kThreads = Waves * 64;
    constexpr uint32_t kRows = norm_block(Waves) / kThreads;
    using Wide = typename Vec<T>::wide;
    // two sets, used in turn: a wave is at most one barrier ahead of another
    __shared__ float sums[2][norm_block(Waves) / 64], tops[2][norm_block(Waves) / 64];
    const uint32_t group = threadIdx.x / kThreads, i = threadIdx.x % kThreads;
    u32x4 w[V];
    load_row<T, V, false>(w, static_cast<const T *>(a.weight), a.cols, i, kThreads);
    int set = 0;
    // a block's rows go round together (the barriers)
    for (uint64_t r0 = (uint64_t)blockIdx.x * kRows; r0 < a.rows;
         r0 += (uint64_t)gridDim.x * kRows, set ^= 1) {
        const bool live = r0 + group < a.rows;
        const uint64_t r = live ? r0 + group : r0;
        u32x4 h[V];
        load_row<T, V, true>(h, static_cast<const T *>(a.x) + r * a.x_stride, a.cols, i, kThreads);
        if (a.residual) {
            u32x4 res[V];
            load_row<T, V, true>(res, static_cast<const T *>(a.residual) + r * a.residual_stride,
                                 a.cols, i, kThreads);
#pragma unroll
            for (int k = 0; k < V; ++k)
                h[k] = Vec<T>::narrow(Vec<T>::widen(h[k]) + Vec<T>::widen(res[k]));
        }
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const Wide f = Vec<T>::widen(h[k]);
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) sum = __builtin_fmaf(f[j], f[j], sum);
        }
        // the outputs may be the inputs: nothing is stored before every wave
        // of the row has loaded (a row of one wave loads before it stores)
        sum = row_reduce<Sum, Waves>(sum, sums[set] + group * Waves);
        const float rstd = 1.0f / __builtin_sqrtf(sum / (float)a.cols + a.eps);
        if (live && a.rstd && i == 0) a.rstd[r] = rstd;
        if (live && a.total) {
            T *const total = static_cast<T *>(a.total) + r * a.total_stride;
#pragma unroll
            for (int k = 0; k < V; ++k) store_vec(total, a.cols, (i + k * kThreads) * N, h[k]);
        }
        if constexpr (!E4M3) {
            T *const y = static_cast<T *>(a.y) + r * a.y_stride;
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (live)
                    store_vec(y, a.cols, (i + k * kThreads) * N,
                              Vec<T>::narrow(Vec<T>::widen(h[k]) * rstd * Vec<T>::widen(w[k])));
        } else {
            uint8_t *const q = static_cast<uint8_t *>(a.y) + r * a.y_stride;
            float *const scales = a.scales + r * a.groups;
            Wide y[V];
            float top[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                y[k] = Vec<T>::widen(h[k]) * rstd * Vec<T>::widen(w[k]);
                top[k] = 0.0f;
#pragma unroll
                for (uint32_t j = 0; j < N; ++j)
                    top[k] = max_or_nan(top[k], __builtin_fabsf(y[k][j]));
            }
            if (a.groups == 1) {
                float all = top[0];
#pragma unroll
                for (int k = 1; k < V; ++k) all = max_or_nan(all, top[k]);
                all = row_reduce<MaxOrNan, Waves>(all, tops[set] + group * Waves);
                const float scale = max_or_nan(all / kE4M3Max, kScaleMin);
                const Quotient by(scale);
                if (live && i == 0) scales[0] = scale;
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (live) store_e4m3<T>(q, a.cols, (i + k * kThreads) * N, y[k], by);
            } else {
                // a group is a power of two of neighbouring lanes of a wave
                const uint32_t lanes = a.group / N;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const uint32_t at = (i + k * kThreads) * N;
                    const float most = lanes_max(top[k], lanes);
                    const float scale = max_or_nan(most / kE4M3Max, kScaleMin);
                    if (live && at < a.cols) {
                        if (i % lanes == 0) scales[at / a.group] = scale;
                        store_e4m3<T>(q, a.cols, at, y[k], Quotient(scale));
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Forward, longer rows: one block a row, two passes over it
// ---------------------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(kNormBlock) ew_norm_kernel(NormArgs a)
{
    __shared__ float scratch[2][kNormWaves];
    const T *const w = static_cast<const T *>(a.weight);
    int flip = 0;
    for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x, flip ^= 1) {
        const T *const x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *const res =
            a.residual ? static_cast<const T *>(a.residual) + r * a.residual_stride : nullptr;
        T *const total = a.total ? static_cast<T *>(a.total) + r * a.total_stride : nullptr;
        const auto value = [&](uint32_t c) -> T {
            return res ? (T)((float)x[c] + (float)res[c]) : x[c];
        };
        float sum = 0.0f;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kNormBlock) {
            const T h = value(c);
            sum += (float)h * (float)h;
            if (total) total[c] = h;
        }
        sum = block_reduce<Sum, kNormWaves>(sum, scratch[flip]);
        const float rstd = 1.0f / __builtin_sqrtf(sum / (float)a.cols + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
        // the first pass stored total where this thread reads it back (total
        // may be x or residual)
        const auto out = [&](uint32_t c) -> float {
            const T h = total ? total[c] : value(c);
            return (float)h * rstd * (float)w[c];
        };
        if (!a.scales) {
            T *const y = static_cast<T *>(a.y) + r * a.y_stride;
            for (uint32_t c = threadIdx.x; c < a.cols; c += kNormBlock) y[c] = (T)out(c);
            continue;
        }
        __syncthreads();      // a group's columns were stored by other threads
        uint8_t *const q = static_cast<uint8_t *>(a.y) + r * a.y_stride;
        const uint32_t lane = threadIdx.x % 64;
        for (uint32_t g = threadIdx.x / 64; g < a.groups; g += kNormWaves) {
            const uint32_t lo = g * a.group;
            const uint32_t hi = a.cols - lo < a.group ? a.cols : lo + a.group;
            float top = 0.0f;
            for (uint32_t c = lo + lane; c < hi; c += 64)
                top = max_or_nan(top, __builtin_fabsf(out(c)));
#pragma unroll
            for (int d = 1; d < 64; d *= 2) top = max_or_nan(top, __shfl_xor(top, d));
            const float scale = max_or_nan(top / kE4M3Max, kScaleMin);
            const Quotient by(scale);
            if (lane == 0) a.scales[(uint64_t)r * a.groups + g] = scale;
            for (uint32_t c = lo + lane; c < hi; c += 64) q[c] = to_e4m3(by.of(out(c)));
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

// dweight is added up in two steps: at most this many blocks sum a part of
// the rows each, then the parts are summed.  One block a CU: each part costs a
// row of sums written and read (8192 x 4096 bf16: 256 parts 50 us in all, 512
// 55 us).
constexpr uint32_t kGradParts = 256;

// Floats from one part's sums to the next: whole vectors of sums.
__host__ __device__ constexpr uint64_t part_pitch(uint64_t cols) { return (cols + 7) & ~(uint64_t)7; }

// Rows that fit in registers: Waves waves a row, V vectors a lane, Groups rows
// at a time in a block, which adds up dweight over its rows.  Bound by memory:
// 8192 x 4096 bf16 45 us, 6.0 TB/s, and 4.7 us for the sum of the parts;
// without the next row's loads ahead 51 us.

template <typename T, int Waves, int V, int Groups>
__global__ void __launch_bounds__(Waves * 64 * Groups) ew_norm_grad_kernel(NormGradArgs a)
{
    constexpr uint32_t N = Vec<T>::N, kThreads = Waves * 64;
    using Wide = typename Vec<T>::wide;
    __shared__ float sums[2][Waves * Groups];
    __shared__ float joined[Groups > 1 ? kThreads * V * N : 1];
    const uint32_t group = threadIdx.x / kThreads, i = threadIdx.x % kThreads;
    // the next row is on its way while this one is worked on, and the weight
    // stays, unless they would not fit in registers
    constexpr bool kAhead = V < 4;
    u32x4 wv[V];
    const auto fetch_weight = [&] {
        load_row<T, V, false>(wv, static_cast<const T *>(a.weight), a.cols, i, kThreads);
    };
    if constexpr (kAhead) fetch_weight();
    Wide dw[V];
#pragma unroll
    for (int k = 0; k < V; ++k) dw[k] = Wide(0.0f);
    u32x4 dy[V], x[V], dt[V];
    float rstd = 0.0f;
    const auto fetch = [&](uint64_t r0) {
        const uint64_t r = r0 + group < a.rows ? r0 + group : r0;
        load_row<T, V, true>(dy, static_cast<const T *>(a.dy) + r * a.dy_stride, a.cols, i, kThreads);
        load_row<T, V, true>(x, static_cast<const T *>(a.x) + r * a.x_stride, a.cols, i, kThreads);
        if (kAhead && a.dtotal)
            load_row<T, V, true>(dt, static_cast<const T *>(a.dtotal) + r * a.dtotal_stride, a.cols,
                                 i, kThreads);
        rstd = a.rstd[r];
    };
    uint64_t r0 = (uint64_t)blockIdx.x * Groups;
    const uint64_t step = (uint64_t)gridDim.x * Groups;
    if (kAhead && r0 < a.rows) fetch(r0);
    for (int set = 0; r0 < a.rows; r0 += step, set ^= 1) {
        const bool live = r0 + group < a.rows;
        if constexpr (!kAhead) {
            fetch(r0);
            fetch_weight();
        }
        const float rs = rstd;
        u32x4 dyv[V], xv[V], dtv[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dyv[k] = dy[k];
            xv[k] = x[k];
            dtv[k] = dt[k];
        }
        if (kAhead && r0 + step < a.rows) fetch(r0 + step);
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const Wide d = Vec<T>::widen(dyv[k]), h = Vec<T>::widen(xv[k]), w = Vec<T>::widen(wv[k]);
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) dot = __builtin_fmaf(h[j], d[j] * w[j], dot);
            if (live) dw[k] += d * (h * rs);
        }
        // dx may be an input: nothing is stored before every wave of the row
        // has loaded
        dot = row_reduce<Sum, Waves>(dot, sums[set] + group * Waves);
        const float c = dot / (float)a.cols * rs * rs * rs;
        const uint64_t r = live ? r0 + group : r0;
        if constexpr (!kAhead) fetch_weight();
        if (!kAhead && a.dtotal)
            load_row<T, V, true>(dtv, static_cast<const T *>(a.dtotal) + r * a.dtotal_stride, a.cols,
                                 i, kThreads);
        T *const dx = static_cast<T *>(a.dx) + r * a.dx_stride;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Wide g = rs * (Vec<T>::widen(dyv[k]) * Vec<T>::widen(wv[k])) - c * Vec<T>::widen(xv[k]);
            if (a.dtotal) g += Vec<T>::widen(dtv[k]);
            if (live) store_vec(dx, a.cols, (i + k * kThreads) * N, Vec<T>::narrow(g));
        }
    }
    if (!a.dweight) return;
    if constexpr (Groups > 1) {
        for (uint32_t from = 1; from < Groups; ++from) {
            if (group == from)
#pragma unroll
                for (int k = 0; k < V; ++k)
#pragma unroll
                    for (uint32_t j = 0; j < N; ++j)
                        joined[(k * N + j) * kThreads + i] = dw[k][j];
            __syncthreads();
            if (group == 0)
#pragma unroll
                for (int k = 0; k < V; ++k)
#pragma unroll
                    for (uint32_t j = 0; j < N; ++j)
                        dw[k][j] += joined[(k * N + j) * kThreads + i];
            __syncthreads();
        }
    }
    if (group != 0) return;
    const bool only = gridDim.x == 1;      // the one part is the sum
    // the workspace is 16-byte aligned, a vector of sums of 16-bit data is 32 bytes
    typedef float Sums __attribute__((ext_vector_type(N), aligned(16)));
    float *const part = a.partial + blockIdx.x * part_pitch(a.cols);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const uint32_t c = (i + k * kThreads) * N;
        if (only) {
#pragma unroll
            for (uint32_t j = 0; j < N; ++j)
                if (c + j < a.cols) a.dweight[c + j] = dw[k][j];
        } else if (c < a.cols) {
            *reinterpret_cast<Sums *>(part + c) = dw[k];
        }
    }
}

// dweight from the blocks' sums: 32 columns a block, 32 threads a column.
constexpr uint32_t kSumCols = 32, kSumParts = 32;

__global__ void __launch_bounds__(kSumCols * kSumParts) ew_norm_dweight_sum_kernel(NormGradArgs a,
                                                                                  uint32_t parts)
{
    __shared__ float sums[kSumParts][kSumCols];
    const uint32_t col = threadIdx.x % kSumCols, p0 = threadIdx.x / kSumCols;
    for (uint64_t c0 = (uint64_t)blockIdx.x * kSumCols; c0 < a.cols; c0 += (uint64_t)gridDim.x * kSumCols) {
        const uint64_t c = c0 + col;
        float sum = 0.0f;
        if (c < a.cols)
            for (uint32_t p = p0; p < parts; p += kSumParts) sum += a.partial[p * part_pitch(a.cols) + c];
        sums[p0][col] = sum;
        __syncthreads();
        if (p0 == 0 && c < a.cols) {
#pragma unroll
            for (uint32_t p = 1; p < kSumParts; ++p) sum += sums[p][col];
            a.dweight[c] = sum;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Gradient, longer rows: dweight's partial sums (a thread a column over a
// part of the rows), their sum, then dx (one block a row, two passes over
// it).  dx comes last: it may be dy or x.
// ---------------------------------------------------------------------------


template <typename T>
__global__ void __launch_bounds__(kNormBlock) ew_norm_dweight_kernel(NormGradArgs a, uint32_t parts)
{
    const uint32_t c = blockIdx.x * kNormBlock + threadIdx.x;
    if (c >= a.cols) return;
    const T *const dy = static_cast<const T *>(a.dy) + c, *const x = static_cast<const T *>(a.x) + c;
    float sum = 0.0f;
    for (uint32_t r = blockIdx.y; r < a.rows; r += parts)
        sum += (float)dy[r * a.dy_stride] * ((float)x[r * a.x_stride] * a.rstd[r]);
    a.partial[blockIdx.y * part_pitch(a.cols) + c] = sum;
}

template <typename T>
__global__ void __launch_bounds__(kNormBlock) ew_norm_dx_kernel(NormGradArgs a)
{
    __shared__ float scratch[2][kNormWaves];
    const T *const w = static_cast<const T *>(a.weight);
    int flip = 0;
    for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x, flip ^= 1) {
        const T *const dy = static_cast<const T *>(a.dy) + r * a.dy_stride;
        const T *const x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *const dt =
            a.dtotal ? static_cast<const T *>(a.dtotal) + r * a.dtotal_stride : nullptr;
        T *const dx = static_cast<T *>(a.dx) + r * a.dx_stride;
        float dot = 0.0f;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kNormBlock)
            dot += (float)x[c] * ((float)dy[c] * (float)w[c]);
        dot = block_reduce<Sum, kNormWaves>(dot, scratch[flip]);
        const float rstd = a.rstd[r], k = dot / (float)a.cols * rstd * rstd * rstd;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kNormBlock) {
            float g = rstd * ((float)dy[c] * (float)w[c]) - k * (float)x[c];
            if (dt) g += (float)dt[c];
            dx[c] = (T)g;
        }
    }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

size_t norm_grad_workspace(uint64_t rows, uint64_t cols)
{
    return (rows < kGradParts ? rows : kGradParts) * part_pitch(cols) * sizeof(float);
}

// Blocks stride over what is beyond this many (2^30 threads at most).
constexpr uint64_t kMaxGrid = 1 << 20;

template <class... A>
static hipError_t go(const void *fn, dim3 grid, int block, hipStream_t s, A... args)
{
    void *kargs[] = {&args...};
    return hipLaunchKernel(fn, grid, dim3(block), kargs, 0, s);
}

static uint32_t row_grid(uint64_t blocks) { return (uint32_t)(blocks < kMaxGrid ? blocks : kMaxGrid); }

static uint32_t row_vectors(RowType t, uint32_t cols)
{
    const uint32_t n = 16 / (uint32_t)row_elem_size(t);
    return (cols + n - 1) / n;
}

#define EW_BY_TYPE(t, K)                                           \
    ((t) == kRowF32 ? reinterpret_cast<const void *>(&K<float>)    \
     : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16>) \
                      : reinterpret_cast<const void *>(&K<__bf16>))

// One row a block (four of one wave each), the next row another block: on
// 2^25 elements of rows of 64 to 512 vectors one vector a lane took 44-46 us
// and blocks that stride over rows 45-52; two or four vectors a lane 46-54.
// Beyond 512 vectors rows of 16 waves leave a CU with one or two blocks that
// all load or all store: eight waves of two vectors took 46.6 us on rows of
// 1024 vectors, sixteen of one 49-67.  For the longest rows sixteen waves win
// (2048 vectors: 50 us as eight of four; 16 rows: 4.6 us against 5.5).  Three
// waves, five, and ten and twelve of two vectors are there because rows just
// past a power of two leave a larger block's lanes idle (e4m3, 1536 vectors of
// bf16: 46 us with twelve, 54 with sixteen; 300 of f32: 44 with five, 53 with
// eight); six, seven and fourteen gained nothing or lost up to 18 %, and plain
// 32-bit rows of 1251 and 1536 vectors lost 3-8 % to ten and twelve.
template <typename T, bool E4M3>
static hipError_t norm_rows(const NormArgs &a, uint32_t vectors, hipStream_t s)
{
#define EW_NORM_ROWS(W, V)                                                                       \
    if (vectors <= W * 64 * V)                                                                   \
        return go(reinterpret_cast<const void *>(&ew_norm_row_kernel<T, W, V, E4M3>),            \
                  dim3(row_grid(((uint64_t)a.rows * W * 64 + norm_block(W) - 1) / norm_block(W))), \
                  norm_block(W), s, a);
    EW_NORM_ROWS(1, 1)
    EW_NORM_ROWS(2, 1)
    EW_NORM_ROWS(3, 1)
    EW_NORM_ROWS(4, 1)
    EW_NORM_ROWS(5, 1)
    EW_NORM_ROWS(8, 1)
    EW_NORM_ROWS(8, 2)
    if constexpr (E4M3 || sizeof(T) == 2) {
        EW_NORM_ROWS(10, 2)
        EW_NORM_ROWS(12, 2)
    }
    EW_NORM_ROWS(16, 2)
    EW_NORM_ROWS(16, 4)
#undef EW_NORM_ROWS
    return hipErrorInvalidValue;
}
constexpr uint32_t kNormVectors = 16 * 64 * 4;       // the longest row it takes

hipError_t launch_norm(RowType t, const NormArgs &a, hipStream_t s, const char **path)
{
    const uint32_t vectors = row_vectors(t, a.cols);
    if (vectors <= kNormVectors) {
        *path = "rows in registers";
        switch (t) {
        case kRowF32:
            return a.scales ? norm_rows<float, true>(a, vectors, s) : norm_rows<float, false>(a, vectors, s);
        case kRowF16:
            return a.scales ? norm_rows<_Float16, true>(a, vectors, s)
                            : norm_rows<_Float16, false>(a, vectors, s);
        default:
            return a.scales ? norm_rows<__bf16, true>(a, vectors, s)
                            : norm_rows<__bf16, false>(a, vectors, s);
        }
    }
    *path = "two passes";
    return go(EW_BY_TYPE(t, ew_norm_kernel), dim3(row_grid(a.rows)), kNormBlock, s, a);
}

// The gradient's rows: one vector a lane as long as they fit, eight waves a
// block or a row's (1024 vectors of bf16: sixteen waves of one vector 52.5 us,
// eight of two 53.7).  Two vectors of 16-bit data a lane are what the 128
// registers of sixteen waves hold; of 32-bit data, whose sums take half as
// many, four.
//
// Up to two rounds of rows are one block's, which writes dweight itself and
// saves the second launch (3.6 us of the host's): on the GPU 1 row of 4096 bf16
// 4.4 us instead of 5.1, 2 rows 5.2 either way; of four rounds 7.0 against 5.2.
constexpr uint64_t kOnePart = 2;
template <typename T>
static hipError_t norm_grad_rows(const NormGradArgs &a, uint32_t vectors, hipStream_t s, uint32_t *parts)
{
#define EW_NORM_GRAD_ROWS(W, V)                                                                   \
    if (vectors <= W * 64 * V) {                                                                  \
        constexpr int kGroups = W < 8 ? 8 / W : 1;                                                \
        const uint64_t blocks = ((uint64_t)a.rows + kGroups - 1) / kGroups;                       \
        *parts = blocks <= kOnePart ? 1 : (uint32_t)(blocks < kGradParts ? blocks : kGradParts);  \
        return go(reinterpret_cast<const void *>(&ew_norm_grad_kernel<T, W, V, kGroups>),         \
                  dim3(*parts), W * 64 * kGroups, s, a);                                          \
    }
    EW_NORM_GRAD_ROWS(1, 1)
    EW_NORM_GRAD_ROWS(2, 1)
    EW_NORM_GRAD_ROWS(4, 1)
    EW_NORM_GRAD_ROWS(8, 1)
    EW_NORM_GRAD_ROWS(16, 1)
    EW_NORM_GRAD_ROWS(16, 2)
    if constexpr (sizeof(T) == 4) {
        EW_NORM_GRAD_ROWS(16, 4)
    }
#undef EW_NORM_GRAD_ROWS
    return hipErrorInvalidValue;
}
static uint32_t grad_vectors(RowType t) { return t == kRowF32 ? 16 * 64 * 4 : 16 * 64 * 2; }

hipError_t launch_norm_grad(RowType t, const NormGradArgs &a, hipStream_t s, const char **path)
{
    const auto sum = [&](uint32_t parts) {
        return go(reinterpret_cast<const void *>(&ew_norm_dweight_sum_kernel),
                  dim3(row_grid(((uint64_t)a.cols + kSumCols - 1) / kSumCols)), kSumCols * kSumParts, s, a,
                  parts);
    };
    if (a.rows == 0) return sum(0);
    const uint32_t vectors = row_vectors(t, a.cols);
    uint32_t parts = 0;
    if (vectors <= grad_vectors(t)) {
        *path = "rows in registers";
        const hipError_t e = t == kRowF32   ? norm_grad_rows<float>(a, vectors, s, &parts)
                             : t == kRowF16 ? norm_grad_rows<_Float16>(a, vectors, s, &parts)
                                            : norm_grad_rows<__bf16>(a, vectors, s, &parts);
        return e != hipSuccess || !a.dweight || parts == 1 ? e : sum(parts);
    }
    *path = "two passes, dweight by columns";
    if (a.dweight) {
        parts = a.rows < kGradParts ? a.rows : kGradParts;
        hipError_t e = go(EW_BY_TYPE(t, ew_norm_dweight_kernel),
                          dim3((a.cols + kNormBlock - 1) / kNormBlock, parts), kNormBlock, s, a, parts);
        if (e == hipSuccess) e = sum(parts);
        if (e != hipSuccess) return e;
    }
    return go(EW_BY_TYPE(t, ew_norm_dx_kernel), dim3(row_grid(a.rows)), kNormBlock, s, a);
}

}  // namespace ew
