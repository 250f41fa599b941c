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
    __device__ Mean() {}
    __device__ explicit Mean(double m) : hi((float)m), lo((float)(m - (double)(float)m)) {}
};

// sum / n, by = 1 / n: exact where the quotient is a binary64 number (a row of
// equal values), without the steps of a division.
__device__ __forceinline__ double divide(double sum, uint32_t n, double by)
{
    const double q = sum * by;
    return __builtin_fma(__builtin_fma(-q, (double)n, sum), by, q);
}

// Sum of one value a wave (x in lanes w, w + Waves, ...) in all lanes: of a
// power of two of them by lane exchanges.
template <int Waves>
__device__ __forceinline__ double sum_of_waves(double x)
{
    if constexpr (Waves > 1) x += dpp64<0xB1>(x);
    if constexpr (Waves > 2) x += dpp64<0x4E>(x);
    if constexpr (Waves > 4) x += dpp64<0x141>(x);
    if constexpr (Waves > 8) x += dpp64<0x140>(x);
    return x;
}
template <int Waves>
__device__ __forceinline__ float sum_of_waves(float x)
{
    if constexpr (Waves > 1) x += dpp<0xB1>(x);
    if constexpr (Waves > 2) x += dpp<0x4E>(x);
    if constexpr (Waves > 4) x += dpp<0x141>(x);
    if constexpr (Waves > 8) x += dpp<0x140>(x);
    return x;
}
// Lanes that hold the values of so many waves: the power of two above.
constexpr uint32_t lanes_of_waves(int waves) { return waves > 8 ? 16 : waves > 4 ? 8 : waves > 2 ? 4 : waves; }

// What a wave knows of its elements of a row: a number near them, and the sums
// of the differences from it and of their squares.  Where binary32 does not hold
// these, the sums are of differences times 2^-up.
struct WaveSums {
    float near, sum, squares;
    int up;
};

// The power of two by which differences are multiplied so that binary32 holds
// the sum of their squares: 0, or another where that is past its range, as that
// of numbers above 2^50 may be, or below it and eps does not cover it.  (Numbers
// within 2^-30 of one above 1 are equal to it.)
constexpr int kShift = 80;
__device__ __forceinline__ int shift_for(float squares, float eps, float near)
{
    const float least = eps < 0x1p-60f ? 0x1p-60f : -1.0f;
    if (squares < 0x1p100f && squares >= least) return 0;
    return !(squares < 1.0f) ? -kShift : __builtin_fabsf(near) <= 1.0f ? kShift : 0;
}

// The number is the mean of the wave's first vector (of equal values: exactly
// theirs, so that their differences are 0).  Where it lies so far from the
// wave's mean that the squares about it are more than four times those about
// the mean, two bits, the wave sums again from its mean: neither an outlier nor
// the distance of the row from 0 costs more.  Where binary32 loses the squares,
// it sums again with differences times a power of two.
template <typename T, int V, RowFit Fit, class At>
__device__ __forceinline__ WaveSums wave_sums(const u32x4 (&h)[V], uint32_t cols, uint32_t n, float eps,
                                              At piece)
{
    constexpr uint32_t N = Vec<T>::N;
    using Wide = typename Vec<T>::wide;
    const auto about = [&](float near, float scale, int up) {
        WaveSums w{near, 0.0f, 0.0f, up};
        const float at = near * scale;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Wide d = Vec<T>::widen(h[k]);
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) d[j] = __builtin_fmaf(d[j], scale, -at);
            if (Fit == kTiny || (Fit == kPart && n < V * 64 * N)) {     // the same in all lanes
                const Piece<T, Fit> p = piece(k);
#pragma unroll
                for (uint32_t j = 0; j < N; ++j)
                    if (!p.live || !p.own(j, cols)) d[j] = 0.0f;
            }
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) {
                w.sum += d[j];
                w.squares = __builtin_fmaf(d[j], d[j], w.squares);
            }
        }
        w.sum = wave_reduce<Sum>(w.sum);
        w.squares = wave_reduce<Sum>(w.squares);
        return w;
    };
    const auto off_centre = [&](const WaveSums &w) { return w.sum * w.sum > 0.75f * (float)n * w.squares; };
    const Wide f = Vec<T>::widen(h[0]) * (1.0f / N);
    float first = (f[0] + f[1]) + (f[2] + f[3]);
    if constexpr (N == 8) first += (f[4] + f[5]) + (f[6] + f[7]);
    if constexpr (Fit == kTiny) first = Vec<T>::widen(h[0])[0];
    WaveSums w = about(lane_value(first, 0), 1.0f, 0);
    const int shift = shift_for(w.squares, eps, w.near);
    // (what decides on other turns is the same in all lanes)
    if (shift != 0 || off_centre(w)) {
        for (bool more = true; more;) {
            more = w.up != -shift;
            // (without the difference by itself, which may be past binary32)
            if (!more) w.near = __builtin_fmaf(w.sum / (float)n, __builtin_ldexpf(1.0f, w.up), w.near);
            w = about(w.near, __builtin_ldexpf(1.0f, shift), -shift);
            more = more && off_centre(w);
        }
    }
    return w;
}

// The sum of a wave's n elements, and the squares about the row's mean times
// 2^(2 shift).
__device__ __forceinline__ double sum_of(const WaveSums &w, uint32_t n)
{
    return __builtin_fma((double)w.near, (double)n, __builtin_ldexp((double)w.sum, w.up));
}
__device__ __forceinline__ float squares_about(const WaveSums &w, uint32_t n, double mean, int shift)
{
    const float off = (float)__builtin_ldexp((double)w.near - mean, shift);
    return __builtin_fmaf(off, __builtin_fmaf(off, (float)n, __builtin_ldexpf(w.sum, w.up + shift + 1)),
                          __builtin_ldexpf(w.squares, 2 * (w.up + shift)));
}

// 1 / sqrt(squares / n + eps), by = 1 / n, through the hardware's reciprocal
// root (off by a last place), which wants no subnormal.
__device__ __forceinline__ float reciprocal_root(float squares, float by, float eps)
{
    squares = squares < 0.0f ? 0.0f : squares;       // (a rounding below 0)
    const float v = __builtin_fmaf(squares, by, eps);
    const bool small = v < 0x1p-100f;
    const float root = __builtin_amdgcn_rsqf(small ? v * 0x1p100f : v);
    return small ? root * 0x1p50f : root;
}

// How a row is normed: differences from the mean times scale, a power of two
// that keeps them inside binary32 and is 1 for all but rows that shift_for()
// names, times root.
struct Place {
    Mean mean;          // times scale
    float root, scale;
    __device__ Place() {}
    // squares: of differences times 2^shift
    __device__ Place(double mean_, float squares, float by, float eps, int shift)
    {
        const float s = __builtin_ldexpf(1.0f, shift);
        root = reciprocal_root(squares, by, eps * s * s);
        // equal numbers, whose mean may be any, are not shifted up; others that
        // close are close to 0
        const bool equal = shift > 0 && !(squares > 0.0f);
        if (equal) root *= s;
        scale = equal ? 1.0f : s;
        mean = Mean(mean_ * (double)scale);
    }
    __device__ float rstd() const { return root * scale; }
    // The same in all of a wave: in scalar registers, which leave room for a
    // wave more a SIMD.  (A vector instruction takes one.)
    __device__ void to_scalars()
    {
        mean.lo = lane_value(mean.lo, 0);
        root = lane_value(root, 0);
        scale = lane_value(scale, 0);
    }
};

template <typename T>
__device__ __forceinline__ u32x4 normed(u32x4 v, const Place &p, typename Vec<T>::wide w,
                                        typename Vec<T>::wide b)
{
    typename Vec<T>::wide y = Vec<T>::widen(v);
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) {
        const float off = __builtin_fmaf(y[j], p.scale, -p.mean.hi) - p.mean.lo;
        y[j] = __builtin_fmaf(off * p.root, w[j], b[j]);
    }
    return Vec<T>::narrow(y);
}

// The weight's (or bias's) vector; `none` where it is absent.
template <typename T>
__device__ __forceinline__ typename Vec<T>::wide affine(const void *p, u32x4 v, float none)
{
    return p ? Vec<T>::widen(v) : typename Vec<T>::wide(none);
}

// ---------------------------------------------------------------------------
// Forward, rows that fit in registers: Waves waves a row, V vectors a lane.
//
// The mean comes before the squares about it, so the row stays in registers:
// it is read once and written once, and its waves meet at one barrier.  Each
// has summed differences from a number of its own (WaveSums) by then, which
// every wave brings to the common mean in binary64 by itself.
// Bound by memory: 8192 x 4096 bf16 with residual, total and statistics take
// 46.4 us, 5.8 TB/s (the vector unit is busy 44 % of the cycles), 1 x 4096 2.7
// us, the latency of one load and the join (0.2 of it what keeps rows of any
// numbers right: 2-8 % of short rows' time).  A block that stays and has its
// next row's loads on their way took 51-58 us: new blocks overlap as well, and
// their registers are free earlier.
// ---------------------------------------------------------------------------

// R rows at a time, whose loads are on their way together and whose sums hide
// each other's latency; weight and bias are read once for both.
template <typename T, int Waves, int V, int R, RowFit Fit>
__device__ __forceinline__ void layernorm_rows_of(const LayerNormArgs &a,
                                                  WaveSums (*shared)[R][layernorm_block(Waves) / 64])
{
    constexpr uint32_t N = Vec<T>::N, kThreads = Waves * 64;
    constexpr uint32_t kRows = layernorm_block(Waves) / kThreads;
    // weight and bias are on their way with the rows, unless they would not fit
    // in registers
    constexpr bool kEarly = V < 3;
    const uint32_t group = row_of_thread<kThreads, kRows>(), i = place_in_row<kThreads, kRows>();
    const uint32_t wave = Waves > 1 ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(i / 64)) : 0;
    const T *const weight = static_cast<const T *>(a.weight), *const bias = static_cast<const T *>(a.bias);
    const uint32_t cols = Fit == kWhole ? kThreads * V * N : a.cols;
    const auto piece = [&](int k) { return Piece<T, Fit>((i + k * kThreads) * N, cols); };
    // elements of wave w of a row
    const auto elements = [&](uint32_t w) {
        if constexpr (Fit == kWhole) return 64 * V * N;
        uint32_t n = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint32_t from = (w * 64 + k * kThreads) * N;
            n += from >= cols ? 0 : cols - from < 64 * N ? cols - from : 64 * N;
        }
        return n;
    };
    int set = 0;
    // a block's rows go round together (the barriers)
    for (uint64_t r0 = (uint64_t)blockIdx.x * (kRows * R); r0 < a.rows;
         r0 += (uint64_t)gridDim.x * (kRows * R), set ^= 1) {
        const auto live = [&](int q) { return r0 + q * kRows + group < a.rows; };
        const auto row = [&](int q) { return live(q) ? r0 + q * kRows + group : r0; };
        u32x4 h[R][V], w[V], b[V];
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int k = 0; k < V; ++k)
                h[q][k] = load_piece<T, true>(static_cast<const T *>(a.x) + row(q) * a.x_stride, cols, piece(k));
        const auto fetch_affine = [&](int k) {
            if (weight) w[k] = load_piece<T, false>(weight, cols, piece(k));
            if (bias) b[k] = load_piece<T, false>(bias, cols, piece(k));
        };
        if (a.residual) {
            u32x4 res[R][V];
#pragma unroll
            for (int q = 0; q < R; ++q)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    res[q][k] = load_piece<T, true>(
                        static_cast<const T *>(a.residual) + row(q) * a.residual_stride, cols, piece(k));
            if constexpr (kEarly)
#pragma unroll
                for (int k = 0; k < V; ++k) fetch_affine(k);
#pragma unroll
            for (int q = 0; q < R; ++q)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    h[q][k] = Vec<T>::narrow(Vec<T>::widen(h[q][k]) + Vec<T>::widen(res[q][k]));
        } else if constexpr (kEarly) {
#pragma unroll
            for (int k = 0; k < V; ++k) fetch_affine(k);
        }
        WaveSums own[R];
#pragma unroll
        for (int q = 0; q < R; ++q) own[q] = wave_sums<T, V, Fit>(h[q], cols, elements(wave), a.eps, piece);
        if constexpr (Waves > 1) {
            // the outputs may be the inputs: nothing is stored before every
            // wave of the rows has loaded (a row of one wave loads before it
            // stores)
            if (threadIdx.x % 64 == 0)
#pragma unroll
                for (int q = 0; q < R; ++q) shared[set][q][group * Waves + wave] = own[q];
            __syncthreads();
        }
        const uint32_t at = threadIdx.x % lanes_of_waves(Waves);
        const bool some = at < (uint32_t)Waves;
        const uint32_t n = Waves == 1 ? cols : some ? elements(at) : 0;
        Place place[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const WaveSums of = Waves == 1 ? own[q] : shared[set][q][group * Waves + (some ? at : 0)];
            const double mean = divide(sum_of_waves<Waves>(n ? sum_of(of, n) : 0.0), cols, a.by_cols);
            const auto squares = [&](int shift) {
                return sum_of_waves<Waves>(n ? squares_about(of, n, mean, shift) : 0.0f);
            };
            const float sq = squares(0);
            place[q] = Place(mean, sq, (float)a.by_cols, a.eps, 0);
            const int shift = shift_for(sq, a.eps, (float)mean);
            if (shift != 0)                  // (the same in all of the wave)
                place[q] = Place(mean, squares(shift), (float)a.by_cols, a.eps, shift);
            if (live(q) && i == 0) {
                if (a.mean) a.mean[row(q)] = (float)mean;
                if (a.rstd) a.rstd[row(q)] = place[q].rstd();
            }
            place[q].to_scalars();
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const uint64_t r = row(q);
            if (live(q) && a.total) {
                T *const total = static_cast<T *>(a.total) + r * a.total_stride;
#pragma unroll
                for (int k = 0; k < V; ++k) store_piece(total, cols, piece(k), h[q][k]);
            }
            if (!live(q)) continue;
            T *const y = static_cast<T *>(a.y) + r * a.y_stride;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (!kEarly && q == 0) fetch_affine(k);
                store_piece(y, cols, piece(k),
                            normed<T>(h[q][k], place[q], affine<T>(weight, w[k], 1.0f),
                                      affine<T>(bias, b[k], 0.0f)));
            }
        }
    }
}

template <typename T, int Waves, int V, int R = 1, bool Tiny = false>
__global__ void __launch_bounds__(layernorm_block(Waves)) ew_layernorm_kernel(LayerNormArgs a)
{
    // two sets, used in turn: a wave is at most one barrier ahead of another
    __shared__ WaveSums shared[2][R][layernorm_block(Waves) / 64];
    if constexpr (Tiny) layernorm_rows_of<T, Waves, V, R, kTiny>(a, shared);
    else if (a.cols == Waves * 64 * V * Vec<T>::N) layernorm_rows_of<T, Waves, V, R, kWhole>(a, shared);
    else layernorm_rows_of<T, Waves, V, R, kPart>(a, shared);
}

// ---------------------------------------------------------------------------
// Forward, longer rows: a block a row, three passes over it (sum, squares,
// output; squares that leave binary32 take one more), of which the caches serve
// the later ones in part: 1820 x 18432 f32 with a residual 141 us, 1000 x 40000
// bf16 94 us (3.8 and 3.4 TB/s of what it cannot do without).
// ---------------------------------------------------------------------------

constexpr int kLongBlock = 1024;
constexpr int kLongWaves = kLongBlock / 64;

// Sum over a block of kLongWaves waves, in all of them.
__device__ __forceinline__ double long_sum(double x, double *scratch)
{
    x = wave_sum64(x);
    if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64] = x;
    __syncthreads();
    return sum_of_waves<kLongWaves>(scratch[threadIdx.x % kLongWaves]);
}
__device__ __forceinline__ float long_sum(float x, float *scratch)
{
    x = wave_reduce<Sum>(x);
    if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64] = x;
    __syncthreads();
    return sum_of_waves<kLongWaves>(scratch[threadIdx.x % kLongWaves]);
}

template <typename T>
__global__ void __launch_bounds__(kLongBlock) ew_layernorm_long_kernel(LayerNormArgs a)
{
    constexpr uint32_t N = Vec<T>::N;
    using Wide = typename Vec<T>::wide;
    __shared__ double sums[2][kLongWaves];
    __shared__ float sqs[2][kLongWaves];
    const T *const weight = static_cast<const T *>(a.weight), *const bias = static_cast<const T *>(a.bias);
    int set = 0;
    for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x, set ^= 1) {
        const T *const x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *const res =
            a.residual ? static_cast<const T *>(a.residual) + r * a.residual_stride : nullptr;
        T *const total = a.total ? static_cast<T *>(a.total) + r * a.total_stride : nullptr;
        const auto value = [&](const LongPiece<T> &p) {
            const u32x4 h = p.template load<false>(x);
            return res ? Vec<T>::narrow(Vec<T>::widen(h) + Vec<T>::widen(p.template load<false>(res))) : h;
        };
        // (the first pass stores total where its thread reads it back: total
        // may be x or residual)
        const auto again = [&](const LongPiece<T> &p) { return total ? p.template load<false>(total) : value(p); };
        double sum = 0.0;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
            const LongPiece<T> p(at, a.cols);
            const u32x4 h = value(p);
            const Wide f = Vec<T>::widen(h);
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) sum += j >= p.p.skip ? (double)f[j] : 0.0;
            if (total) p.store(total, h);
        }
        const double mean = divide(long_sum(sum, sums[set]), a.cols, a.by_cols);
        const auto squares = [&](int shift) {
            const float scale = __builtin_ldexpf(1.0f, shift);
            const Mean m(mean * (double)scale);
            float sq = 0.0f;
            for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
                const LongPiece<T> p(at, a.cols);
                const Wide f = Vec<T>::widen(again(p));
#pragma unroll
                for (uint32_t j = 0; j < N; ++j) {
                    const float d = __builtin_fmaf(f[j], scale, -m.hi) - m.lo;
                    sq = j >= p.p.skip ? __builtin_fmaf(d, d, sq) : sq;
                }
            }
            return long_sum(sq, sqs[set]);
        };
        const float sq = squares(0);
        Place place(mean, sq, (float)a.by_cols, a.eps, 0);
        const int shift = shift_for(sq, a.eps, (float)mean);
        if (shift != 0) {                    // (the same in all of the block)
            __syncthreads();                 // every thread has read the first sum
            place = Place(mean, squares(shift), (float)a.by_cols, a.eps, shift);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = (float)mean;
            if (a.rstd) a.rstd[r] = place.rstd();
        }
        T *const y = static_cast<T *>(a.y) + r * a.y_stride;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
            const LongPiece<T> p(at, a.cols);
            u32x4 w{}, b{};
            if (weight) w = p.template load<false>(weight);
            if (bias) b = p.template load<false>(bias);
            p.store(y, normed<T>(again(p), place, affine<T>(weight, w, 1.0f), affine<T>(bias, b, 0.0f)));
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

// dweight and dbias are added up in two steps: at most this many blocks sum a
// part of the rows each, then the parts are summed.  One block a CU (512: 5-10
// us slower at 8192 x 4096, a row's bytes of sums more a part; 128: 66.0 us
// against 48.0 at 3000 x 8960 bf16).
constexpr uint32_t kParts = 256;

// Floats of one part's sums of dweight (those of dbias follow): whole vectors.
__host__ __device__ constexpr uint64_t sums_pitch(uint64_t cols) { return (cols + 7) & ~(uint64_t)7; }

// A row's differences from its mean in the gradient: times a power of two that
// keeps them, and their products with a gradient, inside binary32, and is 1 for
// standard deviations between 2^-50 and 2^50.  (Numbers that close to one above
// 1 are equal to it.)
struct Differences {
    float scale, at, rstd;      // at: the mean times scale; rstd by scale
    __device__ Differences(float mean, float root)
        : scale(root < 0x1p-50f                                    ? 0x1p-80f
                : root > 0x1p50f && __builtin_fabsf(mean) <= 1.0f ? 0x1p80f
                                                                   : 1.0f),
          at(mean * scale), rstd(root * (scale < 1.0f ? 0x1p80f : scale > 1.0f ? 0x1p-80f : 1.0f))
    {
    }
    template <class Wide>
    __device__ Wide of(Wide x) const
    {
#pragma unroll
        for (uint32_t j = 0; j < sizeof(x) / sizeof(float); ++j) x[j] = __builtin_fmaf(x[j], scale, -at);
        return x;
    }
};

// Whether what the given mean's rounding lost (half of a last place, 2^-24 of it)
// is more than 2^-12 of a deviation: such rows' mean difference, 0 but for that,
// is found from the row again.
__device__ __forceinline__ bool far_from_zero(float mean, float rstd)
{
    return __builtin_fabsf(mean) * rstd > 0x1p12f;
}

// A piece's sums over rows to a row of floats (elements that two pieces hold
// have the same sums in both).
template <typename T, RowFit Fit>
__device__ __forceinline__ void store_sums(float *row, uint32_t cols, const Piece<T, Fit> &p,
                                           typename Vec<T>::wide v)
{
    typedef float Sums __attribute__((ext_vector_type(Vec<T>::N), aligned(4)));
    if (!p.live) return;
    if constexpr (Fit == kTiny) {
#pragma unroll
        for (uint32_t j = 0; j < Vec<T>::N; ++j)
            if (j < cols) row[j] = v[j];
    } else {
        *reinterpret_cast<Sums *>(row + p.first) = v;
    }
}

// Rows that fit in registers: Waves waves a row, V vectors a lane, Groups rows
// at a time in a block, which adds up dweight and dbias over its rows in
// registers.  Bound by memory: 8192 x 4096 bf16 with dtotal 45 us, 6.0 TB/s,
// then 4.0-4.7 us for the sum of the parts.
template <typename T, int Waves, int V, int Groups>
struct GradShared {
    // two sets, used in turn: a wave is at most one barrier ahead of another
    float firsts[2][Waves * Groups], seconds[2][Waves * Groups], thirds[2][Waves * Groups];
    float joined[Groups > 1 ? Waves * 64 * V * Vec<T>::N : 1];
};

template <typename T, int Waves, int V, int Groups, RowFit Fit>
__device__ __forceinline__ void layernorm_grad_rows(const LayerNormGradArgs &a,
                                                    GradShared<T, Waves, V, Groups> &shared)
{
    constexpr uint32_t N = Vec<T>::N, kThreads = Waves * 64;
    using Wide = typename Vec<T>::wide;
    const uint32_t group = row_of_thread<kThreads, Groups>(), i = place_in_row<kThreads, Groups>();
    // the next row is on its way while this one is worked on, and the weight
    // stays, unless they would not fit in registers (bf16 rows of 12288: 64.4 us
    // for 3000, 80.0 without)
    constexpr bool kAhead = V * N <= 8 || (V * N <= 16 && Waves <= 12);
    const T *const weight = static_cast<const T *>(a.weight);
    const uint32_t cols = a.cols;
    const auto piece = [&](int k) { return Piece<T, Fit>((i + k * kThreads) * N, cols); };
    u32x4 wv[kAhead ? V : 1];
    const auto fetch_weight = [&](int k) {
        return weight ? load_piece<T, false>(weight, cols, piece(k)) : u32x4{};
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
            v[k] = load_piece<T, true>(static_cast<const T *>(p) + first, cols, piece(k));
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
    const float by = (float)(1.0 / (double)cols);
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
            dyv[k] = dy[k];
            xv[k] = x[k];
            if constexpr (kAhead) dtv[k] = dt[k];
        }
        if constexpr (kAhead) {
            if (r0 + step < a.rows) fetch_row(r0 + step);
            __builtin_amdgcn_sched_barrier(0);       // the loads stay ahead of the sums
        }
        // with h = (off - low) * diff.rstd: low and that come in once a row
        const Differences diff(mu, rs);
        float first = 0.0f, second = 0.0f, third = 0.0f;
        const bool far = far_from_zero(mu, rs);          // the same in all of the row
#pragma unroll
        for (int k = 0; k < V; ++k) {
            // (past a tiny row and in dead pieces dy is 0)
            const Wide d = Vec<T>::widen(dyv[k]), off = diff.of(Vec<T>::widen(xv[k]));
            Wide g = d * factor(k);
            if (live) {
                dw[k] += (d * diff.rstd) * off;
                db[k] += d;
            }
            if constexpr (Fit == kPart)        // without what is another piece's too
                g = Vec<T>::widen(own_bits(dyv[k], cols, piece(k))) * factor(k);
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) {
                first += g[j];
                second = __builtin_fmaf(g[j], off[j], second);
            }
        }
        const uint32_t wave = group * Waves + i / 64;
        if (far) {
            uint32_t n = cols;
            asm("" : "+s"(n));             // (nothing is kept from above for this rare path)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const Wide off = diff.of(Vec<T>::widen(xv[k]));
                const Piece<T, Fit> p((i + k * kThreads) * N, n);
#pragma unroll
                for (uint32_t j = 0; j < N; ++j) third += p.live && p.own(j, n) ? off[j] : 0.0f;
            }
            third = wave_reduce<Sum>(third);
            if (Waves > 1 && threadIdx.x % 64 == 0) shared.thirds[set][wave] = third;
        }
        // dx may be an input: nothing is stored before every wave of the row
        // has loaded
        first = wave_reduce<Sum>(first);
        second = wave_reduce<Sum>(second);
        const uint32_t at = threadIdx.x % lanes_of_waves(Waves), of = group * Waves + (at < Waves ? at : 0);
        if constexpr (Waves > 1) {
            if (threadIdx.x % 64 == 0) {
                shared.firsts[set][wave] = first;
                shared.seconds[set][wave] = second;
            }
            __syncthreads();
            first = sum_of_waves<Waves>(at < Waves ? shared.firsts[set][of] : 0.0f);
            second = sum_of_waves<Waves>(at < Waves ? shared.seconds[set][of] : 0.0f);
        }
        if (far) {
            if constexpr (Waves > 1) third = sum_of_waves<Waves>(at < Waves ? shared.thirds[set][of] : 0.0f);
            const float low = third * by;
            second -= low * first;
            // (so that dx takes off as it is)
            first -= low * (second * diff.rstd) * diff.rstd;
            if (live)
#pragma unroll
                for (int k = 0; k < V; ++k) dw[k] -= (Vec<T>::widen(dyv[k]) * diff.rstd) * low;
        }
        first *= by;
        second = second * diff.rstd * (diff.rstd * by);
        if (!live) continue;
        T *const dx = static_cast<T *>(a.dx) + r * a.dx_stride;
        u32x4 part{};              // what is the partial vector's own, stored last
        uint32_t part_skip = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const Wide off = diff.of(Vec<T>::widen(xv[k]));
            Wide g = Vec<T>::widen(dyv[k]) * factor(k) - first, dt(0.0f);
            if (a.dtotal) {
                if constexpr (kAhead) dt = Vec<T>::widen(dtv[k]);
                else
                    dt = Vec<T>::widen(load_piece<T, true>(
                        static_cast<const T *>(a.dtotal) + r * a.dtotal_stride, cols, piece(k)));
            }
#pragma unroll
            for (uint32_t j = 0; j < N; ++j)
                g[j] = __builtin_fmaf(rs, __builtin_fmaf(-off[j], second, g[j]), dt[j]);
            // (dx may be dtotal, whose other elements another wave may yet read)
            const Piece<T, Fit> p = piece(k);
            if (kAhead || Fit != kPart || p.skip == 0) {
                store_piece(dx, cols, p, Vec<T>::narrow(g));
            } else if (p.live) {
                part = Vec<T>::narrow(g);
                part_skip = p.skip;
            }
        }
        if (part_skip) {
            const typename Vec<T>::type v = __builtin_bit_cast(typename Vec<T>::type, part);
#pragma unroll
            for (uint32_t j = 1; j < N; ++j)
                if (j >= part_skip) dx[cols - N + j] = v[j];
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
                        for (uint32_t j = 0; j < N; ++j)
                            shared.joined[(k * N + j) * kThreads + i] = v[k][j];
                __syncthreads();
                if (group == 0)
#pragma unroll
                    for (int k = 0; k < V; ++k)
#pragma unroll
                        for (uint32_t j = 0; j < N; ++j)
                            v[k][j] += shared.joined[(k * N + j) * kThreads + i];
                __syncthreads();
            }
        };
        join(dw);
        join(db);
    }
    if (group != 0) return;
    // the one part of a small call is the sum
    float *const part = static_cast<float *>(a.workspace) + blockIdx.x * (2 * sums_pitch(cols));
    float *const to_w = gridDim.x == 1 ? a.dweight : part;
    float *const to_b = gridDim.x == 1 ? a.dbias : part + sums_pitch(cols);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (to_w) store_sums(to_w, cols, piece(k), dw[k]);
        if (to_b) store_sums(to_b, cols, piece(k), db[k]);
    }
}

template <typename T, int Waves, int V, int Groups, bool Tiny = false>
__global__ void __launch_bounds__(Waves * 64 * Groups) ew_layernorm_back_kernel(LayerNormGradArgs a)
{
    __shared__ GradShared<T, Waves, V, Groups> shared;
    if constexpr (Tiny) layernorm_grad_rows<T, Waves, V, Groups, kTiny>(a, shared);
    else layernorm_grad_rows<T, Waves, V, Groups, kPart>(a, shared);
}

// dweight (blockIdx.y 0) and dbias (1) from the parts' sums: 32 columns a
// block, 32 threads a column, eight parts a thread on their way together.
// Latency: 4.0-4.7 us for 256 parts of 4096 columns (8 MB).
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
#pragma unroll 8
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
// Gradient, longer rows: what the rounded means lost, the parts' sums of dweight
// and dbias (a thread a vector of columns over a part of the rows), their sum,
// then dx (a block a row, two passes over it).  dx comes last: it may be dy or x.
// 1820 x 18432 with dtotal 196 us of f32 and 115 of bf16, 1000 x 40000 bf16 145
// (191, 111 and 142 without the first launch): dy and x are read three times, the
// second pass over a row from the caches.
// ---------------------------------------------------------------------------

constexpr uint32_t kColsBlock = 256;

// The mean difference of row r of a block of Waves waves, where the row is far
// from 0, else 0.
template <typename T, int Waves>
__device__ __forceinline__ float lost_mean(const LayerNormGradArgs &a, uint64_t r, const Differences &diff,
                                           float *scratch)
{
    if (!far_from_zero(a.mean[r], a.rstd[r])) return 0.0f;
    __syncthreads();               // scratch may be read for another row yet
    const T *const x = static_cast<const T *>(a.x) + r * a.x_stride;
    float sum = 0.0f;
    for (uint64_t at = threadIdx.x * Vec<T>::N; at < a.cols; at += Waves * 64 * Vec<T>::N) {
        const LongPiece<T> p((uint32_t)at, a.cols);
        const typename Vec<T>::wide off = diff.of(Vec<T>::widen(p.template load<false>(x)));
#pragma unroll
        for (uint32_t j = 0; j < Vec<T>::N; ++j) sum += j >= p.p.skip ? off[j] : 0.0f;
    }
    if constexpr (Waves == kLongWaves) return long_sum(sum, scratch) / (float)a.cols;
    else return block_reduce<Sum, Waves>(sum, scratch) / (float)a.cols;
}

// Rows of cols > kLongCols, in every type, take these kernels; lost: a value a
// row behind the parts' sums.
constexpr uint32_t kLongCols = 16384;
constexpr int kLostWaves = 4;      // few: most rows are not far from 0

template <typename T>
__global__ void __launch_bounds__(kLostWaves * 64) ew_layernorm_lost_kernel(LayerNormGradArgs a, float *lost)
{
    __shared__ float scratch[kLostWaves];
    for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float low = lost_mean<T, kLostWaves>(a, r, Differences(a.mean[r], a.rstd[r]), scratch);
        if (threadIdx.x == 0) lost[r] = low;
    }
}

template <typename T>
__global__ void __launch_bounds__(kColsBlock) ew_layernorm_cols_kernel(LayerNormGradArgs a,
                                                                      uint32_t parts, const float *lost)
{
    using Wide = typename Vec<T>::wide;
    const uint32_t at = (blockIdx.x * kColsBlock + threadIdx.x) * Vec<T>::N;
    if (at >= a.cols) return;
    const LongPiece<T> p(at, a.cols);
    Wide dw(0.0f), db(0.0f);
    for (uint64_t r = blockIdx.y; r < a.rows; r += parts) {
        const Wide d = Vec<T>::widen(p.template load<true>(static_cast<const T *>(a.dy) + r * a.dy_stride));
        const Wide x = Vec<T>::widen(p.template load<true>(static_cast<const T *>(a.x) + r * a.x_stride));
        const Differences diff(a.mean[r], a.rstd[r]);
        dw += d * ((diff.of(x) - lost[r]) * diff.rstd);
        db += d;
    }
    float *const part = static_cast<float *>(a.workspace) + blockIdx.y * (2 * sums_pitch(a.cols));
    store_sums(part + p.first, a.cols, p.p, dw);
    store_sums(part + sums_pitch(a.cols) + p.first, a.cols, p.p, db);
}

template <typename T>
__global__ void __launch_bounds__(kLongBlock) ew_layernorm_dx_kernel(LayerNormGradArgs a)
{
    constexpr uint32_t N = Vec<T>::N;
    using Wide = typename Vec<T>::wide;
    __shared__ float firsts[2][kLongWaves], seconds[2][kLongWaves], thirds[kLongWaves];
    const T *const weight = static_cast<const T *>(a.weight);
    int set = 0;
    for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x, set ^= 1) {
        const T *const dy = static_cast<const T *>(a.dy) + r * a.dy_stride;
        const T *const x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *const dt =
            a.dtotal ? static_cast<const T *>(a.dtotal) + r * a.dtotal_stride : nullptr;
        T *const dx = static_cast<T *>(a.dx) + r * a.dx_stride;
        const float rs = a.rstd[r];
        const Differences diff(a.mean[r], rs);
        const auto slope = [&](const LongPiece<T> &p) {
            const Wide d = Vec<T>::widen(p.template load<false>(dy));
            return weight ? d * Vec<T>::widen(p.template load<false>(weight)) : d;
        };
        const float low = lost_mean<T, kLongWaves>(a, r, diff, thirds);
        const auto place = [&](const LongPiece<T> &p) {
            return (diff.of(Vec<T>::widen(p.template load<false>(x))) - low) * diff.rstd;
        };
        float first = 0.0f, second = 0.0f;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
            const LongPiece<T> p(at, a.cols);
            const Wide g = slope(p), h = place(p);
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) {
                const bool own = j >= p.p.skip;
                first += own ? g[j] : 0.0f;
                second = own ? __builtin_fmaf(g[j], h[j], second) : second;
            }
        }
        first = wave_reduce<Sum>(first);
        second = wave_reduce<Sum>(second);
        if (threadIdx.x % 64 == 0) {
            firsts[set][threadIdx.x / 64] = first;
            seconds[set][threadIdx.x / 64] = second;
        }
        __syncthreads();
        first = sum_of_waves<kLongWaves>(firsts[set][threadIdx.x % kLongWaves]) / (float)a.cols;
        second = sum_of_waves<kLongWaves>(seconds[set][threadIdx.x % kLongWaves]) / (float)a.cols;
        for (uint32_t at = threadIdx.x * N; at < a.cols; at += kLongBlock * N) {
            const LongPiece<T> p(at, a.cols);
            Wide g = rs * ((slope(p) - first) - place(p) * second);
            if (dt) g += Vec<T>::widen(p.template load<false>(dt));
            p.store(dx, Vec<T>::narrow(g));
        }
    }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

// Waves and vectors a lane by the row's length, so that few lanes are idle, and
// by the number of rows: more waves where a block a row is at most one a CU
// (kRowACu), few where the blocks are all there at once (kOneRound), two rows
// at a time where they are more.  us, in a graph, waves x vectors of bf16 with a
// residual, 2^25 elements where no rows are given:
//   512 columns   1x1 46.5, 1x2 60.1         5120    3x4 53.4, 5x2 53.0
//   1024          2x1 46.7, 1x2 47.3         6144    3x4 49.4, 4x4 53.9
//   2048          4x1 46.8, 2x2 47.1         8192    4x4 49.4, 8x2 51.1, 16x1 60.8
//   2560          3x2 50.1, 5x1 54.4         12288   12x2 55.6, 6x4 61.1
//   4096          4x2 48.4, 2x4 48.4, 8x1 49.3   16384   16x2 56.5, 8x4 54.9
//   1024 rows: of 2560 5x1 5.7, 3x2 6.1, 2x4 7.7; of 4096 2x4 7.4, 4x2 7.8, 8x1 8.7
//   one row of 4096: 8x1 2.7, 4x2 2.8, 2x4 3.8
//   f32: 1021 x 5003 without a residual 5x4 9.5, 7x3 10.5, 12x2 12.3
// Two rows at a time against one, without and with a residual: 10000 x 4096
// 32.4, 34.1 and (8192) 50.3, 47.9; 20000 x 1000 20.0, 22.9 and 31.7, 30.7;
// 3000 x 12288 35.6, 44.0 and 58.6, 60.6; of fewer blocks 2600 x 256 4.0, 3.7.
// With a residual a lane of 4x2 has four vectors on their way already: from two
// rounds of blocks on it stays with one row (one row, two: 3000 x 4096 20.4,
// 21.1; 1300 10.6, 9.7).
constexpr uint32_t kRowACu = 256, kOneRound = 1280;

template <typename T>
static hipError_t layernorm_rows(const LayerNormArgs &a, uint32_t vectors, hipStream_t s)
{
#define EW_LAYERNORM_LAUNCH(W, V, R, TINY)                                               \
    return start(reinterpret_cast<const void *>(&ew_layernorm_kernel<T, W, V, R, TINY>), \
                 dim3(row_blocks((blocks_of(W) + R - 1) / R)), layernorm_block(W), 0, s, a);
#define EW_LAYERNORM_ROWS(W, V) \
    if (vectors <= W * 64 * V) EW_LAYERNORM_LAUNCH(W, V, 1, false)
#define EW_LAYERNORM_PAIRS(W, V) \
    if (vectors <= W * 64 * V && blocks_of(W) > kOneRound) EW_LAYERNORM_LAUNCH(W, V, 2, false)
    const auto blocks_of = [&](uint32_t waves) {
        const uint64_t rows = (uint64_t)layernorm_block((int)waves) / (waves * 64);
        return (a.rows + rows - 1) / rows;
    };
    if (a.cols < (uint32_t)Vec<T>::N) EW_LAYERNORM_LAUNCH(1, 1, 1, true)
    EW_LAYERNORM_PAIRS(1, 1)
    EW_LAYERNORM_ROWS(1, 1)
    EW_LAYERNORM_PAIRS(2, 1)
    EW_LAYERNORM_ROWS(2, 1)
    EW_LAYERNORM_PAIRS(3, 1)
    EW_LAYERNORM_ROWS(3, 1)
    EW_LAYERNORM_PAIRS(4, 1)
    EW_LAYERNORM_ROWS(4, 1)
    EW_LAYERNORM_PAIRS(3, 2)
    if (a.residual && a.rows > 2 * kOneRound) {
        EW_LAYERNORM_ROWS(4, 2)
    }
    EW_LAYERNORM_PAIRS(4, 2)
    if (a.rows <= kOneRound) {
        EW_LAYERNORM_ROWS(5, 1)
        if (a.rows <= kRowACu) {
            EW_LAYERNORM_ROWS(8, 1)
            EW_LAYERNORM_ROWS(16, 1)
        }
        EW_LAYERNORM_ROWS(3, 2)
        EW_LAYERNORM_ROWS(2, 4)
    }
    EW_LAYERNORM_ROWS(3, 4)
    EW_LAYERNORM_ROWS(4, 4)
    if constexpr (sizeof(T) == 4) {
        EW_LAYERNORM_ROWS(5, 4)
        EW_LAYERNORM_ROWS(6, 4)
        EW_LAYERNORM_ROWS(8, 4)
        EW_LAYERNORM_ROWS(16, 4)
    } else {
        EW_LAYERNORM_PAIRS(12, 2)
        EW_LAYERNORM_ROWS(12, 2)
        EW_LAYERNORM_PAIRS(16, 2)
        EW_LAYERNORM_ROWS(16, 2)
        EW_LAYERNORM_ROWS(12, 4)
    }
#undef EW_LAYERNORM_PAIRS
#undef EW_LAYERNORM_ROWS
#undef EW_LAYERNORM_LAUNCH
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
    const uint64_t sums = (rows < kParts ? rows : kParts) * 2 * sums_pitch(cols);
    return (sums + (cols > kLongCols ? sums_pitch(rows) : 0)) * sizeof(float);
}

// Up to kOneShort rounds of short rows (of kShort vectors), kOneLong of others,
// are one block's, which writes dweight and dbias itself and saves the second
// launch, 3 us of the host's.  us, in a graph, one block and a block a round:
// bf16 3 x 4096 4.9, 5.7; 32 x 512 6.8, 6.6; 16 x 2048 8.9, 7.2; f32 16 x 1000
// 7.7, 6.1; of longer rows 4 x 12288 bf16 10.7, 8.8; 4 x 16384 17.0, 10.7.
// Long rows, a block each, go two to a part where that still is 81 blocks or
// more: each part's sums are as many bytes as a row and its gradient.  Two rows a
// part and one: 200 and 250 x 4096 bf16 9.0, 10.0 and 9.2, 10.4; 250 x 8192 12.7,
// 15.2; 250 x 16384 25.0, 27.6; 250 x 8192 f32 13.9, 15.6; but 161 x 16384 bf16
// 22.3, 21.4 and f32 26.1, 23.3, where the blocks are few for so many bytes.
// Without sums there is nothing of that to save: a block a round up to one a CU
// (4 x 4096 bf16 2.9 us, 5.3 in one block; 32 x 512 2.7, 5.0; 170 x 16384 8.8,
// 13.5 with two rows a block; 8192 x 4096 44.3, 47 with 512 blocks, 52 with all).
constexpr uint64_t kOneShort = 4, kOneLong = 2, kTwoRowsFrom = 160, kTwoRowsTo = 384;
constexpr uint32_t kShort = 512;

static uint32_t parts_for(uint64_t blocks, int groups, uint32_t vectors, bool sums)
{
    if (!sums) return (uint32_t)(blocks < kParts ? blocks : kParts);
    if (blocks <= (vectors <= kShort ? kOneShort : kOneLong)) return 1;
    if (groups == 1 && blocks > kTwoRowsFrom && blocks <= kTwoRowsTo) return (uint32_t)((blocks + 1) / 2);
    return (uint32_t)(blocks < kParts ? blocks : kParts);
}

template <typename T>
static hipError_t layernorm_grad_by(const LayerNormGradArgs &a, uint32_t vectors, hipStream_t s,
                                      uint32_t *parts)
{
#define EW_LAYERNORM_GRAD_LAUNCH(W, V, G, TINY)                                                   \
    {                                                                                             \
        const uint64_t blocks = ((uint64_t)a.rows + G - 1) / G;                                   \
        *parts = parts_for(blocks, G, vectors, a.dweight || a.dbias);                             \
        return start(reinterpret_cast<const void *>(&ew_layernorm_back_kernel<T, W, V, G, TINY>), \
                     dim3(*parts), W * 64 * G, 0, s, a);                                          \
    }
    // us, in a graph, 2^25 elements with dtotal, waves x vectors x rows at a time:
    //   bf16  2560 6x1x2 52.7, 8x1x1 56.9; 4096 8x1x1 51.3, 16x1x1 57-60; 5120
    //         16x1x1 54.7, 8x2x1 56.0; 3000 x 16384 16x2x1 96.5, 8x4x1 128.9
    //   f32   1280 8x1x2 52.1, 8x1x1 56.7; 6144 16x2x1 53.8; 8192 56.0
    //   short rows: 2000 x 1000 bf16 2x1x4 9.7, 2x1x8 12.3; 250 x 100 1x1x8 6.7,
    //   1x1x16 8.7; 1000 x 1281 3x1x4 11.3, 4x1x4 11.6
#define EW_LAYERNORM_GRAD_ROWS(W, V, G) \
    if (vectors <= W * 64 * V) EW_LAYERNORM_GRAD_LAUNCH(W, V, G, false)
    if (a.cols < (uint32_t)Vec<T>::N) EW_LAYERNORM_GRAD_LAUNCH(1, 1, 8, true)
    EW_LAYERNORM_GRAD_ROWS(1, 1, 8)
    EW_LAYERNORM_GRAD_ROWS(2, 1, 4)
    EW_LAYERNORM_GRAD_ROWS(3, 1, 4)
    EW_LAYERNORM_GRAD_ROWS(4, 1, 4)
    if constexpr (sizeof(T) == 4) {
        if (vectors <= 384) EW_LAYERNORM_GRAD_LAUNCH(8, 1, 2, false)
        EW_LAYERNORM_GRAD_ROWS(8, 1, 1)
        EW_LAYERNORM_GRAD_ROWS(16, 1, 1)
        EW_LAYERNORM_GRAD_ROWS(16, 2, 1)
        EW_LAYERNORM_GRAD_ROWS(16, 4, 1)
    } else {
        EW_LAYERNORM_GRAD_ROWS(6, 1, 2)
        EW_LAYERNORM_GRAD_ROWS(8, 1, 1)
        EW_LAYERNORM_GRAD_ROWS(16, 1, 1)
        EW_LAYERNORM_GRAD_ROWS(12, 2, 1)
        EW_LAYERNORM_GRAD_ROWS(16, 2, 1)
    }
#undef EW_LAYERNORM_GRAD_ROWS
#undef EW_LAYERNORM_GRAD_LAUNCH
    return hipErrorInvalidValue;
}
static_assert(16 * 64 * 4 * 4 == kLongCols && 16 * 64 * 2 * 8 == kLongCols);

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
    if (a.cols <= kLongCols) {
        *path = "rows in registers";
        const hipError_t e = t == kRowF32   ? layernorm_grad_by<float>(a, vectors, s, &parts)
                             : t == kRowF16 ? layernorm_grad_by<_Float16>(a, vectors, s, &parts)
                                            : layernorm_grad_by<__bf16>(a, vectors, s, &parts);
        return e != hipSuccess || !sums || parts == 1 ? e : sum(parts);
    }
    *path = "two passes, dweight and dbias by columns";
    if (sums) {
        parts = a.rows < kParts ? a.rows : kParts;
        float *const lost = static_cast<float *>(a.workspace) + parts * 2 * sums_pitch(a.cols);
        hipError_t e = start(EW_KERNEL_OF(t, ew_layernorm_lost_kernel), dim3(row_blocks(a.rows)),
                             kLostWaves * 64, 0, s, a, lost);
        if (e == hipSuccess)
            e = start(EW_KERNEL_OF(t, ew_layernorm_cols_kernel),
                      dim3((vectors + kColsBlock - 1) / kColsBlock, parts), kColsBlock, 0, s, a, parts,
                      (const float *)lost);
        if (e == hipSuccess) e = sum(parts);
        if (e != hipSuccess) return e;
    }
    return start(EW_KERNEL_OF(t, ew_layernorm_dx_kernel), dim3(row_blocks(a.rows)), kLongBlock, 0, s, a);
}

}  // namespace ew
