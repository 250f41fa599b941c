// ew_norm.hip -- the RMS norm with the residual's addition (plain and e4m3
// output) and its gradient for CDNA4 (gfx950).

#include "ew_rows_device.h"

namespace ew {

constexpr int kNormBlock = 256;
constexpr int kNormWaves = kNormBlock / 64;
constexpr float kE4M3Max = 448.0f;
constexpr float kScaleMin = 0x1p-126f;

// e4m3 bits of x (|x| <= 448 up to a rounding error), nearest even.
__device__ __forceinline__ uint8_t to_e4m3(float x)
{
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xff);
}

// ---------------------------------------------------------------------------
// Forward: one block a row, two passes over it
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
            const float scale = max_or_nan(top / kE4M3Max, kScaleMin), inv = 1.0f / scale;
            if (lane == 0) a.scales[(uint64_t)r * a.groups + g] = scale;
            for (uint32_t c = lo + lane; c < hi; c += 64) q[c] = to_e4m3(out(c) * inv);
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient: dweight's partial sums (a thread a column over a part of the
// rows), their sum, then dx (one block a row, two passes over it).  dx comes
// last: it may be dy or x.
// ---------------------------------------------------------------------------

constexpr uint32_t kGradParts = 512;    // most parts the rows are split into

template <typename T>
__global__ void __launch_bounds__(kNormBlock) ew_norm_dweight_kernel(NormGradArgs a, uint32_t parts)
{
    const uint32_t c = blockIdx.x * kNormBlock + threadIdx.x;
    if (c >= a.cols) return;
    const T *const dy = static_cast<const T *>(a.dy) + c, *const x = static_cast<const T *>(a.x) + c;
    float sum = 0.0f;
    for (uint32_t r = blockIdx.y; r < a.rows; r += parts)
        sum += (float)dy[r * a.dy_stride] * ((float)x[r * a.x_stride] * a.rstd[r]);
    a.partial[(uint64_t)blockIdx.y * a.cols + c] = sum;
}

__global__ void __launch_bounds__(kNormBlock) ew_norm_dweight_sum_kernel(NormGradArgs a, uint32_t parts)
{
    const uint32_t c = blockIdx.x * kNormBlock + threadIdx.x;
    if (c >= a.cols) return;
    float sum = 0.0f;
    for (uint32_t p = 0; p < parts; ++p) sum += a.partial[(uint64_t)p * a.cols + c];
    a.dweight[c] = sum;
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
    return (rows < kGradParts ? rows : kGradParts) * cols * sizeof(float);
}

// A row operator's kernel over `blocks` blocks, at most 2^20 (blocks stride
// over the rest).
template <class... A>
static hipError_t go(const void *fn, dim3 grid, int block, hipStream_t s, A... args)
{
    void *kargs[] = {&args...};
    return hipLaunchKernel(fn, grid, dim3(block), kargs, 0, s);
}

static uint32_t row_grid(uint32_t rows) { return rows < (1u << 20) ? rows : 1u << 20; }

#define EW_BY_TYPE(t, K)                                           \
    ((t) == kRowF32 ? reinterpret_cast<const void *>(&K<float>)    \
     : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16>) \
                      : reinterpret_cast<const void *>(&K<__bf16>))

hipError_t launch_norm(RowType t, const NormArgs &a, int, hipStream_t s, const char **path)
{
    *path = "two passes";
    return go(EW_BY_TYPE(t, ew_norm_kernel), dim3(row_grid(a.rows)), kNormBlock, s, a);
}

hipError_t launch_norm_grad(RowType t, const NormGradArgs &a, int, hipStream_t s, const char **path)
{
    *path = "two passes, dweight by columns";
    if (a.dweight) {
        const uint32_t parts = a.rows < kGradParts ? a.rows : kGradParts;
        const uint32_t blocks = (a.cols + kNormBlock - 1) / kNormBlock;
        hipError_t e = hipSuccess;
        if (parts) e = go(EW_BY_TYPE(t, ew_norm_dweight_kernel), dim3(blocks, parts), kNormBlock, s, a, parts);
        if (e != hipSuccess) return e;
        e = go(reinterpret_cast<const void *>(&ew_norm_dweight_sum_kernel), dim3(blocks), kNormBlock, s, a, parts);
        if (e != hipSuccess || a.rows == 0) return e;
    }
    return go(EW_BY_TYPE(t, ew_norm_dx_kernel), dim3(row_grid(a.rows)), kNormBlock, s, a);
}

}  // namespace ew
