// ew_rows_vec.h -- rows as 16-byte vectors from the row's start, whatever its
// alignment and length: loads and stores whose last vector may be a part, and
// launches (ew_layernorm.hip, ew_policy.hip, ew_experts.hip).  Not installed;
// not part of the C ABI.
#pragma once

#include "ew_rows_device.h"

namespace ew {

template <bool C, class A, class B>
struct Conditional {
    using type = A;
};
template <class A, class B>
struct Conditional<false, A, B> {
    using type = B;
};

// A vector's elements without the first n (0 < n < its number), 0 behind them.
template <typename T>
__device__ __forceinline__ u32x4 drop_first(u32x4 v, uint32_t n)
{
    const uint32_t bits = n * 8 * (uint32_t)sizeof(T);
    uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    if (bits >= 64) {
        lo = hi >> (bits - 64);
        hi = 0;
    } else {
        lo = lo >> bits | hi << (64 - bits);
        hi >>= bits;
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// The vector of a row of cols elements from element `at` on, 0 past the row.
// Its last, partial one is read as the last whole 16 bytes of the row and
// shifted (`settle`, apart so that loads can be on their way together): the
// elements one by one, each waited for, cost 0.5-2 us a row.  Nt: a stream
// read once, else data that other rows read too.  Short: a row below 2^32 bytes.
template <typename T, bool Nt, bool Short = false>
__device__ __forceinline__ u32x4 load_vec(const T *row, uint32_t cols, uint32_t at)
{
    constexpr uint32_t N = Vec<T>::N;
    if (at >= cols) return u32x4{0, 0, 0, 0};
    if (cols < N) {
        typename Vec<T>::type t{};
#pragma unroll
        for (uint32_t j = 0; j < N; ++j)
            if (j < cols) t[j] = row[j];
        return __builtin_bit_cast(u32x4, t);
    }
    // (Short: one register of offset to a row that is the same in all lanes)
    using Offset = typename Conditional<Short, uint32_t, uint64_t>::type;
    const char *const p = reinterpret_cast<const char *>(row) +
                          (Offset)(at + N <= cols ? at : cols - N) * (Offset)sizeof(T);
    if constexpr (Nt) return load16<false, sizeof(T)>(p);
    else if constexpr (sizeof(T) == 4) return *reinterpret_cast<const u32x4_a4 *>(p);
    else return *reinterpret_cast<const u32x4_a2 *>(p);
}

template <typename T>
__device__ __forceinline__ u32x4 settle(u32x4 v, uint32_t cols, uint32_t at)
{
    constexpr uint32_t N = Vec<T>::N;
    if (at < cols && at + N > cols && cols >= N) return drop_first<T>(v, at + N - cols);
    return v;
}

template <typename T, bool Short = false>
__device__ __forceinline__ void store_vec(T *row, uint32_t cols, uint32_t at, u32x4 v)
{
    constexpr uint32_t N = Vec<T>::N;
    using Offset = typename Conditional<Short, uint32_t, uint64_t>::type;
    if (at + N <= cols) {
        store16_row<T>(reinterpret_cast<char *>(row) + (Offset)at * (Offset)sizeof(T), v);
    } else if (at < cols) {
        const typename Vec<T>::type t = __builtin_bit_cast(typename Vec<T>::type, v);
#pragma unroll
        for (uint32_t j = 0; j < N; ++j)
            if (at + j < cols) row[at + j] = t[j];
    }
}

// The value of another lane of the same 16 (binary64).
template <int Ctrl>
__device__ __forceinline__ double dpp64(double x)
{
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const int lo = (int)(uint32_t)v, hi = (int)(uint32_t)(v >> 32);
    const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, Ctrl, 0xf, 0xf, true);
    const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, Ctrl, 0xf, 0xf, true);
    return __builtin_bit_cast(double, l | (uint64_t)h << 32);
}

__device__ __forceinline__ double lane_value64(double x, int lane)
{
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint32_t l = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t h = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return __builtin_bit_cast(double, l | (uint64_t)h << 32);
}

// Sum over the 64 lanes of a wave in every lane (as wave_reduce).
__device__ __forceinline__ double wave_sum64(double x)
{
    x += dpp64<0xB1>(x);
    x += dpp64<0x4E>(x);
    x += dpp64<0x141>(x);
    x += dpp64<0x140>(x);
    return (lane_value64(x, 0) + lane_value64(x, 16)) + (lane_value64(x, 32) + lane_value64(x, 48));
}

// Blocks stride over what is beyond this many.
constexpr uint64_t kMaxBlocks = 1 << 20;

inline uint32_t row_blocks(uint64_t blocks)
{
    return (uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
}

template <class... A>
hipError_t start(const void *fn, dim3 grid, uint32_t block, size_t lds, hipStream_t s, A... args)
{
    void *kargs[] = {&args...};
    return hipLaunchKernel(fn, grid, dim3(block), kargs, lds, s);
}

// Vectors of a row of cols elements.
inline uint32_t vectors_of(RowType t, uint32_t cols)
{
    const uint32_t n = 16 / (uint32_t)row_elem_size(t);
    return cols / n + (cols % n != 0);
}

#define EW_KERNEL_OF(t, K)                                           \
    ((t) == kRowF32 ? reinterpret_cast<const void *>(&K<float>)      \
     : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16>) \
                      : reinterpret_cast<const void *>(&K<__bf16>))

}  // namespace ew
