// ew_rows_vec.h -- rows as 16-byte vectors whatever their alignment and length,
// sums in binary64 and launches, for ew_layernorm.hip, ew_policy.hip and
// ew_experts.hip.  Not installed; not part of the C ABI.
#pragma once

#include "ew_rows_device.h"

namespace ew {

// What is known of a row's vectors: all are whole; the last may be a part; the
// row is shorter than one.
enum RowFit : int { kWhole = 0, kPart, kTiny };

// Where a vector of a row of cols elements lies: element `first` of the row on,
// N of them.  A row's vectors start at its start, one behind another; its last,
// partial one is taken as the last N elements of the row instead, of which the
// first `skip` are the vector's before it.  Loads and stores are so of 16 bytes
// everywhere (elements one by one, each waited for, cost 0.5-2 us a row); both
// vectors hold, compute and store the same there, and only sums and stores of
// what depends on an output's old value leave out what is not their own.
// A tiny row is one piece with zeros behind the row.
template <typename T, RowFit Fit>
struct Piece {
    static constexpr uint32_t N = Vec<T>::N;
    uint32_t first, skip;
    bool live;
    // back: elements of the row before element 0 of the stretch
    __device__ Piece(uint32_t at, uint32_t cols, uint32_t back = 0)
        : first(back + (Fit != kPart || at + N <= cols ? at : cols - N)), skip(back + at - first),
          live(Fit == kWhole || at < cols)
    {
    }
    // whether element j of a live piece is its own
    __device__ bool own(uint32_t j, uint32_t cols) const
    {
        return Fit == kWhole || (Fit == kTiny ? j < cols : j >= skip);
    }
};

// Loads and stores of a piece; `row` is best the same in all lanes, whose
// offsets are of 32 bits then.  A stretch of a row far below 2^32 bytes.
// Nt: a stream read once, else data that others read too.
template <typename T, bool Nt, RowFit Fit>
__device__ __forceinline__ u32x4 load_piece(const T *row, uint32_t cols, const Piece<T, Fit> &p)
{
    if (!p.live) return u32x4{0, 0, 0, 0};
    if constexpr (Fit == kTiny) {
        typename Vec<T>::type t{};
#pragma unroll
        for (uint32_t j = 0; j < Vec<T>::N; ++j)
            if (j < cols) t[j] = row[j];
        return __builtin_bit_cast(u32x4, t);
    }
    const char *const at = reinterpret_cast<const char *>(row) + p.first * (uint32_t)sizeof(T);
    if constexpr (Nt) return load16<false, sizeof(T)>(at);
    else if constexpr (sizeof(T) == 4) return *reinterpret_cast<const u32x4_a4 *>(at);
    else return *reinterpret_cast<const u32x4_a2 *>(at);
}

template <typename T, RowFit Fit>
__device__ __forceinline__ void store_piece(T *row, uint32_t cols, const Piece<T, Fit> &p, u32x4 v)
{
    if (!p.live) return;
    if constexpr (Fit == kTiny) {
        const typename Vec<T>::type t = __builtin_bit_cast(typename Vec<T>::type, v);
#pragma unroll
        for (uint32_t j = 0; j < Vec<T>::N; ++j)
            if (j < cols) row[j] = t[j];
    } else {
        store16_row<T>(reinterpret_cast<char *>(row) + p.first * (uint32_t)sizeof(T), v);
    }
}

// The elements of a piece that are its own, one by one where those are not all.
template <typename T, RowFit Fit>
__device__ __forceinline__ void store_own(T *row, uint32_t cols, const Piece<T, Fit> &p, u32x4 v)
{
    if (Fit != kPart || p.skip == 0) return store_piece(row, cols, p, v);
    const typename Vec<T>::type t = __builtin_bit_cast(typename Vec<T>::type, v);
#pragma unroll
    for (uint32_t j = 0; j < Vec<T>::N; ++j)
        if (p.live && j >= p.skip) row[p.first + j] = t[j];
}

// The bits of v that are a piece's own, 0 elsewhere.
template <typename T, RowFit Fit>
__device__ __forceinline__ u32x4 own_bits(u32x4 v, uint32_t cols, const Piece<T, Fit> &p)
{
    if constexpr (Fit == kPart) {
        constexpr uint32_t kPerWord = 4 / (uint32_t)sizeof(T);
#pragma unroll
        for (uint32_t w = 0; w < 4; ++w) {
            uint32_t bits = 0;
#pragma unroll
            for (uint32_t h = 0; h < kPerWord; ++h)
                if (p.own(w * kPerWord + h, cols))
                    bits |= (kPerWord == 1 ? 0xffffffffu : 0xffffu) << (16 * h);
            v[w] &= bits;
        }
    }
    return v;             // (a tiny row's and dead pieces' others are 0)
}

// The piece at element `at` of a row of any length: element `first` of the row
// on, with offsets of 64 bits.
template <typename T, RowFit Fit = kPart>
struct LongPiece {
    uint64_t first;
    uint32_t cols;
    Piece<T, Fit> p;           // of the vector at `first`, a row of its own
    __device__ LongPiece(uint32_t at, uint32_t cols_)
        : first(Fit == kTiny || at + Vec<T>::N <= cols_ ? at : cols_ - Vec<T>::N), cols(cols_),
          p(0, Fit == kTiny ? cols_ : Vec<T>::N)
    {
        p.skip = at - (uint32_t)first;
    }
    template <bool Nt>
    __device__ u32x4 load(const T *row) const { return load_piece<T, Nt>(row + first, cols, p); }
    // (an output may be an input, whose other elements are another thread's)
    __device__ void store(T *row, u32x4 v) const { store_own(row + first, cols, p, v); }
};

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
