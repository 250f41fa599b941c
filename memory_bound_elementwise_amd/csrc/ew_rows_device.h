// ew_rows_device.h -- device-side building blocks of the row operators
// (gfx950): element types, reductions over a wave and a block, and the
// running statistics of a softmax.  Not installed; not part of the C ABI.
#pragma once

#include "ew_device.h"
#include "ew_rows_args.h"

namespace ew {

constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

// max(a, b), a NaN if either is one (the hardware's plain maximum returns the
// other operand).
__device__ __forceinline__ float max_or_nan(float a, float b)
{
    return __builtin_elementwise_maximum(a, b);
}

struct Sum {
    __device__ static float f(float a, float b) { return a + b; }
};
struct Max {        // ignores NaNs
    __device__ static float f(float a, float b) { return __builtin_fmaxf(a, b); }
};

struct MaxOrNan {
    __device__ static float f(float a, float b) { return max_or_nan(a, b); }
};

// The value of another lane of the same 16: dpp control word Ctrl.
template <int Ctrl>
__device__ __forceinline__ float dpp(float x)
{
    const int v = __builtin_bit_cast(int, x);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(v, v, Ctrl, 0xf, 0xf, true));
}

__device__ __forceinline__ float lane_value(float x, int lane)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// R over each four neighbouring lanes, in each of them.
template <class R>
__device__ __forceinline__ float quad_reduce(float x)
{
    x = R::f(x, dpp<0xB1>(x));
    return R::f(x, dpp<0x4E>(x));
}

// R over the 64 lanes of a wave, in every lane; all lanes must be active.
// Within each row of 16 by lane exchanges (xor 1, xor 2, then mirrors of 8
// and 16, which after the first two steps hold the other half's value), then
// the four rows through scalar registers.
template <class R>
__device__ __forceinline__ float wave_reduce(float x)
{
    x = quad_reduce<R>(x);
    x = R::f(x, dpp<0x141>(x));
    x = R::f(x, dpp<0x140>(x));
    return R::f(R::f(lane_value(x, 0), lane_value(x, 16)),
                R::f(lane_value(x, 32), lane_value(x, 48)));
}

// R over a block of Waves waves, in every thread.  scratch: Waves floats of
// LDS that no other reduction uses until the block's next barrier.
template <class R, int Waves>
__device__ __forceinline__ float block_reduce(float x, float *scratch)
{
    x = wave_reduce<R>(x);
    if constexpr (Waves > 1) {
        if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64] = x;
        __syncthreads();
        x = scratch[0];
#pragma unroll
        for (int w = 1; w < Waves; ++w) x = R::f(x, scratch[w]);
    }
    return x;
}

// ---------------------------------------------------------------------------
// Vectors: the 16-byte vector of an element type and its widening
// ---------------------------------------------------------------------------

template <typename T>
struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);        // elements
    typedef T type __attribute__((ext_vector_type(N)));
    typedef float wide __attribute__((ext_vector_type(N)));
    __device__ static wide widen(u32x4 v)
    {
        return __builtin_convertvector(__builtin_bit_cast(type, v), wide);
    }
    __device__ static u32x4 narrow(wide v)               // nearest even
    {
        return __builtin_bit_cast(u32x4, __builtin_convertvector(v, type));
    }
    // every element -inf
    __device__ static u32x4 masked()
    {
        const uint32_t w = sizeof(T) == 4 ? 0xff800000u
                           : __is_same(T, __bf16) ? 0xff80ff80u : 0xfc00fc00u;
        return u32x4{w, w, w, w};
    }
};

// Store a vector of T that is only element aligned.
template <typename T>
__device__ __forceinline__ void store16_row(char *p, u32x4 v)
{
    if constexpr (sizeof(T) == 4) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a4 *>(p));
    else __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2 *>(p));
}

// How a row of n elements starting at p splits: `head` elements up to the
// first 16-byte boundary, `vectors` aligned vectors, `tail` elements.
template <typename T>
struct RowSplit {
    uint32_t head, vectors, tail;
    __device__ RowSplit(const T *p, uint32_t n)
    {
        const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) % 16);
        head = (off ? 16 - off : 0) / (uint32_t)sizeof(T);
        if (head > n) head = n;
        vectors = (n - head) / Vec<T>::N;
        tail = n - head - vectors * Vec<T>::N;
    }
};

// exp(x) through the hardware's power of two: relative error about
// |x| * 2^-24, of either sign (the arguments of a softmax are x <= 0, log ratios
// any).
__device__ __forceinline__ float exp_nat(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

}  // namespace ew
