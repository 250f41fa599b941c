// ew_vocab.hip -- operators over rows of logits for CDNA4 (gfx950): log
// probabilities with entropy and top alternatives, distillation from a
// teacher's top logits, and their gradients.

#include "ew_rows_device.h"

namespace ew {

constexpr int kVocabBlock = 256;
constexpr int kVocabWaves = kVocabBlock / 64;

// What a softmax over a row needs.  With m the row's largest logit (NaNs
// ignored) and d = scale * (x - m): z = sum exp(d), b = sum exp(d) * d.  The
// difference is taken before the product so that d is exactly 0 at the
// largest logit, whatever its size.  Masked logits (-inf) add nothing; a NaN
// or +inf makes z a NaN.
struct RowSum {
    float m, z, b;
};

// lse and entropy from a row's sums.  empty: the scaled logits are all -inf.
struct RowStat {
    float lse, entropy;
    bool empty;
};

__device__ __forceinline__ RowStat row_stat(const RowSum &s, float scale)
{
    RowStat st;
    const float top = s.m * scale;
    // all NaN: m stays -inf while z is a NaN
    st.empty = top == -kInf && s.z == s.z;
    const float log_z = __builtin_logf(s.z);
    st.lse = st.empty ? -kInf : top == kInf ? __builtin_nanf("") : top + log_z;
    st.entropy = st.empty ? 0.0f : st.lse != st.lse ? st.lse : log_z - s.b / s.z;
    return st;
}

// scale * x - lse of one logit, from the sums (exact where x is the largest).
__device__ __forceinline__ float log_prob(float x, const RowSum &s, const RowStat &st, float scale)
{
    if (st.empty) return -kInf;
    if (st.lse != st.lse) return st.lse;
    return (x - s.m) * scale - __builtin_logf(s.z);
}

template <typename T>
__device__ RowSum block_row_sum(const T *x, uint32_t cols, float scale, float (*scratch)[kVocabWaves])
{
    RowSum s;
    float m = -kInf;
    for (uint32_t c = threadIdx.x; c < cols; c += kVocabBlock) m = __builtin_fmaxf(m, (float)x[c]);
    s.m = block_reduce<Max, kVocabWaves>(m, scratch[0]);
    const float base = s.m == -kInf ? 0.0f : s.m;
    float z = 0.0f, b = 0.0f;
    for (uint32_t c = threadIdx.x; c < cols; c += kVocabBlock) {
        const float d = ((float)x[c] - base) * scale, e = exp_nat(d);
        z += e;
        if (e > 0.0f) b += e * d;
    }
    s.z = block_reduce<Sum, kVocabWaves>(z, scratch[1]);
    s.b = block_reduce<Sum, kVocabWaves>(b, scratch[2]);
    __syncthreads();
    return s;
}

// A logit's rank as one number: larger is more likely, ties to the lowest
// column, a NaN as -inf.  -0 and +0 rank alike.
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t c)
{
    if (x != x) x = -kInf;
    x += 0.0f;
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (uint64_t)k << 32 | (uint32_t)~c;
}

template <typename T>
__global__ void __launch_bounds__(kVocabBlock) ew_logprobs_kernel(LogprobsArgs a)
{
    __shared__ float scratch[3][kVocabWaves];
    __shared__ uint64_t best[kVocabWaves];
    for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *const x = static_cast<const T *>(a.logits) + r * a.stride;
        const RowSum s = block_row_sum(x, a.cols, a.scale, scratch);
        const RowStat st = row_stat(s, a.scale);
        if (threadIdx.x == 0) {
            const int64_t t = a.targets[r];
            const bool given = t >= 0 && t < (int64_t)a.cols;
            a.logp[r] = given ? log_prob((float)x[t], s, st, a.scale) : 0.0f;
            if (a.lse) a.lse[r] = st.lse;
            if (a.entropy) a.entropy[r] = st.entropy;
        }
        uint64_t last = ~(uint64_t)0;
        for (uint32_t k = 0; k < a.top; ++k) {
            uint64_t key = 0;
            for (uint32_t c = threadIdx.x; c < a.cols; c += kVocabBlock) {
                const uint64_t q = rank_key((float)x[c], c);
                if (q < last && q > key) key = q;
            }
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const uint64_t o = __shfl_xor((unsigned long long)key, d);
                key = o > key ? o : key;
            }
            if (threadIdx.x % 64 == 0) best[threadIdx.x / 64] = key;
            __syncthreads();
            last = best[0];
            for (int w = 1; w < kVocabWaves; ++w) last = best[w] > last ? best[w] : last;
            __syncthreads();
            if (threadIdx.x == 0) {
                const uint32_t c = ~(uint32_t)last;
                a.top_ids[(uint64_t)r * a.top + k] = c;
                a.top_logp[(uint64_t)r * a.top + k] = log_prob((float)x[c], s, st, a.scale);
            }
        }
    }
}

// p = exp(scale * x - lse), at most 1 (a difference of large numbers may
// round to above 0).
__device__ __forceinline__ float log_p(float x, float scale, float lse)
{
    return min_or_nan(__builtin_fmaf(x, scale, -lse), 0.0f);
}

template <typename T>
__global__ void __launch_bounds__(kVocabBlock) ew_logprobs_grad_kernel(LogprobsGradArgs a)
{
    for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *const x = static_cast<const T *>(a.logits) + r * a.stride;
        T *const dx = static_cast<T *>(a.dlogits) + r * a.dlogits_stride;
        const int64_t t = a.targets[r];
        const bool given = t >= 0 && t < (int64_t)a.cols;
        const float lse = a.lse[r], dlogp = given ? a.dlogp[r] : 0.0f;
        const float dent = a.dentropy ? a.dentropy[r] : 0.0f, ent = a.dentropy ? a.entropy[r] : 0.0f;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kVocabBlock) {
            const float v = (float)x[c];
            float g = 0.0f;
            if (v * a.scale != -kInf && lse != -kInf) {
                const float l = log_p(v, a.scale, lse), p = exp_nat(l);
                g = -p * (dlogp + dent * (l + ent));
                if (given && c == (uint32_t)t) g += dlogp;
                g *= a.scale;
            }
            dx[c] = (T)g;
        }
    }
}

// The teacher's distribution over its kept entries: the scaled logits'
// maximum and sum, in every thread.
struct Teacher {
    float m, z;
};

__device__ __forceinline__ bool kept_entry(int64_t id, float scaled, uint32_t cols)
{
    return id >= 0 && id < (int64_t)cols && scaled != -kInf;
}

__device__ Teacher block_teacher(const float *teacher, const int64_t *ids, uint32_t kept,
                                 uint32_t cols, float scale, float (*scratch)[kVocabWaves])
{
    Teacher t;
    float m = -kInf;
    for (uint32_t k = threadIdx.x; k < kept; k += kVocabBlock) {
        const float s = teacher[k] * scale;
        if (kept_entry(ids[k], s, cols)) m = __builtin_fmaxf(m, s);
    }
    t.m = block_reduce<Max, kVocabWaves>(m, scratch[0]);
    float z = 0.0f;
    for (uint32_t k = threadIdx.x; k < kept; k += kVocabBlock) {
        const float s = teacher[k] * scale;
        if (kept_entry(ids[k], s, cols)) z += exp_nat(s - t.m);
    }
    t.z = block_reduce<Sum, kVocabWaves>(z, scratch[1]);
    __syncthreads();
    return t;
}

template <typename T>
__global__ void __launch_bounds__(kVocabBlock) ew_distill_kernel(DistillArgs a)
{
    __shared__ float scratch[3][kVocabWaves];
    for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *const x = static_cast<const T *>(a.logits) + r * a.stride;
        const float *const teacher = a.teacher + (uint64_t)r * a.kept;
        const int64_t *const ids = a.ids + (uint64_t)r * a.kept;
        const RowSum s = block_row_sum(x, a.cols, a.scale, scratch);
        const RowStat st = row_stat(s, a.scale);
        const Teacher t = block_teacher(teacher, ids, a.kept, a.cols, a.scale, scratch);
        const float log_tz = __builtin_logf(t.z);
        float loss = 0.0f;
        for (uint32_t k = threadIdx.x; k < a.kept; k += kVocabBlock) {
            const float v = teacher[k] * a.scale;
            if (!kept_entry(ids[k], v, a.cols)) continue;
            const float l = v - t.m - log_tz, p = exp_nat(v - t.m) / t.z;
            if (p >= 0x1p-126f || p != p) loss += p * (l - log_prob((float)x[ids[k]], s, st, a.scale));
        }
        loss = block_reduce<Sum, kVocabWaves>(loss, scratch[2]);
        if (threadIdx.x == 0) {
            a.loss[r] = loss;
            if (a.lse) a.lse[r] = st.lse;
        }
        __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(kVocabBlock) ew_distill_grad_kernel(DistillGradArgs a)
{
    __shared__ float scratch[2][kVocabWaves];
    for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T *const x = static_cast<const T *>(a.logits) + r * a.stride;
        T *const dx = static_cast<T *>(a.dlogits) + r * a.dlogits_stride;
        const float *const teacher = a.teacher + (uint64_t)r * a.kept;
        const int64_t *const ids = a.ids + (uint64_t)r * a.kept;
        const Teacher t = block_teacher(teacher, ids, a.kept, a.cols, a.scale, scratch);
        const float lse = a.lse[r], g = t.z == 0.0f ? 0.0f : a.dloss[r] * a.scale;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kVocabBlock) {
            const float v = (float)x[c];
            float d = 0.0f;
            if (v * a.scale != -kInf && lse != -kInf && t.z != 0.0f) {
                float q = 0.0f;
                for (uint32_t k = 0; k < a.kept; ++k) {
                    const float s = teacher[k] * a.scale;
                    if (ids[k] == (int64_t)c && kept_entry(ids[k], s, a.cols))
                        q += exp_nat(s - t.m) / t.z;
                }
                d = g * (exp_nat(log_p(v, a.scale, lse)) - q);
            }
            dx[c] = (T)d;
        }
    }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

size_t logprobs_workspace(uint64_t, uint64_t, uint64_t) { return 0; }
size_t distill_workspace(uint64_t, uint64_t) { return 0; }

#define EW_BY_TYPE(t, K)                                           \
    ((t) == kRowF32 ? reinterpret_cast<const void *>(&K<float>)    \
     : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16>) \
                      : reinterpret_cast<const void *>(&K<__bf16>))

template <class A>
static hipError_t go(const void *fn, const A &args, hipStream_t s)
{
    A a = args;
    void *kargs[] = {&a};
    const uint32_t grid = a.rows < (1u << 20) ? a.rows : 1u << 20;
    return hipLaunchKernel(fn, dim3(grid), dim3(kVocabBlock), kargs, 0, s);
}

hipError_t launch_logprobs(RowType t, const LogprobsArgs &a, int, hipStream_t s, const char **path)
{
    *path = "a block a row";
    return go(EW_BY_TYPE(t, ew_logprobs_kernel), a, s);
}

hipError_t launch_logprobs_grad(RowType t, const LogprobsGradArgs &a, int, hipStream_t s,
                                const char **path)
{
    *path = "a block a row";
    return go(EW_BY_TYPE(t, ew_logprobs_grad_kernel), a, s);
}

hipError_t launch_distill(RowType t, const DistillArgs &a, int, hipStream_t s, const char **path)
{
    *path = "a block a row";
    return go(EW_BY_TYPE(t, ew_distill_kernel), a, s);
}

hipError_t launch_distill_grad(RowType t, const DistillGradArgs &a, int, hipStream_t s,
                               const char **path)
{
    *path = "a block a row";
    return go(EW_BY_TYPE(t, ew_distill_grad_kernel), a, s);
}

}  // namespace ew
