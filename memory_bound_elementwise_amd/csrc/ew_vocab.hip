// ew_vocab.hip -- operators over rows of logits for CDNA4 (gfx950): log
// probabilities with entropy and top alternatives, distillation from a
// teacher's top logits, and their gradients.

#include "ew_rows_device.h"

#include <type_traits>

namespace ew {

constexpr int kVocabBlock = 256;
constexpr int kVocabWaves = kVocabBlock / 64;

// ---------------------------------------------------------------------------
// Softmax statistics of a row
// ---------------------------------------------------------------------------

// With m the largest logit seen (NaNs ignored), c = scale * log2(e) and d(x)
// the distance of x from m in powers of two (below): z = sum 2^d, b = sum
// 2^d * d.  Masked logits (-inf) add nothing; a NaN or +inf makes z a NaN.
struct RowSum {
    float m, z, b;
};

// Where a difference of exponents is -inf its term is 0; this finite stand-in
// keeps 0 * d from being a NaN, times a sum of 2^31 terms too, and 2^d is 0
// all the same.
constexpr float kFarBelow = -1e4f;

// d(x) is c * x - t with t = c * m rounded: the product and difference in one
// fma, rounded once, and the sums are relative to 2^t, whatever the rounding
// of t.  Where |t| is past kNear its rounding would be larger than the
// differences that matter (a row of one large number must give d = 0, not the
// error of t), so there d(x) is c * (x - m) and the sums are relative to c * m
// itself.  A sum that moves from one base to another takes the roundings of
// both along.  t is the same number wherever it is used: the functions that
// form it leave its product alone (contract off).
constexpr float kNear = 0x1p16f;

// c * x is unit * x, exact, times c: in two factors where the product of scale
// and log2(e) overflows (scales above 2.36e38), and of halves where the
// difference of two logits may overflow though c times it does not come to
// -infinity (scales below kTinyScale).
struct Rate {
    float c, unit;
    __device__ explicit Rate(float scale)
        : c(scale * kLog2e), unit(1.0f)
    {
        if (c == kInf) c = 0.5f * scale * kLog2e, unit = 2.0f;
        if (scale < kTinyScale) c *= 2.0f, unit = 0.5f;
    }
};

// unit * m, kept finite from below: where m is -inf, or times c is anyway, all
// distances come out as -inf.
__device__ __forceinline__ float unit_base(float m, Rate k)
{
    return __builtin_fmaxf(m * k.unit, -__FLT_MAX__);
}

// What d(x) = c * (unit * x - far) - near is formed with, for a largest logit m:
// near is t, or far is unit * m.
struct Base {
    float near, far;
    __device__ Base(float m, Rate k)
    {
#pragma clang fp contract(off)
        const float u = unit_base(m, k), t = u * k.c;
        const bool is_near = __builtin_fabsf(t) <= kNear;
        near = is_near ? t : 0.0f;
        far = is_near ? 0.0f : u;
    }
    __device__ float distance(float x, Rate k) const
    {
        return __builtin_fmaf(__builtin_fmaf(x, k.unit, -far), k.c, -near);
    }
};

// c * m minus the base of sums whose largest logit is m.
__device__ __forceinline__ float base_rounding(float m, Rate k)
{
#pragma clang fp contract(off)
    const float u = unit_base(m, k), t = u * k.c;
    return __builtin_fabsf(t) <= kNear ? __builtin_fmaf(u, k.c, -t) : 0.0f;
}

// s re-based from s.m to m >= s.m.
template <bool Ent>
__device__ __forceinline__ void rebase(RowSum &s, float m, Rate k)
{
#pragma clang fp contract(off)
    const float d = __builtin_fmaf(s.m, k.unit, -unit_base(m, k)) * k.c +
                    (base_rounding(m, k) - base_rounding(s.m, k));
    const float shift = __builtin_fmaxf(d, kFarBelow), f = __builtin_amdgcn_exp2f(shift);
    if constexpr (Ent) s.b = f * __builtin_fmaf(shift, s.z, s.b);
    s.z *= f;
    s.m = m;
}

template <int N>
__device__ __forceinline__ float largest(const float (&v)[N])
{
    float top = v[0];
#pragma unroll
    for (int k = 1; k < N; ++k) top = __builtin_fmaxf(top, v[k]);   // three operands each
    return top;
}

// N more logits of this lane, whatever they are.  Their largest is found by
// comparisons: the hardware's maximum ignores a quiet NaN but drops its other
// operand for a signalling one (which widening 16-bit data does not quiet).
template <bool Ent, int N>
__device__ __forceinline__ void absorb_any(RowSum &s, const float (&v)[N], Rate rate)
{
    float m = s.m;
    asm("" : "+v"(m));       // no value the compiler knows, or it makes a maximum of these
#pragma unroll
    for (int k = 0; k < N; ++k) m = v[k] > m ? v[k] : m;
    rebase<Ent>(s, m, rate);
    const Base base(s.m, rate);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float d = base.distance(v[k], rate), e = __builtin_amdgcn_exp2f(d);
        s.z += e;
        if constexpr (Ent) s.b = __builtin_fmaf(e, __builtin_fmaxf(d, kFarBelow), s.b);
    }
}

// The same in fewer instructions, for logits and an s of ordinary size (or an
// empty s), no NaN among them and, with entropy, none masked: returns whether
// the logits were so for this lane (s is of no use otherwise).  16-bit rows
// are bound by the vector unit: an element costs its widening, half a maximum,
// an fma, a power, an addition and, with entropy, another fma.
template <bool Ent, int N>
__device__ __forceinline__ bool absorb_plain(RowSum &s, const float (&v)[N], float c)
{
#pragma clang fp contract(off)
    const float m = __builtin_fmaxf(s.m, largest(v));
    const float t = m == -kInf ? 0.0f : m * c;
    const float shift = __builtin_fmaxf(s.m * c - t, kFarBelow);
    const float f = __builtin_amdgcn_exp2f(shift);
    if constexpr (Ent) s.b = f * __builtin_fmaf(shift, s.z, s.b);
    s.z *= f;
    s.m = m;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float d = __builtin_fmaf(v[k], c, -t), e = __builtin_amdgcn_exp2f(d);
        s.z += e;
        if constexpr (Ent) s.b = __builtin_fmaf(e, d, s.b);
    }
    const float sum = Ent ? s.b : s.z;
    return __builtin_fabsf(t) <= kNear && sum == sum;
}

// The sums of the wave's lanes, in every lane.
template <bool Ent>
__device__ __forceinline__ void wave_join(RowSum &s, Rate k)
{
    rebase<Ent>(s, wave_reduce<Max>(s.m), k);
    s.z = wave_reduce<Sum>(s.z);
    if constexpr (Ent) s.b = wave_reduce<Sum>(s.b);
}

// The sums of the block's threads, in every thread; one barrier.
template <bool Ent>
__device__ __forceinline__ void block_join(RowSum &s, Rate k, RowSum *part)
{
    wave_join<Ent>(s, k);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = s;
    __syncthreads();
    // each four lanes hold the four waves' sums: one re-basing in all
    static_assert(kVocabWaves == 4, "the exchanges below are within four lanes");
    s = part[threadIdx.x % kVocabWaves];
    rebase<Ent>(s, quad_reduce<Max>(s.m), k);
    s.z = quad_reduce<Sum>(s.z);
    if constexpr (Ent) s.b = quad_reduce<Sum>(s.b);
}

// lse and entropy from a row's sums.  empty: the scaled logits are all -inf.
// log_z is relative to the sums' base, lse rounded once from the largest logit
// itself.
struct RowStat {
    float lse, entropy, log_z;
    bool empty;
};

__device__ __forceinline__ RowStat row_stat(const RowSum &s, float scale)
{
    RowStat st;
    const float top = s.m * scale;
    // all NaN: m stays -inf while z is a NaN
    st.empty = top == -kInf && s.z == s.z;
    st.log_z = __builtin_logf(s.z);
    const float past = __builtin_fmaf(-kLn2, base_rounding(s.m, Rate(scale)), st.log_z);
    st.lse = st.empty ? -kInf : top == kInf ? __builtin_nanf("") : __builtin_fmaf(s.m, scale, past);
    st.entropy = st.empty ? 0.0f
                 : st.lse != st.lse ? st.lse : __builtin_fmaf(-kLn2, s.b / s.z, st.log_z);
    return st;
}

// scale * x - lse of one logit, from the sums (-log z where x is the largest).
__device__ __forceinline__ float log_prob(float x, const RowSum &s, const RowStat &st, float scale)
{
    if (st.empty) return -kInf;
    if (st.lse != st.lse) return st.lse;
    const Rate k(scale);
    const float d = Base(s.m, k).distance(x, k);
    // far away (where d, and x - m, may overflow though their product with
    // scale does not) the rounding of t no longer matters
    return d < -kNear ? (0.5f * x - 0.5f * s.m) * scale * 2.0f - st.log_z
                      : __builtin_fmaf(d, kLn2, -st.log_z);
}

// ---------------------------------------------------------------------------
// The largest logits of a row
// ---------------------------------------------------------------------------

// A logit as a number that orders as it does (-0 as +0, a NaN as -inf), and
// back.
__device__ __forceinline__ uint32_t order(float x)
{
    if (x != x) x = -kInf;
    x += 0.0f;
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_logit(uint32_t k)
{
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kOrderMasked = 0x007fffffu;      // order(-inf)

// A logit's rank as one number: larger is more likely, ties to the lowest
// column.  Never 0.
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t col)
{
    return (uint64_t)order(x) << 32 | (uint32_t)~col;
}
__device__ __forceinline__ float key_logit(uint64_t key) { return order_logit((uint32_t)(key >> 32)); }
__device__ __forceinline__ uint32_t key_col(uint64_t key) { return ~(uint32_t)key; }

__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)k, lane);
}

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// What this wave's lanes wrote to LDS is visible to its other lanes.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A number that at least k (1..64) of the lanes' orders are at or above, and
// hardly below the k-th largest of them: each lane's order with its last six
// bits replaced by the lane, which makes them different, is counted against
// all others.
__device__ __forceinline__ uint32_t lanes_kth(uint32_t own, uint32_t k)
{
    own = (own & ~63u) | (63 - threadIdx.x % 64);
    uint32_t above = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i)
        above += (uint32_t)__builtin_amdgcn_readlane((int)own, i) > own;
    const int at = __builtin_ctzll(__ballot(above == k - 1));
    return (uint32_t)__builtin_amdgcn_readlane((int)own, at) & ~63u;
}

// One wave's candidates for the k largest keys: an unordered list in LDS that
// holds every key offered above the bar, at least the k largest of them.  A
// list that grows too long is cut to its k largest, and the smallest of
// those becomes the bar.
constexpr uint32_t kListKeys = 256;

struct TopList {
    uint64_t *keys;      // kListKeys of LDS, this wave's
    uint32_t count, k;   // the same in every lane, as is the bar
    uint64_t bar;

    // A value with exactly k keys at or above it is found bit by bit.
    __device__ void cut()
    {
        wave_sync();
        const uint32_t lane = threadIdx.x % 64;
        uint64_t own[kListKeys / 64];
#pragma unroll
        for (uint32_t i = 0; i < kListKeys / 64; ++i)
            own[i] = i * 64 + lane < count ? keys[i * 64 + lane] : 0;
        uint64_t at = 0;
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t trial = at | (uint64_t)1 << bit;
            uint32_t n = 0;
#pragma unroll
            for (uint32_t i = 0; i < kListKeys / 64; ++i)
                n += __builtin_popcountll(__ballot(own[i] >= trial));
            if (n >= k) at = trial;
            if (n == k) break;
        }
        count = 0;
        bar = ~(uint64_t)0;
#pragma unroll
        for (uint32_t i = 0; i < kListKeys / 64; ++i) {
            const bool stay = own[i] >= at;
            const uint64_t mask = __ballot(stay);
            if (stay) {
                keys[count + lanes_below(mask)] = own[i];
                bar = own[i] < bar ? own[i] : bar;
            }
            count += __builtin_popcountll(mask);
        }
        wave_sync();
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint64_t o = __shfl_xor((unsigned long long)bar, d);
            bar = o < bar ? o : bar;
        }
        bar = lane_key(bar, 0);
    }

    // Each lane offers one key (0: none).
    __device__ void offer(uint64_t key)
    {
        const bool enter = key > bar;
        const uint64_t mask = __ballot(enter);
        if (mask == 0) return;
        if (enter) keys[count + lanes_below(mask)] = key;
        count += __builtin_popcountll(mask);
        if (count > kListKeys - 64) cut();
    }
};

struct TopShared {
    uint64_t keys[kVocabWaves][kListKeys];
    uint64_t best[64];
    uint32_t counts[kVocabWaves], bars[kVocabWaves];
    uint8_t lanes[kVocabWaves][64];
};

// The k largest keys of all waves' lists, best first: the first wave's lane i
// returns the i-th (0 past their number).  Every wave calls it; two barriers.
// Each key counts the keys above it.
__device__ __forceinline__ uint64_t block_top(TopList &list, TopShared &sh)
{
    const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    if (list.count > 63) list.cut();
    if (lane == 0) {
        sh.counts[wave] = list.count;
        list.keys[list.count] = 0;             // pairs are read below
    }
    if (wave == 0) sh.best[lane] = 0;
    __syncthreads();
    const uint64_t key = lane < list.count ? list.keys[lane] : 0;
    uint32_t above = 0;
#pragma unroll
    for (int w = 0; w < kVocabWaves; ++w) {
        const uint32_t n = sh.counts[w];
#pragma unroll 4
        for (uint32_t i = 0; i < n; i += 2) {
            const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(&sh.keys[w][i]);
            above += (two.x > key) + (two.y > key);
        }
    }
    if (key != 0 && above < list.k) sh.best[above] = key;
    __syncthreads();
    return wave == 0 ? sh.best[lane] : 0;
}

// ---------------------------------------------------------------------------
// One pass over a row, or over one of its parts
// ---------------------------------------------------------------------------

// Elements a lane takes at a time: two 16-byte vectors of 16-bit logits, four
// of 32-bit ones.
constexpr int kPerLane = 16;

// The columns of part `part` of `parts` of a row: a range of its aligned
// vectors; the first part has the head too, the last the tail.
struct Part {
    uint32_t lo, hi;
    bool first, last;
    __device__ Part(uint32_t vectors, uint32_t part, uint32_t parts)
    {
        // whole kilobytes each, so that no two parts share a cache line
        const uint32_t each = ((vectors + parts - 1) / parts + 63) & ~63u;
        const uint64_t start = (uint64_t)each * part;
        lo = start < vectors ? (uint32_t)start : vectors;
        hi = vectors - lo < each ? vectors : lo + each;
        first = part == 0;
        last = part + 1 == parts;
    }
};

// The next vectors are on their way while the lane's last ones are added up.
// 4096 x 131072 bf16: reading alone, in this pattern, takes 157 us (151 at
// best, with blocks of 1024 threads, whose few rows at a time leave the ends
// of rows uncovered).
template <typename T, bool Ent>
__device__ __forceinline__ RowSum stream_part(const T *x, uint32_t cols, const Part &p,
                                              const RowSplit<T> &split, Rate k)
{
    constexpr int N = Vec<T>::N, U = kPerLane / N;
    constexpr uint32_t kStep = kVocabBlock * U;
    const char *const body = reinterpret_cast<const char *>(x + split.head);
    RowSum s{-kInf, 0.0f, 0.0f};

    u32x4 next[U];
    const auto fetch = [&](uint32_t v) {       // v: the block's first vector
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = v + threadIdx.x + u * kVocabBlock;
            if (i < p.hi) next[u] = load16<true, sizeof(T)>(body + (uint64_t)i * 16);
        }
    };
    fetch(p.lo);
    // up to a vector's elements before and after the aligned body: one lane each
    if (threadIdx.x < split.head && p.first) {
        const float v[1] = {(float)x[threadIdx.x]};
        absorb_any<Ent>(s, v, k);
    }
    if (threadIdx.x < split.tail && p.last) {
        const float v[1] = {(float)x[cols - split.tail + threadIdx.x]};
        absorb_any<Ent>(s, v, k);
    }
    // until the wave meets logits that are not (the head's and tail's first)
    bool plain = k.unit == 1.0f && __ballot(s.m != -kInf && __builtin_fabsf(s.m * k.c) > kNear) == 0;
    uint32_t v = p.lo;
    for (; p.hi - v >= kStep; v += kStep) {
        float f[kPerLane];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const typename Vec<T>::wide w = Vec<T>::widen(next[u]);
#pragma unroll
            for (int j = 0; j < N; ++j) f[u * N + j] = w[j];
        }
        fetch(v + kStep);
        if (plain) {
            RowSum more = s;
            plain = __ballot(!absorb_plain<Ent>(more, f, k.c)) == 0;
            if (plain) s = more;
        }
        if (!plain) absorb_any<Ent>(s, f, k);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (v + threadIdx.x + u * kVocabBlock < p.hi) {
            const typename Vec<T>::wide w = Vec<T>::widen(next[u]);
            float f[N];
#pragma unroll
            for (int j = 0; j < N; ++j) f[j] = w[j];
            absorb_any<Ent>(s, f, k);
        }
    }
    return s;
}

// The part's `top` largest logits.  The stream has left each lane the largest
// of its own (lane_top); at least `top` logits are at or above the top-th
// largest of a wave's 64, so that the highest of the waves' is a bar that few
// more than `top` logits pass, and only lanes whose largest passes it hold
// any: all their vectors are read again.  Eight lanes share a cache line, so
// that is a third of the row at 5 alternatives, nearly all of it from 20 on
// (2048 x 50257 bf16, of 206 MB: 276 MB read at 5, 390 at 20, 411 at 32).
// Where fewer lanes than that have a logit that is not masked the bar is -inf:
// then every such logit is taken, and the lowest masked columns after them.
template <typename T>
__device__ __forceinline__ uint64_t part_top(const T *x, uint32_t cols, const Part &p,
                                             const RowSplit<T> &split, float lane_top,
                                             uint32_t top, TopShared &sh)
{
    constexpr uint32_t N = Vec<T>::N;
    const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const uint32_t kth = lanes_kth(order(lane_top), top);
    if (lane == 0) sh.bars[wave] = kth;
    __syncthreads();
    uint32_t bar = sh.bars[0];
#pragma unroll
    for (int w = 1; w < kVocabWaves; ++w) bar = sh.bars[w] > bar ? sh.bars[w] : bar;
    bar = __builtin_amdgcn_readfirstlane(bar);
    const bool masked = bar <= kOrderMasked;
    TopList list{sh.keys[wave], 0, top, masked ? (uint64_t)kOrderMasked << 32 | ~0u
                                               : (uint64_t)bar << 32};
    // lanes to read again, and the vectors each took
    const bool again = masked ? lane_top > -kInf : order(lane_top) >= bar;
    const uint64_t mask = __ballot(again);
    if (again) sh.lanes[wave][lanes_below(mask)] = (uint8_t)lane;
    wave_sync();
    const uint32_t count = __builtin_popcountll(mask);
    const uint32_t each = (p.hi - p.lo + kVocabBlock - 1) / kVocabBlock;
    const char *const body = reinterpret_cast<const char *>(x + split.head);
    for (uint32_t i0 = 0; i0 < count * each; i0 += 64) {
        const uint32_t i = i0 + lane;
        // the lowest columns first
        const uint32_t v = i < count * each
                               ? p.lo + i / count * kVocabBlock + wave * 64 + sh.lanes[wave][i % count]
                               : p.hi;
        const typename Vec<T>::wide f = Vec<T>::widen(
            v < p.hi ? load16<true, sizeof(T)>(body + (uint64_t)v * 16) : Vec<T>::masked());
#pragma unroll
        for (uint32_t j = 0; j < N; ++j)
            list.offer(v < p.hi ? rank_key(f[j], split.head + v * N + j) : 0);
    }
    if (wave == 0) {
        if (p.first && split.head) list.offer(lane < split.head ? rank_key((float)x[lane], lane) : 0);
        if (p.last && split.tail) {
            const uint32_t at = cols - split.tail + lane;
            list.offer(lane < split.tail ? rank_key((float)x[at], at) : 0);
        }
        if (masked) {
            // fewer than `top` (or the list has them all): masked columns, of
            // which the first 128 hold enough
            list.bar = 0;
            const uint32_t from = p.first ? 0 : split.head + p.lo * N;
            const uint32_t to = p.last ? cols : split.head + p.hi * N;
            for (uint32_t k = 0; k < 2; ++k) {
                const uint32_t at = from + k * 64 + lane;
                const float f = at < to ? (float)x[at] : 0.0f;
                list.offer(order(f) == kOrderMasked ? rank_key(f, at) : 0);
            }
        }
    }
    return block_top(list, sh);
}

// ---------------------------------------------------------------------------
// Forward: a block a row, or a block a part of a row and a block a row that
// joins the parts
// ---------------------------------------------------------------------------

// The teacher's distribution over its kept entries: the largest logit and the
// sum of exp((logit - m) * scale), in every thread.
struct Teacher {
    float m, z;
};

// (t - m) * scale.  The difference comes first: scaled logits would each bring
// a rounding of their own size along.  Of halves (by.part) where it may
// overflow though scale times it does not come to -infinity.
__device__ __forceinline__ float teacher_distance(float t, float m, const TeacherScale &by)
{
    return __builtin_fmaf(t, by.part, -(m * by.part)) * by.whole;
}

__device__ __forceinline__ bool kept_entry(int64_t id, float scaled, uint32_t cols)
{
    return id >= 0 && id < (int64_t)cols && scaled != -kInf;
}

// What a forward call does with a row's sums, for all threads of a block.
struct Logprobs {
    using Args = LogprobsArgs;
    struct Ahead {              // loaded before the row is streamed
        float logit;
        bool given;
    };
    template <typename T>
    __device__ static Ahead ahead(const Args &a, uint32_t r, const T *x)
    {
        const int64_t t = a.targets[r];
        const bool given = t >= 0 && t < (int64_t)a.cols;
        return Ahead{given ? (float)x[t] : 0.0f, given};
    }
    // key: lane i of the first wave has the i-th best
    template <typename T>
    __device__ static void finish(const Args &a, uint32_t r, const T *, const Ahead &h,
                                  const RowSum &s, uint64_t key, float (*)[kVocabWaves])
    {
        const RowStat st = row_stat(s, a.scale);
        if (threadIdx.x == 0) {
            a.logp[r] = h.given ? log_prob(h.logit, s, st, a.scale) : 0.0f;
            if (a.lse) a.lse[r] = st.lse;
            if (a.entropy) a.entropy[r] = st.entropy;
        }
        if (threadIdx.x < a.top) {
            const uint64_t i = (uint64_t)r * a.top + threadIdx.x;
            a.top_ids[i] = key_col(key);
            a.top_logp[i] = log_prob(key_logit(key), s, st, a.scale);
        }
    }
    __host__ __device__ static uint32_t top(const Args &a) { return a.top; }
};

struct Distill {
    using Args = DistillArgs;
    struct Ahead {              // thread k's entry k: loaded before the row is streamed
        float teacher, logit;   // the teacher's logit, -inf if there is none
    };
    template <typename T>
    __device__ static Ahead entry(const Args &a, uint32_t r, const T *x, uint32_t k)
    {
        Ahead h{-kInf, 0.0f};
        if (k < a.kept) {
            const int64_t id = a.ids[(uint64_t)r * a.kept + k];
            const float t = a.teacher[(uint64_t)r * a.kept + k];
            if (kept_entry(id, t * a.scale, a.cols)) h = Ahead{t, (float)x[id]};
        }
        return h;
    }
    template <typename T>
    __device__ static Ahead ahead(const Args &a, uint32_t r, const T *x)
    {
        return entry(a, r, x, threadIdx.x);
    }
    template <typename T>
    __device__ static void finish(const Args &a, uint32_t r, const T *x, const Ahead &h,
                                  const RowSum &s, uint64_t, float (*scratch)[kVocabWaves])
    {
        const RowStat st = row_stat(s, a.scale);
        // the entries past the block's size are read where they are needed
        const auto each = [&](const auto &f) {
            f(h);
            for (uint32_t k = threadIdx.x + kVocabBlock; k < a.kept; k += kVocabBlock)
                f(entry(a, r, x, k));
        };
        float m = -kInf;
        each([&](const Ahead &e) { m = __builtin_fmaxf(m, e.teacher); });
        m = block_reduce<Max, kVocabWaves>(m, scratch[0]);
        float z = 0.0f;
        each([&](const Ahead &e) {
            z += e.teacher == -kInf ? 0.0f : exp_nat(teacher_distance(e.teacher, m, a.by));
        });
        z = block_reduce<Sum, kVocabWaves>(z, scratch[1]);
        const float log_z = __builtin_logf(z);
        float loss = 0.0f;
        each([&](const Ahead &e) {
            if (e.teacher == -kInf) return;
            const float d = teacher_distance(e.teacher, m, a.by);
            const float l = d - log_z, p = exp_nat(d) / z;
            if (p >= 0x1p-126f || p != p) loss += p * (l - log_prob(e.logit, s, st, a.scale));
        });
        loss = block_reduce<Sum, kVocabWaves>(loss, scratch[2]);
        if (threadIdx.x == 0) {
            a.loss[r] = loss;
            if (a.lse) a.lse[r] = st.lse;
        }
    }
    __host__ __device__ static uint32_t top(const Args &) { return 0; }
};

// The workspace of a call that splits rows: a RowSum padded to 16 bytes for
// each part of each row, then each part's keys.
__device__ __forceinline__ float4 *part_sums(void *ws) { return static_cast<float4 *>(ws); }
__device__ __forceinline__ uint64_t *part_keys(void *ws, uint32_t rows, uint32_t parts)
{
    return reinterpret_cast<uint64_t *>(part_sums(ws) + (uint64_t)rows * parts);
}

struct Nothing {};

template <bool Top>
struct ForwardShared {
    std::conditional_t<Top, TopShared, Nothing> top;
    RowSum part[kVocabWaves];
    float scratch[3][kVocabWaves];
};

// One pass over the logits: each lane keeps a running maximum and sums, joined
// at the row's end.  4096 x 131072 bf16 with entropy 162-171 us, 6.3-6.6 TB/s
// (reading alone in this pattern: 157 us); distillation 2048 x 131072 bf16 85
// us, 6.3 TB/s; 2048 x 50257 49 us with 5 alternatives, 38 without, the floor
// is 29: the blocks' starts and ends come all at the same time; 20
// alternatives 73 us, 32 80, 64 119 (read again: part_top); 8 x 131072 f32
// with 20 alternatives 8.5 us and 4.7 for the join, latency.
//
// Eight waves a SIMD for 16-bit logits: with the 74 registers the compiler
// would take, the 2048 blocks of as many rows need a second round on 256 CUs
// (2048 x 50257 bf16, 5 alternatives: 54.6 us; 50.6 with 64).  32-bit rows,
// twice as long in bytes, would spill.
template <typename T, class Op, bool Ent, bool Top>
__global__ void __launch_bounds__(kVocabBlock, sizeof(T) == 2 ? 8 : 4) ew_vocab_forward_kernel(typename Op::Args a,
                                                                       uint32_t parts)
{
    __shared__ __align__(16) ForwardShared<Top> sh;
    const uint64_t items = (uint64_t)a.rows * parts;
    const Rate rate(a.scale);
    for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t r = (uint32_t)(item / parts), part = (uint32_t)(item % parts);
        const T *const x = static_cast<const T *>(a.logits) + r * a.stride;
        typename Op::Ahead h{};
        if (parts == 1) h = Op::ahead(a, r, x);
        const RowSplit<T> split(x, a.cols);
        const Part p(split.vectors, part, parts);
        RowSum s = stream_part<T, Ent>(x, a.cols, p, split, rate);
        uint64_t key = 0;
        if constexpr (Top) key = part_top(x, a.cols, p, split, s.m, Op::top(a), sh.top);
        block_join<Ent>(s, rate, sh.part);
        if (parts == 1) {
            Op::finish(a, r, x, h, s, key, sh.scratch);
        } else {
            if (threadIdx.x == 0) part_sums(a.workspace)[item] = float4{s.m, s.z, s.b, 0.0f};
            if constexpr (Top)
                if (threadIdx.x < Op::top(a))
                    part_keys(a.workspace, a.rows, parts)[item * Op::top(a) + threadIdx.x] = key;
        }
        if (item + gridDim.x < items) __syncthreads();
    }
}

template <typename T, class Op, bool Ent, bool Top>
__global__ void __launch_bounds__(kVocabBlock) ew_vocab_join_kernel(typename Op::Args a,
                                                                    uint32_t parts)
{
    __shared__ __align__(16) ForwardShared<Top> sh;
    const Rate rate(a.scale);
    const uint64_t r = blockIdx.x;       // rows that are split are fewer than a grid's blocks
    const T *const x = static_cast<const T *>(a.logits) + r * a.stride;
    const typename Op::Ahead h = Op::ahead(a, (uint32_t)r, x);
    RowSum s{-kInf, 0.0f, 0.0f};
    if (threadIdx.x < parts) {
        const float4 q = part_sums(a.workspace)[r * parts + threadIdx.x];
        s = RowSum{q.x, q.y, q.z};
    }
    uint64_t key = 0;
    if constexpr (Top) {
        // the parts' lists are in order: the top-th largest of 64 keys
        // from their heads is a bar for all
        const uint32_t top = Op::top(a), n = parts * top, lane = threadIdx.x % 64;
        const uint64_t *const keys = part_keys(a.workspace, a.rows, parts) + r * n;
        constexpr int kEarly = 4;      // keys loaded before the bar is known
        uint64_t early[kEarly];
#pragma unroll
        for (int k = 0; k < kEarly; ++k)
            early[k] = k * kVocabBlock + threadIdx.x < n ? keys[k * kVocabBlock + threadIdx.x] : 0;
        const uint32_t from = lane % parts * top + lane / parts;
        const uint32_t head = lane / parts < top ? (uint32_t)(keys[from] >> 32) : 0;
        const uint32_t bar = lanes_kth(head, top);
        TopList list{sh.top.keys[threadIdx.x / 64], 0, top, (uint64_t)bar << 32};
#pragma unroll
        for (int k = 0; k < kEarly; ++k) list.offer(early[k]);
        for (uint32_t i = kEarly * kVocabBlock + threadIdx.x / 64 * 64; i < n; i += kVocabBlock)
            list.offer(i + lane < n ? keys[i + lane] : 0);
        key = block_top(list, sh.top);
    }
    block_join<Ent>(s, rate, sh.part);
    Op::finish(a, (uint32_t)r, x, h, s, key, sh.scratch);
}

// ---------------------------------------------------------------------------
// Gradients
// ---------------------------------------------------------------------------

// A gradient's rows are cut into tiles of kGradSteps steps, a block each; a
// step is kGradLane elements a thread.  The first step's loads are in flight
// while the block works out what it needs of the row, each later one's while
// the step before is worked on.  Vectors start at the row's start, whatever
// alignment it has.  4096 x 131072 bf16, log probabilities: two steps of 16
// elements 348 us, one 353-365, four 359, one of 32 354, two of 32 358; the
// distillation's 2048 x 131072: 182, 203, 186, 189, 185.
constexpr int kGradLane = 16, kGradSteps = 2;

template <typename T>
struct GradTile {
    static constexpr int N = Vec<T>::N, U = kGradLane / N;
    static constexpr uint32_t kStepVectors = kVocabBlock * U;
    static constexpr uint32_t kCols = kStepVectors * N * kGradSteps;
    const char *in;
    char *out;
    uint32_t first, cols;      // the tile's first column and its number of columns
    bool aligned;              // dlogits on 16-byte boundaries: stored at device scope (1 % faster)
    u32x4 v[U];

    __device__ GradTile(const T *x, T *dx, uint32_t row_cols, uint32_t tile)
    {
        first = tile * kCols;
        cols = row_cols - first < kCols ? row_cols - first : kCols;
        in = reinterpret_cast<const char *>(x + first);
        out = reinterpret_cast<char *>(dx + first);
        aligned = reinterpret_cast<uintptr_t>(out) % 16 == 0;
    }
    // this thread's u-th vector of a step, as one of the tile's
    __device__ static uint32_t vector(uint32_t step, int u)
    {
        return step * kStepVectors + threadIdx.x + u * kVocabBlock;
    }
    // whole vectors are loaded as such, the row's last elements one by one
    __device__ void fetch(uint32_t step)
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = vector(step, u);
            v[u] = u32x4{0, 0, 0, 0};
            if ((i + 1) * N <= cols) v[u] = load16<false, sizeof(T)>(in + i * 16);
        }
        if (cols % N) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (vector(step, u) == cols / N) v[u] = load_some(cols / N);
        }
    }
    __device__ u32x4 load_some(uint32_t i) const
    {
        typename Vec<T>::type t{};
        const T *const p = reinterpret_cast<const T *>(in) + i * N;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (i * N + j < cols) t[j] = p[j];
        return __builtin_bit_cast(u32x4, t);
    }
    __device__ void store(uint32_t i, typename Vec<T>::wide g) const
    {
        const u32x4 w = Vec<T>::narrow(g);
        if ((i + 1) * N <= cols) {
            if (aligned) store16_device(out, kCols * sizeof(T), i * 16, w);
            else store16_row<T>(out + i * 16, w);
        } else if (i * N < cols) {
            const typename Vec<T>::type t = __builtin_bit_cast(typename Vec<T>::type, w);
            T *const p = reinterpret_cast<T *>(out) + i * N;
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (i * N + j < cols) p[j] = t[j];
        }
    }
    // f(vector of the tile, its widened elements) for each step's vectors;
    // the first step has been fetched
    template <class F>
    __device__ void each(const F &f)
    {
        for (uint32_t step = 0; step * kStepVectors * N < cols; ++step) {
            u32x4 own[U];
#pragma unroll
            for (int u = 0; u < U; ++u) own[u] = v[u];
            if ((step + 1) * kStepVectors * N < cols) fetch(step + 1);
#pragma unroll
            for (int u = 0; u < U; ++u) store(vector(step, u), f(vector(step, u), Vec<T>::widen(own[u])));
        }
    }
    // the same, a vector at a time: for rare rows beside the loop above,
    // whose registers it must not add to (the log probabilities' 16-bit
    // gradient 173-174 us with it, 178-180 with a second loop like the first;
    // the distillation's, with fewer registers, gains nothing)
    template <class F>
    __device__ void each_in_turn(const F &f) const
    {
        for (uint32_t i = threadIdx.x; i * N < cols; i += kVocabBlock) {
            const u32x4 w = (i + 1) * N <= cols ? load16<false, sizeof(T)>(in + i * 16) : load_some(i);
            store(i, f(i, Vec<T>::widen(w)));
        }
    }
};

// scale * x - lse, at most 0 (a difference of large numbers may round to
// above it) and at least kLeast, below which its exponential is 0 anyway
// (from -88 on): what it is multiplied by stays small where x is masked or far
// below the rest.
constexpr float kLeast = -110.0f;

__device__ __forceinline__ float log_p(float x, float scale, float lse)
{
    return __builtin_amdgcn_fmed3f(__builtin_fmaf(x, scale, -lse), kLeast, 0.0f);
}

// A row's gradient is scale times slopes times terms of p.  Where a slope and
// scale together pass kLargeFactor the product with p may still be ordinary
// (and infinite times a p of 0 a NaN), so there the slopes come in 2^-8 times
// as large, enough for their terms (a logarithm is at most 110) to stay finite,
// and without a scale above 1; both are made up for once the terms are whole.
constexpr float kLargeFactor = 1e38f, kShrink = 0x1p-8f;

struct Factors {
    float shrink, scale;       // before: (1, the scale), or of a large row (2^-8, at most 1)
    float above;               // after, in a large row: with 2^8
    __device__ Factors(bool large, float s)
        : shrink(large ? kShrink : 1.0f), scale(large ? __builtin_fminf(s, 1.0f) : s),
          above(large ? __builtin_fmaxf(s, 1.0f) : 1.0f) {}
    __device__ float whole(float d) const { return shrink == 1.0f ? d : d * (1.0f / kShrink) * above; }
};

// Bound by memory: 4096 x 131072 bf16 340 us, 6.3 TB/s (copy 6.64).
// dlogits = scale * (dlogp * (hot - p) - dent * p * (l + ent)), l = log p:
// p * (l * k2 + k1), and dlogp * scale at the target.  Masked logits get their
// 0 whatever the factors are; everything else in a row with a NaN is one.
template <typename T>
__global__ void __launch_bounds__(kVocabBlock) ew_logprobs_grad_kernel(LogprobsGradArgs a,
                                                                       uint32_t tiles)
{
    constexpr int N = Vec<T>::N;
    const uint64_t items = (uint64_t)a.rows * tiles;
    for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t r = (uint32_t)(item / tiles);
        GradTile<T> g(static_cast<const T *>(a.logits) + r * a.stride,
                      static_cast<T *>(a.dlogits) + r * a.dlogits_stride, a.cols,
                      (uint32_t)(item % tiles));
        g.fetch(0);
        const int64_t target = a.targets[r];
        const bool given = target >= 0 && target < (int64_t)a.cols;
        const float row_lse = a.lse[r], row_dlogp = a.dlogp[r];
        const bool empty = row_lse == -kInf;
        const float lse = empty ? 0.0f : row_lse, dlogp = given ? row_dlogp : 0.0f;
        const float dent = a.dentropy ? a.dentropy[r] : 0.0f;
        const float ent = a.dentropy ? a.entropy[r] : 0.0f;
        const bool large = !((__builtin_fabsf(dlogp) + __builtin_fabsf(dent) * -kLeast) * a.scale <
                             kLargeFactor);
        const Factors f(large, a.scale);
        const float k1 = empty ? 0.0f : -(dlogp * f.shrink + dent * f.shrink * ent) * f.scale;
        const float k2 = empty ? 0.0f : -(dent * f.shrink) * f.scale;
        const float hot = dlogp * f.shrink * f.scale;
        // the target's place in the tile, past the tile's end without one
        const uint32_t hit = given && !empty ? (uint32_t)target - g.first : ~0u;
        const auto gradient = [&](uint32_t i, typename Vec<T>::wide x) {
            typename Vec<T>::wide d;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float l = log_p(x[j], a.scale, lse);
                d[j] = exp_nat(l) * __builtin_fmaf(l, k2, k1);
            }
            if (hit / N == i) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (hit % N == j && x[j] * a.scale != -kInf) d[j] += hot;
            }
            return d;
        };
        if (large || lse != lse) {
            g.each_in_turn([&](uint32_t i, typename Vec<T>::wide x) {
                typename Vec<T>::wide d = gradient(i, x);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    d[j] = empty || x[j] * a.scale == -kInf ? 0.0f : lse != lse ? lse : f.whole(d[j]);
                return d;
            });
        } else {
            g.each(gradient);
        }
    }
}

// The teacher's distribution, in one wave.
__device__ __forceinline__ Teacher wave_teacher(const float *teacher, const int64_t *ids,
                                                uint32_t kept, uint32_t cols, float scale,
                                                const TeacherScale &by)
{
    Teacher t;
    float m = -kInf;
    for (uint32_t k = threadIdx.x % 64; k < kept; k += 64) {
        const float own = teacher[k];
        if (kept_entry(ids[k], own * scale, cols)) m = __builtin_fmaxf(m, own);
    }
    t.m = wave_reduce<Max>(m);
    float z = 0.0f;
    for (uint32_t k = threadIdx.x % 64; k < kept; k += 64) {
        const float own = teacher[k];
        if (kept_entry(ids[k], own * scale, cols)) z += exp_nat(teacher_distance(own, t.m, by));
    }
    t.z = wave_reduce<Sum>(z);
    return t;
}

// dlogits = k1 * (p - w), w the weight of the entries that name the column.
// The tile is written as if w were 0; the few columns that entries name are
// written again after it, one thread each, from the logits that the first
// wave set aside (dlogits may be logits).  Looking for the entries while
// streaming took more instructions than the softmax: 220 us for 2048 rows of
// 131072 bf16 with 64 entries, where this takes 182.
template <typename T>
__global__ void __launch_bounds__(kVocabBlock) ew_distill_grad_kernel(DistillGradArgs a,
                                                                      uint32_t tiles)
{
    constexpr int N = Vec<T>::N;
    // the kept entries that fall into the tile, in their order: place,
    // weight, logit
    __shared__ uint32_t at[kMaxKept];
    __shared__ float weight[kMaxKept], logit[kMaxKept];
    __shared__ uint32_t found;
    __shared__ float teacher_sum;
    const uint64_t items = (uint64_t)a.rows * tiles;
    for (uint64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const uint32_t r = (uint32_t)(item / tiles);
        const T *const x = static_cast<const T *>(a.logits) + r * a.stride;
        GradTile<T> g(x, static_cast<T *>(a.dlogits) + r * a.dlogits_stride, a.cols,
                      (uint32_t)(item % tiles));
        g.fetch(0);
        const float row_lse = a.lse[r], row_dloss = a.dloss[r];
        if (threadIdx.x < 64) {
            const float *const teacher = a.teacher + (uint64_t)r * a.kept;
            const int64_t *const ids = a.ids + (uint64_t)r * a.kept;
            const Teacher t = wave_teacher(teacher, ids, a.kept, a.cols, a.scale, a.by);
            uint32_t n = 0;
            for (uint32_t k0 = 0; k0 < a.kept; k0 += 64) {
                const uint32_t k = k0 + threadIdx.x;
                const int64_t id = k < a.kept ? ids[k] : -1;
                const float own = k < a.kept ? teacher[k] : -kInf;
                const bool here =
                    kept_entry(id, own * a.scale, a.cols) && (uint64_t)id - g.first < g.cols;
                const uint64_t mask = __ballot(here);
                if (here) {
                    const uint32_t slot = n + lanes_below(mask);
                    at[slot] = (uint32_t)id - g.first;
                    weight[slot] = exp_nat(teacher_distance(own, t.m, a.by)) / t.z;
                    logit[slot] = (float)x[id];
                }
                n += __builtin_popcountll(mask);
            }
            if (threadIdx.x == 0) {
                found = n;
                teacher_sum = t.z;
            }
        }
        __syncthreads();
        const uint32_t entries = found;
        const float tz = teacher_sum;
        const bool empty = row_lse == -kInf || tz == 0.0f, nan = row_lse != row_lse || tz != tz;
        const float lse = empty ? 0.0f : row_lse, dloss = empty ? 0.0f : row_dloss;
        const bool large = !(__builtin_fabsf(dloss) * a.scale < kLargeFactor);
        const Factors f(large, a.scale);
        const float k1 = dloss * f.shrink * f.scale;
        const auto gradient = [&](uint32_t, typename Vec<T>::wide v) {
            typename Vec<T>::wide d;
#pragma unroll
            for (int j = 0; j < N; ++j) d[j] = k1 * exp_nat(log_p(v[j], a.scale, lse));
            return d;
        };
        if (large || nan) {
            g.each([&](uint32_t i, typename Vec<T>::wide v) {
                typename Vec<T>::wide d = gradient(i, v);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    d[j] = v[j] * a.scale == -kInf ? 0.0f : nan ? lse + tz : f.whole(d[j]);
                return d;
            });
        } else {
            g.each(gradient);
        }
        __syncthreads();       // the tile is stored
        if (!nan) {
            for (uint32_t e = threadIdx.x; e < entries; e += kVocabBlock) {
                // the first entry of a column adds up all of them, in order
                const uint32_t place = at[e];
                bool first = logit[e] * a.scale != -kInf;
                float w = 0.0f;
                for (uint32_t o = 0; o < entries; ++o) {
                    const bool same = at[o] == place;
                    first = first && !(same && o < e);
                    w += same ? weight[o] : 0.0f;
                }
                if (first)
                    reinterpret_cast<T *>(g.out)[place] =
                        (T)f.whole(k1 * (exp_nat(log_p(logit[e], a.scale, lse)) - w));
            }
        }
        if (item + gridDim.x < items) __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

// A row is split where there are too few to fill the GPU and it is long enough
// to pay for the second launch, which costs the host 3.5 us and the GPU about
// 3 (one block a row against parts, GPU time in us, bf16: distillation of 37
// rows of 32001 7.1 / 6.9, 1 of 131072 19.3 / 6.1; log probabilities of 256
// rows of 8000 4.9 / 7.0, 256 of 131072 24.3 / 16.9, 512 28.4 / 28.4).
// Ranking makes a block's row dearer (5 of 64 rows of 50257 15.7 / 13.1, 20 of
// 32 rows of 32000 f32 20.2 / 12.3, 5 of 1 row of 4000 6.0 / 6.0).  A
// function of the sizes alone, so that the workspace is too.
constexpr uint64_t kWholeRows = 512;                            // from here on no row is split
constexpr uint64_t kWholeCols = 49152, kWholeTopCols = 16384;   // nor up to here
constexpr uint64_t kWantBlocks = 1024, kPartCols = 4096, kMaxParts = 256;
static_assert(kMaxParts <= kVocabBlock, "the join takes a part a thread");

static uint32_t row_parts(uint64_t rows, uint64_t cols, uint64_t top)
{
    if (rows == 0 || rows >= kWholeRows || cols <= (top ? kWholeTopCols : kWholeCols)) return 1;
    uint64_t parts = (kWantBlocks + rows - 1) / rows;
    const uint64_t most = (cols + kPartCols - 1) / kPartCols;
    if (parts > most) parts = most;
    return (uint32_t)(parts < kMaxParts ? parts : kMaxParts);
}

size_t logprobs_workspace(uint64_t rows, uint64_t cols, uint64_t top)
{
    const uint64_t parts = row_parts(rows, cols, top);
    return parts == 1 ? 0 : rows * parts * (sizeof(float4) + top * sizeof(uint64_t));
}
size_t distill_workspace(uint64_t rows, uint64_t cols) { return logprobs_workspace(rows, cols, 0); }

#define EW_BY_TYPE(t, K)                                           \
    ((t) == kRowF32 ? reinterpret_cast<const void *>(&K<float>)    \
     : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16>) \
                      : reinterpret_cast<const void *>(&K<__bf16>))

// Blocks stride over what is beyond this many.
constexpr uint64_t kMaxGrid = 1 << 23;

static uint32_t grad_tiles(uint32_t cols)
{
    constexpr uint64_t tile = (uint64_t)kVocabBlock * kGradLane * kGradSteps;
    return (uint32_t)((cols + tile - 1) / tile);
}

template <class... A>
static hipError_t go(const void *fn, uint64_t blocks, hipStream_t s, A... args)
{
    void *kargs[] = {&args...};
    return hipLaunchKernel(fn, dim3((uint32_t)(blocks < kMaxGrid ? blocks : kMaxGrid)),
                           dim3(kVocabBlock), kargs, 0, s);
}

template <class Op, bool Ent, bool Top>
static hipError_t forward(RowType t, const typename Op::Args &a, hipStream_t s, const char **path)
{
    const uint32_t parts = row_parts(a.rows, a.cols, Op::top(a));
#define EW_FORWARD(K)                                                                      \
    (t == kRowF32 ? reinterpret_cast<const void *>(&K<float, Op, Ent, Top>)                \
     : t == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16, Op, Ent, Top>)           \
                    : reinterpret_cast<const void *>(&K<__bf16, Op, Ent, Top>))
    const hipError_t e = go(EW_FORWARD(ew_vocab_forward_kernel), (uint64_t)a.rows * parts, s, a, parts);
    *path = parts == 1 ? "a block a row" : "rows in parts, then joined";
    if (e != hipSuccess || parts == 1) return e;
    return go(EW_FORWARD(ew_vocab_join_kernel), a.rows, s, a, parts);
#undef EW_FORWARD
}

hipError_t launch_logprobs(RowType t, const LogprobsArgs &a, hipStream_t s, const char **path)
{
    if (a.top)
        return a.entropy ? forward<Logprobs, true, true>(t, a, s, path)
                         : forward<Logprobs, false, true>(t, a, s, path);
    return a.entropy ? forward<Logprobs, true, false>(t, a, s, path)
                     : forward<Logprobs, false, false>(t, a, s, path);
}

hipError_t launch_logprobs_grad(RowType t, const LogprobsGradArgs &a, hipStream_t s,
                                const char **path)
{
    *path = "a block a tile";
    const uint32_t tiles = grad_tiles(a.cols);
    return go(EW_BY_TYPE(t, ew_logprobs_grad_kernel), (uint64_t)a.rows * tiles, s, a, tiles);
}

hipError_t launch_distill(RowType t, const DistillArgs &a, hipStream_t s, const char **path)
{
    return forward<Distill, false, false>(t, a, s, path);
}

hipError_t launch_distill_grad(RowType t, const DistillGradArgs &a, hipStream_t s,
                               const char **path)
{
    *path = "a block a tile";
    const uint32_t tiles = grad_tiles(a.cols);
    return go(EW_BY_TYPE(t, ew_distill_grad_kernel), (uint64_t)a.rows * tiles, s, a, tiles);
}

}  // namespace ew
