// ew_policy.hip -- the clipped policy loss with a KL term, and its gradient,
// for CDNA4 (gfx950).

#include "ew.h"
#include "ew_policy_marks.h"
#include "ew_rows_vec.h"

namespace ew {

// exp(d) - 1 and exp(d) - 1 - d, which are of the order of d and d^2: for
// |d| < 1 by the series (the first term left out is below 2^-26 of the sum),
// beyond from exp(d), where less than two bits cancel.
struct Growth {
    float one, line;
    __device__ explicit Growth(float d)
    {
        float p = 1.0f / 479001600.0f;                       // 1 / 12!
        p = __builtin_fmaf(p, d, 1.0f / 39916800.0f);
        p = __builtin_fmaf(p, d, 1.0f / 3628800.0f);
        p = __builtin_fmaf(p, d, 1.0f / 362880.0f);
        p = __builtin_fmaf(p, d, 1.0f / 40320.0f);
        p = __builtin_fmaf(p, d, 1.0f / 5040.0f);
        p = __builtin_fmaf(p, d, 1.0f / 720.0f);
        p = __builtin_fmaf(p, d, 1.0f / 120.0f);
        p = __builtin_fmaf(p, d, 1.0f / 24.0f);
        p = __builtin_fmaf(p, d, 1.0f / 6.0f);
        p = __builtin_fmaf(p, d, 0.5f);
        const float bend = p * d * d;
        one = d + bend;
        line = bend;
        if (!(__builtin_fabsf(d) < 1.0f)) {                  // (few lanes, if any)
            one = exp_nat(d) - 1.0f;
            line = one == kInf ? one : one - d;              // (not inf - inf)
        }
    }
};

// What a token adds.
struct Token {
    double x;          // logp - old_logp, exact
    float ratio;       // exp(x), finite for an advantage of 0
    bool clipped;      // the gain is that of the border
    float one, line;   // of d = ref_logp - logp: exp(d) - 1, exp(d) - 1 - d
};

template <bool Ref>
__device__ __forceinline__ Token token(const PolicyTokens &in, float logp, float old, float ref, float a)
{
    Token t;
    t.x = (double)logp - (double)old;
    const bool gains = a > 0.0f, pays = a < 0.0f;
    t.clipped = (gains && t.x > in.above) || (pays && t.x < in.below);
    t.ratio = exp_nat((float)t.x);
    // a token of no advantage gains nothing, also where binary32 does not hold the
    // ratio (a NaN stays)
    if (t.ratio == kInf && !gains && !pays) t.ratio = 1.0f;
    t.one = 0.0f;
    t.line = 0.0f;
    if constexpr (Ref) {
        const Growth g(ref - logp);
        t.one = g.one;
        t.line = g.line;
    }
    return t;
}

// A row's pointers.
struct PolicyRow {
    const float *logp, *old, *ref, *advantage;
    const uint8_t *mask;
    float each;                // the advantage of all its tokens, if one
    __device__ PolicyRow(const PolicyTokens &in, uint64_t r)
        : logp(in.logp + r * in.logp_stride), old(in.old + r * in.old_stride),
          ref(in.ref + r * in.ref_stride), advantage(in.advantage + r * in.advantage_stride),
          mask(in.mask + r * in.mask_stride),
          each(in.advantage_stride ? 0.0f : in.advantage[r])
    {
    }
};

// A stretch of a row: `lanes` lanes take four neighbouring tokens of it each,
// from token `from` on.
template <RowFit Fit>
struct Tokens {
    using Place = Piece<float, Fit>;
    uint64_t from;
    uint32_t cols, back;       // its tokens; tokens before it that a piece may reach
    __device__ Tokens(uint64_t from_, uint32_t all, uint32_t lanes)
        : from(from_), cols(all - from_ < lanes * 4 ? (uint32_t)(all - from_) : lanes * 4),
          back(from_ ? 4 : 0)
    {
    }
    __device__ Place place(uint32_t lane) const { return Place(lane * 4, cols, back); }
    template <class E>
    __device__ E *row(E *p) const { return p + (from - back); }
};

// Four tokens of a lane.  Which of them count comes first: of tokens that do
// not, nothing else is read.
struct Four {
    uint32_t counted;          // bit 8 j + 7: token j is the piece's own and counts
    f32x4 logp, old, ref, a;

    // The mask's bytes of the lane's piece.
    template <RowFit Fit>
    __device__ static uint32_t mark(const PolicyTokens &in, const PolicyRow &row, const Tokens<Fit> &t,
                                    uint32_t lane)
    {
        typedef uint32_t word __attribute__((aligned(1)));
        const auto p = t.place(lane);
        if (!p.live) return 0;
        if (!in.mask) return 0x01010101u;
        if constexpr (Fit == kTiny) {
            uint32_t bytes = 0;
            for (uint32_t j = 0; j < t.cols; ++j) bytes |= (uint32_t)row.mask[j] << 8 * j;
            return bytes;
        }
        return __builtin_nontemporal_load(reinterpret_cast<const word *>(t.row(row.mask) + p.first));
    }
    template <bool Ref, RowFit Fit>
    __device__ void load(const PolicyTokens &in, const PolicyRow &row, const Tokens<Fit> &t,
                         uint32_t lane, uint32_t mark)
    {
        const auto p = t.place(lane);
        counted = counted_tokens(mark, Fit == kPart ? p.skip : 0);
        if constexpr (Fit == kTiny) counted &= (1u << 8 * t.cols) - 1;
        if (!counted) return;
        const auto take = [&](const float *v) {
            return __builtin_bit_cast(f32x4, load_piece<float, true>(t.row(v), t.cols, p));
        };
        logp = take(row.logp);
        old = take(row.old);
        if constexpr (Ref) ref = take(row.ref);
        a = in.advantage_stride ? take(row.advantage) : f32x4{row.each, row.each, row.each, row.each};
    }
    template <bool Ref>
    __device__ Token token(const PolicyTokens &in, int j) const
    {
        return ew::token<Ref>(in, logp[j], old[j], Ref ? ref[j] : 0.0f, a[j]);
    }
    __device__ uint32_t number() const { return (uint32_t)__builtin_popcount(counted); }
    __device__ bool counts(int j) const { return (counted >> (8 * j + 7) & 1u) != 0; }
};

// Calls f for a lane's pieces of a row's tokens [from, to), stretch by stretch
// of `lanes` lanes.  Two whole stretches' pieces are on their way together, and
// the marks of the next two.  One: the row is one stretch.
// Reading only what the marks leave took the loss of 4096 sequences of up to
// 4096 tokens, half of them counted, from 59 to 38 us and its gradient from 64
// to 40.
template <bool Ref, bool Few, bool One, class F>
__device__ __forceinline__ void each_four(const PolicyTokens &in, const PolicyRow &row, uint64_t from,
                                          uint32_t to, uint32_t lanes, uint32_t lane, F f)
{
    const auto last = [&](uint64_t at) {
        const Tokens<Few ? kTiny : kPart> t(at, to, lanes);
        Four four;
        four.load<Ref>(in, row, t, lane, Four::mark(in, row, t, lane));
        f(four, t);
    };
    if constexpr (One) {
        last(0);
        return;
    }
    const auto step = (uint64_t)lanes * 4;
    using Whole = Tokens<kWhole>;
    const auto mark = [&](uint64_t at) {
        return at + step <= to ? Four::mark(in, row, Whole(at, to, lanes), lane) : 0;
    };
    uint32_t next1 = mark(from), next2 = mark(from + step);
    uint64_t at = from;
    for (; at + step <= to; at += 2 * step) {
        const uint32_t mark1 = next1, mark2 = next2;
        next1 = mark(at + 2 * step);
        next2 = mark(at + 3 * step);
        const bool more = at + 2 * step <= to;
        const Whole t1(at, to, lanes), t2(more ? at + step : at, to, lanes);
        Four f1, f2;
        f1.load<Ref>(in, row, t1, lane, mark1);
        f2.load<Ref>(in, row, t2, lane, mark2);
        f(f1, t1);
        __builtin_amdgcn_sched_barrier(0);      // one piece's numbers in registers at a time
        if (!more) {
            at += step;
            break;
        }
        f(f2, t2);
    }
    if (at < to) last(at);
}

// ---------------------------------------------------------------------------
// Forward: sums over parts of the batch, then their join (a second launch: a
// last block that joins would need a counter that is 0 before the call).  Both
// in one block for few tokens.  4096 x 4096 tokens, half of them counted: 36.4
// us, of which 4.5 are the join's.  143 MB are read, 21 us; the rest is that
// sequences end at different times, and a block's sequences after another on
// the way (every block is on the chip at once; the vector unit is busy 51 % of
// the cycles).  8 x 512 tokens: 5.5 us, latency.
// ---------------------------------------------------------------------------

// Sums over tokens: of -gain, of exp(d) - 1 - d (both weighed within their
// sequence where the mean is over sequences), of old_logp - logp, and counts
// (exact below 2^53).
struct PolicySums {
    double policy, kl, fall;
    double clipped, tokens, rows;       // rows: sequences with counted tokens
    __device__ void add(const PolicySums &o)
    {
        policy += o.policy;
        kl += o.kl;
        fall += o.fall;
        clipped += o.clipped;
        tokens += o.tokens;
        rows += o.rows;
    }
};

constexpr int kPolicyBlock = 256;
constexpr int kSmallBlock = 1024;

__device__ __forceinline__ double sixteen_sum(double x)
{
    x += dpp64<0xB1>(x);
    x += dpp64<0x4E>(x);
    x += dpp64<0x141>(x);
    return x + dpp64<0x140>(x);
}

// F of each of the sums.
template <class F>
__device__ __forceinline__ PolicySums each_sum(const PolicySums &s, F f)
{
    return PolicySums{f(s.policy), f(s.kl), f(s.fall), f(s.clipped), f(s.tokens), f(s.rows)};
}

// The sums of a block of Waves waves (at most 16) in all its threads, in a
// fixed order.
template <int Waves>
__device__ __forceinline__ PolicySums block_sums(const PolicySums &mine, PolicySums *scratch)
{
    const PolicySums wave = each_sum(mine, [](double x) { return wave_sum64(x); });
    if (threadIdx.x % 64 == 0) scratch[threadIdx.x / 64] = wave;
    __syncthreads();
    const uint32_t at = threadIdx.x % 16;
    const PolicySums some = at < Waves ? scratch[at] : PolicySums{};
    return each_sum(some, [](double x) { return sixteen_sum(x); });
}

// What a lane sums.  Its counts fit in 32 bits: its tokens are of one sequence
// (below 2^31), or there are kRecords blocks, whose lanes share what the memory
// holds (below 2^37 tokens) in equal numbers of sequences.
struct LaneSums {
    double policy, kl, fall;
    uint32_t clipped, tokens, rows;
    __device__ LaneSums() : policy(0.0), kl(0.0), fall(0.0), clipped(0), tokens(0), rows(0) {}
    __device__ PolicySums all() const
    {
        return PolicySums{policy, kl, fall, (double)clipped, (double)tokens, (double)rows};
    }
};

// Four tokens: policy and kl of their sequence's sums, the rest of all.  Each
// term is binary32, but the log ratio, which is exact, and every sum binary64.
template <bool Ref>
__device__ __forceinline__ void add_four(const PolicyTokens &in, const Four &f, double &row_policy,
                                         double &row_kl, LaneSums &s)
{
    uint32_t clipped = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Token t = f.token<Ref>(in, j);
        const bool counted = f.counts(j);
        const float bound = f.a[j] > 0.0f ? in.most : in.least;
        const float loss = -f.a[j] * (t.clipped ? bound : t.ratio);
        row_policy += (double)(counted ? loss : 0.0f);
        if constexpr (Ref) row_kl += (double)(counted ? t.line : 0.0f);
        s.fall -= counted ? t.x : 0.0;
        clipped += counted && t.clipped;
    }
    s.clipped += clipped;
    s.tokens += f.number();
}

// A lane's share of a sequence's tokens [from, to): its sums of them, and of the
// rest in s.
template <bool Ref, bool Few, bool One>
__device__ __forceinline__ void sum_tokens(const PolicyTokens &in, uint64_t r, uint64_t from, uint32_t to,
                                           uint32_t lanes, uint32_t lane, double &row_policy,
                                           double &row_kl, LaneSums &s)
{
    if (from >= to) return;        // (the advantage of no tokens may be absent)
    const PolicyRow row(in, r);
    each_four<Ref, Few, One>(in, row, from, to, lanes, lane, [&](const Four &f, const auto &) {
        if (f.counted) add_four<Ref>(in, f, row_policy, row_kl, s);
    });
}

// Loss and stats from the batch's sums.
__device__ __forceinline__ void write_loss(const PolicyLossArgs &a, const PolicySums &s)
{
    const bool some = s.tokens > 0.0;
    const double n = a.mean == EW_MEAN_TOKENS ? s.tokens : a.mean == EW_MEAN_SEQUENCES ? s.rows : 1.0;
    const double w = some ? (double)a.scale / n : 0.0;
    const double policy = some ? s.policy * w : 0.0, kl = some ? s.kl * w : 0.0;
    // (a KL term that does not count may be infinite)
    a.loss[0] = (float)(a.in.kl != 0.0f ? policy + (double)a.in.kl * kl : policy);
    if (a.stats) {
        a.stats[0] = (float)policy;
        a.stats[1] = (float)kl;
        a.stats[2] = some ? (float)(s.clipped / s.tokens) : 0.0f;
        a.stats[3] = some ? (float)(s.fall / s.tokens) : 0.0f;
    }
}

// Weight of a counted token of a sequence that has n of them.
__device__ __forceinline__ float token_weight(const PolicyLossArgs &a, const PolicySums &s, uint32_t n)
{
    if (n == 0) return 0.0f;
    if (a.mean == EW_MEAN_TOKENS) return (float)((double)a.scale / s.tokens);
    if (a.mean == EW_MEAN_NONE) return a.scale;
    return (float)((double)a.scale / ((double)n * s.rows));
}

// Sum over `lanes` neighbouring lanes (a power of two), in each of them.
__device__ __forceinline__ uint32_t lanes_sum(uint32_t x, uint32_t lanes)
{
    for (uint32_t d = 1; d < lanes; d *= 2) x += (uint32_t)__shfl_xor((int)x, (int)d);
    return x;
}

// A sequence's sums (or a part's, or a lane's of them) as the batch counts
// them: divided by the sequence's tokens where the mean is over sequences.
__device__ __forceinline__ void add_sequence(PolicySums &all, const PolicySums &s, bool by_sequence,
                                             uint32_t tokens, bool first)
{
    const double w = by_sequence && tokens ? 1.0 / (double)tokens : 1.0;
    all.policy += s.policy * w;
    all.kl += s.kl * w;
    all.fall += s.fall;
    all.clipped += s.clipped;
    all.tokens += s.tokens;
    all.rows += first && tokens ? 1.0 : 0.0;
}

// Which sequence of a round a thread works on; Wave: the same for a wave.
template <bool Wave>
__device__ __forceinline__ uint32_t row_in_round(uint32_t lanes)
{
    const uint32_t row = threadIdx.x / lanes;
    return Wave ? (uint32_t)__builtin_amdgcn_readfirstlane((int)row) : row;
}

// Sequences from r0 on, `step` of them apart and `lanes` lanes each (a power of
// two up to Block), added to all; their tokens to counts.  Whole waves and
// blocks go round together.
template <bool Ref, bool Few, bool Wave, uint32_t Block>
__device__ __forceinline__ void add_sequences(const PolicyLossArgs &a, uint64_t r0, uint64_t step,
                                              uint32_t lanes, uint32_t *counts, LaneSums &all)
{
    // two sets, used in turn: a wave is at most one barrier ahead of another
    __shared__ uint32_t tokens_of[2][Block / 64];
    const uint32_t lane = threadIdx.x % lanes;
    for (int set = 0; r0 < a.rows; r0 += step, set ^= 1) {
        const uint64_t r = r0 + row_in_round<Wave>(lanes);
        double policy = 0.0, kl = 0.0;
        const uint32_t before = all.tokens;
        if (r < a.rows) sum_tokens<Ref, Few, !Wave>(a.in, r, 0, a.cols, lanes, lane, policy, kl, all);
        uint32_t tokens = lanes_sum(all.tokens - before, lanes < 64 ? lanes : 64);
        if (lanes > 64) {
            if (threadIdx.x % 64 == 0) tokens_of[set][threadIdx.x / 64] = tokens;
            __syncthreads();
            tokens = 0;
            const uint32_t waves = lanes / 64, mine = threadIdx.x / lanes * waves;
            for (uint32_t w = 0; w < waves; ++w) tokens += tokens_of[set][mine + w];
        }
        const double w = a.mean == EW_MEAN_SEQUENCES && tokens ? 1.0 / (double)tokens : 1.0;
        all.policy += policy * w;
        all.kl += kl * w;
        all.rows += lane == 0 && tokens ? 1 : 0;
        if (r < a.rows && lane == 0) counts[r] = tokens;
    }
}

// Few tokens: one block.
template <bool Ref, bool Few, bool Wave>
__global__ void __launch_bounds__(kSmallBlock) ew_policy_small_kernel(PolicyLossArgs a, uint32_t lanes)
{
    __shared__ PolicySums scratch[kSmallBlock / 64];
    uint32_t *const counts = static_cast<uint32_t *>(a.workspace);
    LaneSums mine;
    add_sequences<Ref, Few, Wave, kSmallBlock>(a, 0, kSmallBlock / lanes, lanes, counts, mine);
    const PolicySums all = block_sums<kSmallBlock / 64>(mine.all(), scratch);
    if (threadIdx.x == 0) write_loss(a, all);
    if (a.weights)
        for (uint32_t r = threadIdx.x; r < a.rows; r += kSmallBlock)
            a.weights[r] = token_weight(a, all, counts[r]);
}

// Whole sequences: a record of sums a block, a count of tokens a sequence.
template <bool Ref, bool Few, bool Wave>
__global__ void __launch_bounds__(kPolicyBlock) ew_policy_rows_kernel(PolicyLossArgs a, uint32_t lanes,
                                                                     PolicySums *records,
                                                                     uint32_t *counts)
{
    __shared__ PolicySums scratch[kPolicyBlock / 64];
    LaneSums mine;
    const uint64_t per = kPolicyBlock / lanes;
    add_sequences<Ref, Few, Wave, kPolicyBlock>(a, blockIdx.x * per, gridDim.x * per, lanes, counts, mine);
    const PolicySums all = block_sums<kPolicyBlock / 64>(mine.all(), scratch);
    if (threadIdx.x == 0) records[blockIdx.x] = all;
}

// Parts of few long sequences: block (part, sequence), a record each.
template <bool Ref>
__global__ void __launch_bounds__(kPolicyBlock) ew_policy_parts_kernel(PolicyLossArgs a,
                                                                      uint64_t part_tokens,
                                                                      PolicySums *records)
{
    __shared__ PolicySums scratch[kPolicyBlock / 64];
    LaneSums mine;
    const uint64_t from = blockIdx.x * part_tokens, to = from + part_tokens;
    sum_tokens<Ref, false, false>(a.in, blockIdx.y, from, to < a.cols ? (uint32_t)to : a.cols, kPolicyBlock,
                                  threadIdx.x, mine.policy, mine.kl, mine);
    const PolicySums s = block_sums<kPolicyBlock / 64>(mine.all(), scratch);
    if (threadIdx.x == 0) records[(uint64_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// Sequences that are cut into parts: fewer than this, one a CU.
constexpr uint32_t kCutRows = 256;

// The join: every block adds up all records; the first writes loss and stats,
// each the weights of its sequences.  parts > 0: records are of parts of
// sequences, and a sequence's tokens are counted here.
__global__ void __launch_bounds__(kSmallBlock) ew_policy_join_kernel(PolicyLossArgs a,
                                                                    const PolicySums *records,
                                                                    uint32_t n, uint32_t parts,
                                                                    const uint32_t *counts)
{
    __shared__ PolicySums scratch[kSmallBlock / 64];
    __shared__ uint32_t tokens_of[kCutRows];
    PolicySums all{};
    if (parts) {
        for (uint32_t r = threadIdx.x / 64; r < a.rows; r += kSmallBlock / 64) {
            uint32_t tokens = 0;
            for (uint32_t p = threadIdx.x % 64; p < parts; p += 64)
                tokens += (uint32_t)records[(uint64_t)r * parts + p].tokens;
            tokens = lanes_sum(tokens, 64);
            if (threadIdx.x % 64 == 0) tokens_of[r] = tokens;
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < n; i += kSmallBlock)
            add_sequence(all, records[i], a.mean == EW_MEAN_SEQUENCES, tokens_of[i / parts],
                         i % parts == 0);
    } else {
        for (uint32_t i = threadIdx.x; i < n; i += kSmallBlock) all.add(records[i]);
    }
    // (on their way meanwhile)
    const uint64_t first = (uint64_t)blockIdx.x * kSmallBlock + threadIdx.x;
    const uint32_t mine = a.weights && !parts && first < a.rows ? counts[first] : 0;
    all = block_sums<kSmallBlock / 64>(all, scratch);
    if (blockIdx.x == 0 && threadIdx.x == 0) write_loss(a, all);
    if (!a.weights) return;
    for (uint64_t r = first; r < a.rows; r += (uint64_t)gridDim.x * kSmallBlock)
        a.weights[r] = token_weight(a, all, parts ? tokens_of[r] : r == first ? mine : counts[r]);
}

// ---------------------------------------------------------------------------
// Gradient: `lanes` lanes a sequence (or a part of one).  Bound by memory: 4096
// x 4096 tokens, half of them counted, 37.8-39.7 us for 210 MB read and
// written, 5.4 TB/s.
// ---------------------------------------------------------------------------

// Threads of a block: kWideBlock for sequences of more than kWideTokens tokens
// that are not cut into parts, else kPolicyBlock.  us, 512 and 256 threads: 4096
// x 4096 39.7, 41.8; 1500 x 4001 19.0, 20.7; 2048 x 2500 17.8, 17.1; 2048 x 2048
// 13.7, 12.9.
constexpr uint32_t kWideBlock = 512, kWideTokens = 2560;

template <bool Ref, bool Few, bool Wave>
__global__ void __launch_bounds__(kWideBlock) ew_policy_grad_kernel(PolicyGradArgs a, uint32_t lanes,
                                                                     uint64_t part_tokens)
{
    const uint32_t lane = threadIdx.x % lanes, per = blockDim.x / lanes;
    const float dloss = a.dloss ? a.dloss[0] : 1.0f;
    const uint64_t from = blockIdx.y * part_tokens, end = from + part_tokens;
    const uint32_t to = end < a.cols ? (uint32_t)end : a.cols;
    for (uint64_t r0 = (uint64_t)blockIdx.x * per; r0 < a.rows; r0 += (uint64_t)gridDim.x * per) {
        const uint64_t r = r0 + row_in_round<Wave>(lanes);
        if (r >= a.rows) break;
        const PolicyRow row(a.in, r);
        float *const out = a.dlogp + r * a.dlogp_stride;
        const float w = a.weights[r] * dloss;
        each_four<Ref, Few, !Wave>(
            a.in, row, from, to, lanes, lane, [&](const Four &f, const auto &t) {
                f32x4 g{0.0f, 0.0f, 0.0f, 0.0f};
                if (f.counted) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Token k = f.token<Ref>(a.in, j);
                        float slope = k.clipped ? 0.0f : -f.a[j] * k.ratio;
                        if constexpr (Ref) slope -= a.in.kl * k.one;
                        g[j] = f.counts(j) ? w * slope : 0.0f;
                    }
                }
                // (dlogp may be an input, whose other elements another lane takes)
                store_own(t.row(out), t.cols, t.place(lane), __builtin_bit_cast(u32x4, g));
            });
    }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

// One block sums up to so many tokens, if it takes no more than so many rounds:
// 1 x 16000 tokens 8.4 us in two rounds, 6.9 in two launches, whose second
// costs the host 3 us; 100 x 80 10.8 in four, 6.9; 160 x 100 14.6 in five, 6.9;
// 1 x 32000 14.4, 7.2.
constexpr uint64_t kSmallTokens = 16384, kSmallRounds = 4;
// A sequence of more than kBlockTokens tokens (of fewer than kSomeRows
// sequences: kSomeTokens) is a block's, else a wave's or less.  us, a block, a
// wave: 30 x 1000 7.6, 9.9; 1000 x 1000 11.5, 12.8; 1000 x 512 10.9, 9.2; 2000 x
// 1000 14.6, 14.6; 1500 x 4001 22.5, 31.3; 4096 x 4096 39.5, 43.5.
constexpr uint32_t kBlockTokens = 1024, kSomeTokens = 512, kSomeRows = 1024;
// Records of sums: at most this many blocks, five a CU, which the kernel's
// registers (up to 96 a lane) leave room for.  4096 x 4096 and 1115 x 13042 38.7
// and 38.8 us; with 1024 41.9, 45.7; 1536 41.6, 39.2; 2048 42.4, 39.0; 4096 42.5,
// 39.3.
constexpr uint64_t kRecords = 1280;

// Lanes that share a sequence: each takes four tokens at a time.  (Fewer than
// a wave hold all of it.)
static uint32_t lanes_for(uint64_t cols, uint32_t most)
{
    uint32_t lanes = 1;
    while (lanes < most && lanes * 4 < cols) lanes *= 2;
    return lanes;
}

// Few long sequences are cut into parts of whole steps of a block.
static uint64_t parts_of(uint64_t rows, uint64_t cols)
{
    constexpr uint64_t kStep = kPolicyBlock * 4;
    if (rows == 0 || rows >= kCutRows) return 1;
    const uint64_t most = (cols + kStep - 1) / kStep, want = kRecords / rows;
    return most < want ? most : want;
}

size_t policy_loss_workspace(uint64_t rows, uint64_t cols)
{
    return kRecords * sizeof(PolicySums) + (rows * sizeof(uint32_t) + 15) / 16 * 16;
}

// A kernel with or without the reference, of sequences below four tokens, below
// a wave's or others.
#define EW_POLICY_OF(K, REF, cols, lanes)                                            \
    ((cols) < 4     ? reinterpret_cast<const void *>(&K<REF, true, false>)           \
     : (lanes) < 64 ? reinterpret_cast<const void *>(&K<REF, false, false>)          \
                    : reinterpret_cast<const void *>(&K<REF, false, true>))
#define EW_POLICY_KERNEL(K, ref, cols, lanes) \
    ((ref) ? EW_POLICY_OF(K, true, cols, lanes) : EW_POLICY_OF(K, false, cols, lanes))

hipError_t launch_policy_loss(RowType, const PolicyLossArgs &a, hipStream_t s, const char **path)
{
    const bool ref = a.in.ref;
    if ((uint64_t)a.rows * (a.cols ? a.cols : 1) <= kSmallTokens) {
        // more than a wave a sequence where that takes fewer rounds
        uint32_t lanes = lanes_for(a.cols, 64);
        const auto rounds = [&](uint64_t l) {
            const uint64_t at_once = kSmallBlock / l;
            return (a.rows + at_once - 1) / at_once * ((a.cols + 8 * l - 1) / (8 * l));
        };
        if (lanes == 64)
            for (uint32_t more = 128; more <= kSmallBlock; more *= 2)
                if (rounds(more) < rounds(lanes)) lanes = more;
        if (rounds(lanes) <= kSmallRounds) {
            *path = "one block";
            return start(EW_POLICY_KERNEL(ew_policy_small_kernel, ref, a.cols, lanes), dim3(1), kSmallBlock,
                         0, s, a, lanes);
        }
    }
    PolicySums *const records = static_cast<PolicySums *>(a.workspace);
    uint32_t *const counts = reinterpret_cast<uint32_t *>(records + kRecords);
    const uint64_t parts = parts_of(a.rows, a.cols);
    uint32_t n;
    hipError_t e;
    if (parts > 1) {
        *path = "parts of sequences";
        constexpr uint64_t kStep = kPolicyBlock * 4;
        const uint64_t tokens = ((a.cols + parts - 1) / parts + kStep - 1) / kStep * kStep;
        const uint32_t used = (uint32_t)((a.cols + tokens - 1) / tokens);
        n = a.rows * used;
        e = start(ref ? reinterpret_cast<const void *>(&ew_policy_parts_kernel<true>)
                      : reinterpret_cast<const void *>(&ew_policy_parts_kernel<false>),
                  dim3(used, a.rows), kPolicyBlock, 0, s, a, tokens, records);
        if (e != hipSuccess) return e;
        return start(reinterpret_cast<const void *>(&ew_policy_join_kernel), dim3(1), kSmallBlock, 0, s,
                     a, (const PolicySums *)records, n, used, (const uint32_t *)counts);
    }
    *path = "whole sequences";
    const uint32_t lanes = a.cols > (a.rows < kSomeRows ? kSomeTokens : kBlockTokens)
                               ? kPolicyBlock
                               : lanes_for(a.cols, 64);
    const uint64_t blocks = ((uint64_t)a.rows * lanes + kPolicyBlock - 1) / kPolicyBlock;
    n = (uint32_t)(blocks < kRecords ? blocks : kRecords);
    e = start(EW_POLICY_KERNEL(ew_policy_rows_kernel, ref, a.cols, lanes), dim3(n), kPolicyBlock, 0, s, a,
              lanes, records, counts);
    if (e != hipSuccess) return e;
    const uint64_t joins = a.weights ? ((uint64_t)a.rows + kSmallBlock - 1) / kSmallBlock : 1;
    return start(reinterpret_cast<const void *>(&ew_policy_join_kernel),
                 dim3((uint32_t)(joins < kRecords ? joins : kRecords)), kSmallBlock, 0, s, a,
                 (const PolicySums *)records, n, (uint32_t)0, (const uint32_t *)counts);
}

hipError_t launch_policy_grad(RowType, const PolicyGradArgs &a, hipStream_t s, const char **path)
{
    const uint64_t cut = a.cols > kPolicyBlock * 2 ? parts_of(a.rows, a.cols) : 1;
    const uint32_t block = cut == 1 && a.cols > kWideTokens ? kWideBlock : kPolicyBlock;
    const uint32_t lanes = lanes_for(a.cols, block);
    const uint64_t blocks = ((uint64_t)a.rows * lanes + block - 1) / block;
    constexpr uint64_t kStep = kPolicyBlock * 4;
    const uint64_t tokens = cut > 1 ? ((a.cols + cut - 1) / cut + kStep - 1) / kStep * kStep
                                    : (uint64_t)a.cols;
    const uint32_t used = (uint32_t)((a.cols + tokens - 1) / tokens);
    *path = used > 1 ? "parts of sequences" : "whole sequences";
    // a KL term that does not count is not read
    return start(EW_POLICY_KERNEL(ew_policy_grad_kernel, a.in.ref && a.in.kl != 0.0f, a.cols, lanes),
                 dim3(row_blocks(blocks), used), block, 0, s, a, lanes, tokens);
}

}  // namespace ew
