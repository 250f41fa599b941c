// ew_experts.hip -- tokens sorted by expert, their rows moved to the experts and
// back with weights, and the gradient, for CDNA4 (gfx950).

#include "ew_rows_vec.h"

namespace ew {

// ---------------------------------------------------------------------------
// Sorting: a stable counting sort.  Each wave takes consecutive entries, 64 at
// a time, and keeps a counter an expert of its own in LDS; lanes with the same
// expert find each other by ballots over the bits of its number, and the
// lowest of them moves the counter on.  No atomics: an entry's place is a
// function of the entries before it.
// Latency: 64 entries 3.0 us, 8000 8.6 in one block; 65536 of 128 experts 10.1
// in two launches (blocks count; then each adds up all blocks' counts and
// places its entries), 500000 of 256 experts 22.2.
// ---------------------------------------------------------------------------

// Lanes whose key equals this lane's; keys below 2^bits, live lanes only.
__device__ __forceinline__ uint64_t lanes_of(uint32_t key, bool live, uint32_t bits)
{
    uint64_t same = __ballot(live);
    for (uint32_t b = 0; b < bits; ++b) {
        const uint64_t ones = __ballot((key & 1u << b) != 0);
        same &= key & 1u << b ? ones : ~ones;
    }
    return same;
}

// The expert of entry i, or experts if it has none.
__device__ __forceinline__ uint32_t expert_of(const ExpertsSortArgs &a, uint64_t i, uint64_t end)
{
    if (i >= end) return a.cols;
    const int64_t id = a.ids[i];
    return id >= 0 && id < (int64_t)a.cols ? (uint32_t)id : a.cols;
}

// A wave holds this many rounds of 64 entries in registers from the counting
// to the placing (their loads are on their way together), and reads longer
// ones twice.
constexpr uint32_t kHeld = 8;

// How a sorting is split: `chunk` entries a block, `per` (a multiple of 64) a
// counting wave.
struct SortSplit {
    uint32_t chunk, per, waves;      // waves: of a block that count
    uint32_t bits;                   // of an expert's number
};

// The entries [from, end) of a wave.
struct WaveEntries {
    uint64_t from, end;
    __device__ WaveEntries(const ExpertsSortArgs &a, const SortSplit &split)
    {
        const uint32_t wave = threadIdx.x / 64;
        const uint64_t first = (uint64_t)blockIdx.x * split.chunk;
        const uint64_t last = first + split.chunk < a.rows ? first + split.chunk : a.rows;
        from = wave < split.waves ? first + (uint64_t)wave * split.per : last;
        from = from < last ? from : last;
        end = from + split.per < last ? from + split.per : last;
    }
};

// A lane's entry: its expert, and its place among the wave's entries of that
// expert.
struct Entry {
    uint32_t expert, place;
};

// Counts a round's entries, one a lane, in the wave's counters.
__device__ __forceinline__ Entry count_entry(uint32_t expert, uint32_t experts, uint32_t bits,
                                             uint32_t *counter)
{
    const bool live = expert < experts;
    const uint64_t same = lanes_of(expert, live, bits);
    const uint32_t lane = threadIdx.x % 64, first = live ? counter[expert] : 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (live && (uint32_t)__builtin_ctzll(same) == lane)
        counter[expert] = first + (uint32_t)__builtin_popcountll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return Entry{expert, first + (uint32_t)__builtin_popcountll(same & (((uint64_t)1 << lane) - 1))};
}

// The waves' counters of a block's entries by expert, and the entries (Held).
template <bool Held>
__device__ __forceinline__ void count_entries(const ExpertsSortArgs &a, const SortSplit &split,
                                              const WaveEntries &own, Entry (&held)[kHeld],
                                              uint32_t *counters)
{
    const uint32_t experts = a.cols, lane = threadIdx.x % 64;
    uint32_t *const mine = counters + threadIdx.x / 64 * experts;
    if constexpr (Held)
#pragma unroll
        for (uint32_t k = 0; k < kHeld; ++k)
            held[k].expert = expert_of(a, own.from + 64 * k + lane, own.end);
    for (uint32_t i = threadIdx.x; i < split.waves * experts; i += blockDim.x) counters[i] = 0;
    __syncthreads();
    if constexpr (Held) {
#pragma unroll
        for (uint32_t k = 0; k < kHeld; ++k)
            if (own.from + 64 * k < own.end) held[k] = count_entry(held[k].expert, experts, split.bits, mine);
    } else {
        for (uint64_t i = own.from; i < own.end; i += 64)
            count_entry(expert_of(a, i + lane, own.end), experts, split.bits, mine);
    }
    __syncthreads();
}

// The value n lanes before this one in its 16, 0 before the first.
template <int N>
__device__ __forceinline__ uint32_t lanes_before(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x110 + N, 0xf, 0xf, true);
}

__device__ __forceinline__ uint32_t lane_value_u32(uint32_t x, int lane)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x)
{
    x += lanes_before<1>(x);
    x += lanes_before<2>(x);
    x += lanes_before<4>(x);
    x += lanes_before<8>(x);
    const uint32_t a = lane_value_u32(x, 15), b = a + lane_value_u32(x, 31), c = b + lane_value_u32(x, 47);
    const uint32_t row = threadIdx.x % 64 / 16;
    return x + (row == 0 ? 0 : row == 1 ? a : row == 2 ? b : c);
}

// Inclusive sum over a block's threads (at most 16 waves), and the block's sum;
// scratch: a value a wave.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *scratch, uint32_t &all)
{
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, waves = blockDim.x / 64;
    x = wave_scan(x);
    if (lane == 63) scratch[wave] = x;
    __syncthreads();
    const uint32_t before = wave_scan(lane < waves ? scratch[lane] : 0);
    all = lane_value_u32(before, 63);
    const uint32_t mine = (uint32_t)__builtin_amdgcn_readfirstlane((int)wave);
    return x + (mine ? lane_value_u32(before, (int)mine - 1) : 0);
}

// The first row of each expert and the places of a block's entries.  One: all
// entries are the block's; else every block adds up the counts of all blocks
// (totals: a row of them each, by ew_experts_count_kernel).
// LDS: the waves' counters, then (not One) the threads' sums.
template <bool One, bool Held>
__global__ void __launch_bounds__(1024) ew_experts_sort_kernel(ExpertsSortArgs a, SortSplit split,
                                                               const uint32_t *totals)
{
    extern __shared__ uint32_t counters[];
    __shared__ uint32_t scratch[16];
    const uint32_t experts = a.cols, wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const WaveEntries own(a, split);
    uint32_t *const mine = counters + wave * experts;
    // a thread an expert (the host gives a block at least as many)
    const uint32_t e = threadIdx.x, tile = 1u << split.bits;
    // (the blocks' counts are on their way while the entries are counted; threads
    // of the same expert share the blocks)
    uint32_t before = 0, all = 0;
    if constexpr (!One) {
        const uint32_t of = threadIdx.x % tile, part = threadIdx.x / tile, parts = blockDim.x / tile;
        if (of < experts) {
#pragma unroll 8
            for (uint32_t b = part; b < gridDim.x; b += parts) {
                const uint32_t n = totals[b * experts + of];
                all += n;
                before += b < blockIdx.x ? n : 0;
            }
        }
    }
    Entry held[kHeld];
    count_entries<Held>(a, split, own, held, counters);
    if constexpr (!One) {
        uint32_t *const sums = counters + split.waves * experts;
        // within a wave by lane exchanges, then the waves
        for (uint32_t d = tile; d < 64; d *= 2) {
            before += (uint32_t)__shfl_xor((int)before, (int)d);
            all += (uint32_t)__shfl_xor((int)all, (int)d);
        }
        sums[threadIdx.x] = before;
        sums[blockDim.x + threadIdx.x] = all;
        __syncthreads();
        before = all = 0;
        if (threadIdx.x < tile)
#pragma unroll 8
            for (uint32_t q = threadIdx.x; q < blockDim.x; q += tile < 64 ? 64 : tile) {
                before += sums[q];
                all += sums[blockDim.x + q];
            }
    }
    const bool expert = e < experts;
    uint32_t counted[16];                // by the block's waves, read together
#pragma unroll
    for (uint32_t w = 0; w < 16; ++w)
        counted[w] = expert && w < split.waves ? counters[w * experts + e] : 0;
    if constexpr (One)
#pragma unroll
        for (uint32_t w = 0; w < 16; ++w) all += counted[w];
    const uint32_t room = expert ? (all + a.align - 1) / a.align * a.align : 0;
    uint32_t rooms;                      // of all experts
    const uint32_t after = block_scan(room, scratch, rooms);
    if (expert) {
        const uint32_t first = after - room;
        uint32_t next = first + before;
#pragma unroll
        for (uint32_t w = 0; w < 16; ++w) {
            if (w < split.waves) counters[w * experts + e] = next;
            next += counted[w];
        }
        if (blockIdx.x == 0) {
            a.offsets[e] = (int32_t)first;
            if (e + 1 == experts) a.offsets[experts] = (int32_t)after;
            if (a.counts) a.counts[e] = (int32_t)all;
        }
        // rows without an entry; the blocks share the experts
        if (a.source && e % gridDim.x == blockIdx.x)
            for (uint32_t r = first + all; r < after; ++r) a.source[r] = -1;
    }
    __syncthreads();
    const auto put = [&](uint64_t i, const Entry &entry, uint32_t row) {
        if (i >= own.end) return;
        const bool live = entry.expert < experts;
        a.slot[i] = live ? (int32_t)row : -1;
        if (live && a.source) a.source[row] = (int32_t)i;
    };
    if constexpr (Held) {
#pragma unroll
        for (uint32_t k = 0; k < kHeld; ++k)
            if (own.from + 64 * k < own.end)
                put(own.from + 64 * k + lane, held[k],
                    held[k].place + (held[k].expert < experts ? mine[held[k].expert] : 0));
    } else {
        // (the counters start at the experts' rows now)
        for (uint64_t i = own.from; i < own.end; i += 64) {
            const Entry entry = count_entry(expert_of(a, i + lane, own.end), experts, split.bits, mine);
            put(i + lane, entry, entry.place);
        }
    }
    if (a.source)
        for (uint64_t r = rooms + (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; r < a.source_rows;
             r += (uint64_t)gridDim.x * blockDim.x)
            a.source[r] = -1;
}

// Counts of each block's entries by expert.
template <bool Held>
__global__ void __launch_bounds__(1024) ew_experts_count_kernel(ExpertsSortArgs a, SortSplit split,
                                                                uint32_t *totals)
{
    extern __shared__ uint32_t counters[];
    const uint32_t experts = a.cols;
    Entry held[kHeld];
    count_entries<Held>(a, split, WaveEntries(a, split), held, counters);
    for (uint32_t e = threadIdx.x; e < experts; e += blockDim.x) {
        uint32_t n = 0;
#pragma unroll 16
        for (uint32_t w = 0; w < split.waves; ++w) n += counters[w * experts + e];
        totals[blockIdx.x * experts + e] = n;
    }
}

// ---------------------------------------------------------------------------
// Movement of rows, bound by memory.  8192 tokens of 4096 bf16 to 8 experts each,
// one in sixteen dropped: gathered in 97 us, 6.0 TB/s of the rows moved, combined
// in 110 us, 5.8 TB/s; the gradient for 4096 tokens 103.6 us, 5.3 TB/s.  A token at a time: its row is read once (an
// expert's row at a time, which reads a token's row for each choice, took
// 137-151 us, 98-101 this way).  Waves waves share a token (a wave each for short rows, the
// block for long ones) and go along its columns a stretch at a time, 16 bytes a
// lane and vector; the token's own row is read once.  A token's slots lie in
// the lanes of each of its waves.
// ---------------------------------------------------------------------------

constexpr uint32_t kMoveBlock = 256, kMoveWaves = kMoveBlock / 64;

// Which token of a round a thread's wave works on, the same in all its lanes,
// and the thread's place among the token's.
template <uint32_t Waves>
struct Worker {
    static constexpr uint32_t kTokens = kMoveWaves / Waves, kLanes = Waves * 64;
    uint32_t token, place;
    __device__ Worker()
        : token(Waves == kMoveWaves
                    ? 0 : (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / kLanes))),
          place(threadIdx.x % kLanes)
    {
    }
};

// A token's slots, choice j's in lane j: -1 where it names no row.
struct Slots {
    int32_t mine;
    __device__ Slots(const ExpertsMoveArgs &a, uint64_t t) : mine(-1)
    {
        const uint32_t lane = threadIdx.x % 64;
        if (lane < a.top) mine = a.slot[t * a.top + lane];
        if ((uint32_t)mine >= a.places) mine = -1;
    }
    __device__ int32_t of(uint32_t j) const { return __builtin_amdgcn_readlane(mine, (int)j); }
};

// A token's weights, choice j's in lane j.
struct Weights {
    float mine;
    __device__ Weights(const ExpertsMoveArgs &a, uint64_t t) : mine(1.0f)
    {
        const uint32_t lane = threadIdx.x % 64;
        if (a.weights && lane < a.top) mine = a.weights[t * a.top + lane];
    }
    __device__ float of(uint32_t j) const { return lane_value(mine, (int)j); }
};

// A lane's vectors of a stretch of columns, from column `from` on: pieces of
// the stretch, whose row starts `back` elements before it (the last piece of a
// stretch shorter than a vector does).
template <typename T, uint32_t Lanes, uint32_t U, RowFit Fit>
struct Stretch {
    static constexpr uint32_t N = Vec<T>::N, kCols = Lanes * U * N;
    uint64_t from;
    uint32_t cols, place, back;
    __device__ Stretch(uint64_t from_, uint32_t all, uint32_t place_)
        : from(from_), cols(all - from_ < kCols ? (uint32_t)(all - from_) : kCols), place(place_),
          back(from_ ? N : 0)
    {
    }
    __device__ Piece<T, Fit> piece(uint32_t u) const
    {
        return Piece<T, Fit>((place + u * Lanes) * N, cols, back);
    }
    __device__ const T *row(const void *base, uint64_t r, uint64_t stride) const
    {
        return static_cast<const T *>(base) + r * stride + from - back;
    }
    __device__ T *row(void *base, uint64_t r, uint64_t stride) const
    {
        return static_cast<T *>(base) + r * stride + from - back;
    }
    template <bool Nt>
    __device__ u32x4 load(const void *base, uint64_t r, uint64_t stride, uint32_t u) const
    {
        return load_piece<T, Nt>(row(base, r, stride), cols, piece(u));
    }
};

// Zeros in the padding rows of an expert, by one of kPadBlocks blocks of it.  us,
// sorting and gathering, 8, 1 and 32 blocks: 16 tokens, 32 experts, align 16 6.2,
// 7.3, 6.2; 2048 tokens, 64 experts, align 128 48.4, 56.8, 48.5; 64 tokens, 256
// experts, align 16 9.8, 9.8, 12.2.
constexpr uint32_t kPadBlocks = 8;

template <typename T, RowFit Fit>
__device__ __forceinline__ void clear_padding(const ExpertsMoveArgs &a, uint32_t block)
{
    const uint32_t e = block / kPadBlocks;
    using Cols = Stretch<T, kMoveBlock, 1, Fit>;
    const int64_t first = (int64_t)a.offsets[e] + a.counts[e], after = a.offsets[e + 1];
    const int64_t from = first < 0 ? 0 : first, to = after < a.places ? after : a.places;
    for (int64_t r = from + block % kPadBlocks; r < to; r += kPadBlocks) {
        for (uint64_t first = 0; first < a.cols; first += Cols::kCols) {
            const Cols part(first, a.cols, threadIdx.x);
            store_piece(part.row(a.out, (uint64_t)r, a.out_stride), part.cols, part.piece(0),
                           u32x4{0, 0, 0, 0});
        }
    }
}

template <typename T, uint32_t Waves, RowFit Fit>
__global__ void __launch_bounds__(kMoveBlock) ew_experts_gather_kernel(ExpertsMoveArgs a, uint32_t blocks)
{
    constexpr uint32_t U = 1;
    using Cols = Stretch<T, Waves * 64, U, Fit>;
    if (blockIdx.x >= blocks) {
        if (blockIdx.y == 0) clear_padding<T, Fit>(a, blockIdx.x - blocks);
        return;
    }
    const Worker<Waves> worker;
    for (uint64_t t0 = (uint64_t)blockIdx.x * worker.kTokens; t0 < a.rows;
         t0 += (uint64_t)blocks * worker.kTokens) {
        const uint64_t t = t0 + worker.token;
        if (t >= a.rows) break;
        const Slots slots(a, t);
        for (uint64_t first = blockIdx.y * Cols::kCols; first < a.cols; first += gridDim.y * Cols::kCols) {
            const Cols part(first, a.cols, worker.place);
            u32x4 v[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) v[u] = part.template load<false>(a.in, t, a.in_stride, u);
            // (non-temporal stores: 116 us for sorting and gathering, plain ones 133)
            for (uint32_t j = 0; j < a.top; ++j) {
                const int32_t s = slots.of(j);
                if (s < 0) continue;
                T *const row = part.row(a.out, (uint32_t)s, a.out_stride);
#pragma unroll
                for (uint32_t u = 0; u < U; ++u) store_piece(row, part.cols, part.piece(u), v[u]);
            }
        }
    }
}

// C choices of U vectors are on their way together: 8192 x 4096 bf16 4x2 115.5
// us, 8x2 115.5, 8x1 118, 2x4 127 (the gradient 4x2 107.7, 8x2 110, 8x1 118.5,
// 2x4 121.7).
template <typename T, uint32_t Waves, uint32_t C, uint32_t U, RowFit Fit>
__global__ void __launch_bounds__(kMoveBlock) ew_experts_combine_kernel(ExpertsMoveArgs a, uint32_t blocks)
{
    using Cols = Stretch<T, Waves * 64, U, Fit>;
    using Wide = typename Vec<T>::wide;
    const Worker<Waves> worker;
    for (uint64_t t0 = (uint64_t)blockIdx.x * worker.kTokens; t0 < a.rows;
         t0 += (uint64_t)blocks * worker.kTokens) {
        const uint64_t t = t0 + worker.token;
        if (t >= a.rows) break;
        const Slots slots(a, t);
        const Weights weights(a, t);
        for (uint64_t first = blockIdx.y * Cols::kCols; first < a.cols; first += gridDim.y * Cols::kCols) {
            const Cols part(first, a.cols, worker.place);
            u32x4 r[U];
            if (a.residual)
#pragma unroll
                for (uint32_t u = 0; u < U; ++u)
                    r[u] = part.template load<true>(a.residual, t, a.residual_stride, u);
            Wide sum[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) sum[u] = Wide(0.0f);
            for (uint32_t j0 = 0; j0 < a.top; j0 += C) {
                u32x4 v[C][U];
#pragma unroll
                for (uint32_t c = 0; c < C; ++c)
                    if (slots.of(j0 + c) >= 0)
#pragma unroll
                        for (uint32_t u = 0; u < U; ++u)
                            v[c][u] = part.template load<true>(a.z, (uint32_t)slots.of(j0 + c),
                                                               a.z_stride, u);
#pragma unroll
                for (uint32_t c = 0; c < C; ++c)
                    if (slots.of(j0 + c) >= 0) {
                        const float w = weights.of(j0 + c);
#pragma unroll
                        for (uint32_t u = 0; u < U; ++u) {
                            const Wide z = Vec<T>::widen(v[c][u]);
#pragma unroll
                            for (uint32_t k = 0; k < Cols::N; ++k)
                                sum[u][k] = __builtin_fmaf(w, z[k], sum[u][k]);
                        }
                    }
            }
            if (a.residual)
#pragma unroll
                for (uint32_t u = 0; u < U; ++u) sum[u] += Vec<T>::widen(r[u]);
            // (y may be the residual: a piece's other elements may hold sums)
            T *const y = part.row(a.out, t, a.out_stride);
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                store_own(y, part.cols, part.piece(u), Vec<T>::narrow(sum[u]));
        }
    }
}

// dz and the weights' gradients, C choices of U vectors at a time; dy is read
// again for each C choices.
template <typename T, uint32_t Waves, uint32_t C, uint32_t U, RowFit Fit>
__global__ void __launch_bounds__(kMoveBlock) ew_experts_combine_grad_kernel(ExpertsMoveArgs a,
                                                                            uint32_t blocks)
{
    using Cols = Stretch<T, Waves * 64, U, Fit>;
    using Wide = typename Vec<T>::wide;
    // two sets, used in turn: a wave is at most one barrier ahead of another
    __shared__ float scratch[2][kMoveWaves][C];
    if (blockIdx.x >= blocks) {
        if (blockIdx.y == 0) clear_padding<T, Fit>(a, blockIdx.x - blocks);
        return;
    }
    const Worker<Waves> worker;
    const uint32_t lane = threadIdx.x % 64;
    int set = 0;
    // (a token that a block's waves share is the same in all of them: the barrier)
    for (uint64_t t0 = (uint64_t)blockIdx.x * worker.kTokens; t0 < a.rows;
         t0 += (uint64_t)blocks * worker.kTokens) {
        const uint64_t t = t0 + worker.token;
        if (t >= a.rows) break;
        const Slots slots(a, t);
        const Weights weights(a, t);
        for (uint32_t j0 = blockIdx.y * C; j0 < a.top; j0 += gridDim.y * C, set ^= 1) {
            float dots[C];
#pragma unroll
            for (uint32_t c = 0; c < C; ++c) dots[c] = 0.0f;
            for (uint64_t first = 0; first < a.cols; first += Cols::kCols) {
                const Cols part(first, a.cols, worker.place);
                u32x4 d[U], v[C][U];
#pragma unroll
                for (uint32_t u = 0; u < U; ++u) d[u] = part.template load<false>(a.in, t, a.in_stride, u);
#pragma unroll
                for (uint32_t c = 0; c < C; ++c) {
                    const int32_t s = slots.of(j0 + c);
                    if (s >= 0)
#pragma unroll
                        for (uint32_t u = 0; u < U; ++u)
                            v[c][u] = part.template load<true>(a.z, (uint32_t)s, a.z_stride, u);
                }
                Wide g[U];
#pragma unroll
                for (uint32_t u = 0; u < U; ++u) g[u] = Vec<T>::widen(d[u]);
#pragma unroll
                for (uint32_t c = 0; c < C; ++c) {
                    const int32_t s = slots.of(j0 + c);
                    if (s < 0) continue;
                    const float w = weights.of(j0 + c);
                    T *const dz = part.row(a.out, (uint32_t)s, a.out_stride);
#pragma unroll
                    for (uint32_t u = 0; u < U; ++u) {
                        const Wide z = Vec<T>::widen(own_bits(v[c][u], part.cols, part.piece(u)));
#pragma unroll
                        for (uint32_t k = 0; k < Cols::N; ++k) dots[c] = __builtin_fmaf(g[u][k], z[k], dots[c]);
                        // (a partial vector: below)
                        if (Fit != kPart || part.piece(u).skip == 0)
                            store_piece(dz, part.cols, part.piece(u), Vec<T>::narrow(w * g[u]));
                    }
                }
                // what is a partial vector's own, one by one: dz may be z, whose
                // other elements another wave may yet read
                if (Fit == kPart && part.cols % Cols::N != 0)
#pragma unroll 1
                    for (uint32_t c = 0; c < C; ++c) {
                        const int32_t s = slots.of(j0 + c);
                        if (s < 0) continue;
                        const float w = weights.of(j0 + c);
                        T *const dz = part.row(a.out, (uint32_t)s, a.out_stride);
#pragma unroll
                        for (uint32_t u = 0; u < U; ++u)
                            if (part.piece(u).skip != 0)
                                store_own(dz, part.cols, part.piece(u), Vec<T>::narrow(w * g[u]));
                    }
            }
            float mine = 0.0f;             // choice j0 + c in lane c
#pragma unroll
            for (uint32_t c = 0; c < C; ++c) {
                const float dot = wave_reduce<Sum>(dots[c]);
                if (lane == c) mine = dot;
            }
            if constexpr (Waves > 1) {
                if (lane < C) scratch[set][threadIdx.x / 64][lane] = mine;
                __syncthreads();
                if (threadIdx.x < C) {
                    mine = scratch[set][0][lane];
#pragma unroll
                    for (uint32_t w = 1; w < Waves; ++w) mine += scratch[set][w][lane];
                }
            }
            if (worker.place < C && j0 + worker.place < a.top)
                a.dweights[t * a.top + j0 + worker.place] = mine;
        }
    }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

// One block sorts up to this many entries: what its 16 waves hold.
constexpr uint32_t kOneSort = 16 * 64 * kHeld;
// Blocks of a larger sorting: each adds up all the others' counts.  65536
// entries of 128 experts take 12.2 us with 16, 10.3 with 32, 10.1 with 64 or 128;
// 500000 of 256 experts 72.7, 42.2, 22.2, 20.5 (for twice the workspace).
constexpr uint32_t kSortBlocks = 64;
// Counters of a block's waves: 32 KB of LDS.
constexpr uint32_t kCounters = 8192;

size_t experts_sort_workspace(uint64_t entries, uint64_t experts)
{
    return entries <= kOneSort ? 0 : kSortBlocks * ((experts + 3) / 4 * 4) * sizeof(uint32_t);
}

hipError_t launch_experts_sort(RowType, const ExpertsSortArgs &a, hipStream_t s, const char **path)
{
    const uint32_t experts = a.cols;
    SortSplit split{};
    while ((1u << split.bits) < experts) ++split.bits;
    const uint32_t most = kCounters / experts < 16 ? kCounters / experts : 16;    // 8 or more
    const auto waves_for = [&](uint32_t entries) {
        const uint32_t n = (entries + 63) / 64;
        split.waves = n < 1 ? 1 : n < most ? n : most;
        split.per = ((entries + split.waves - 1) / split.waves + 63) / 64 * 64;
        split.chunk = entries;
        // threads enough for an expert each, in whole waves, a power of two
        uint32_t threads = 64;
        while (threads < 1024 && (threads < split.waves * 64 || threads < experts)) threads *= 2;
        return threads;
    };
    if (a.rows <= kOneSort) {
        *path = "one block";
        const uint32_t threads = waves_for(a.rows);
        return start(split.per <= kHeld * 64
                         ? reinterpret_cast<const void *>(&ew_experts_sort_kernel<true, true>)
                         : reinterpret_cast<const void *>(&ew_experts_sort_kernel<true, false>),
                     dim3(1), threads, split.waves * experts * sizeof(uint32_t), s, a, split,
                     (const uint32_t *)nullptr);
    }
    *path = "counts, then places";
    // (fewer blocks where a block's entries are fewer than twice its counts:
    // 65536 entries of 1024 experts 20.4 us with 32, 26.4 with 64)
    const uint32_t least = (a.rows + kSortBlocks - 1) / kSortBlocks;
    const uint32_t chunk = ((least > 2 * experts ? least : 2 * experts) + 1023) / 1024 * 1024;
    const uint32_t blocks = (a.rows + chunk - 1) / chunk, threads = waves_for(chunk);
    const bool held = split.per <= kHeld * 64;
    const size_t lds = split.waves * experts * sizeof(uint32_t);
    uint32_t *const totals = static_cast<uint32_t *>(a.workspace);
    const hipError_t e =
        start(held ? reinterpret_cast<const void *>(&ew_experts_count_kernel<true>)
                   : reinterpret_cast<const void *>(&ew_experts_count_kernel<false>),
              dim3(blocks), threads, lds, s, a, split, totals);
    if (e != hipSuccess) return e;
    return start(held ? reinterpret_cast<const void *>(&ew_experts_sort_kernel<false, true>)
                      : reinterpret_cast<const void *>(&ew_experts_sort_kernel<false, false>),
                 dim3(blocks), threads, lds + 2 * threads * sizeof(uint32_t), s, a, split,
                 (const uint32_t *)totals);
}

// Rows of up to 64 vectors are a wave's, of up to 256 too where tokens abound;
// else a block shares a token, and of few tokens several do: its columns, or
// in the gradient, whose dot products go over them, its choices.  us, bf16 with
// 8 choices a token, this way and one block a token: combine 16 x 7168 3.6, 7.2;
// 100 x 7168 7.2, 13.6; 600 x 4096 10.9, 11.0; its gradient 16 x 7168 6.6, 16.9;
// 300 x 4096 14.6, 16.5; 600 x 4096 24.3, 21.6.  A block and a wave a token, 600
// x 1024: combine 7.3, 7.6; 8192 x 4096: combine 115, 144, gradient 108, 152.
constexpr uint32_t kFewTokens = 512, kSomeTokens = 1024;
// (more stretches of columns than this go round)
constexpr uint32_t kMaxShares = 256;

// The kernel of a type and the row's fit.
#define EW_MOVE_OF(t, K, W, ...)                                             \
    ((t) == kRowF32   ? reinterpret_cast<const void *>(&K<float, W, ##__VA_ARGS__>)    \
     : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16, W, ##__VA_ARGS__>) \
                      : reinterpret_cast<const void *>(&K<__bf16, W, ##__VA_ARGS__>))

struct MoveSplit {
    bool each, tiny;      // a block a token; rows shorter than a vector
    bool few;             // a block a token, and blocks a token are more than one
    bool narrow;          // a vector a lane at most
    uint32_t shares;      // blocks that share a token's columns
    uint32_t blocks;      // of tokens
};

static MoveSplit move_split(RowType t, const ExpertsMoveArgs &a, const char **path)
{
    MoveSplit m;
    const uint32_t vectors = vectors_of(t, a.cols), stretches = (vectors + kMoveBlock - 1) / kMoveBlock;
    m.few = a.rows < kFewTokens && vectors > 64;
    m.each = vectors > (a.rows < kSomeTokens ? 64u : 256u);
    m.narrow = vectors <= 64;
    m.shares = !m.few ? 1 : stretches < kMaxShares ? stretches : kMaxShares;
    m.tiny = a.cols < 16 / (uint32_t)row_elem_size(t);
    m.blocks = row_blocks(m.each ? a.rows : ((uint64_t)a.rows + kMoveWaves - 1) / kMoveWaves);
    *path = m.few ? "blocks a token" : m.each ? "a block a token" : m.tiny ? "short rows" : "a wave a token";
    return m;
}

hipError_t launch_experts_gather(RowType t, const ExpertsMoveArgs &a, hipStream_t s, const char **path)
{
    const MoveSplit m = move_split(t, a, path);
    return start(m.tiny   ? EW_MOVE_OF(t, ew_experts_gather_kernel, 1, kTiny)
                 : m.each ? EW_MOVE_OF(t, ew_experts_gather_kernel, kMoveWaves, kPart)
                          : EW_MOVE_OF(t, ew_experts_gather_kernel, 1, kPart),
                 dim3(m.blocks + a.experts * kPadBlocks, m.shares), kMoveBlock, 0, s, a, m.blocks);
}

hipError_t launch_experts_combine(RowType t, const ExpertsMoveArgs &a, hipStream_t s, const char **path)
{
    const MoveSplit m = move_split(t, a, path);
#define EW_COMBINE(W, C, U, FIT) EW_MOVE_OF(t, ew_experts_combine_kernel, W, C, U, FIT)
    return start(m.tiny         ? EW_COMBINE(1, 8, 1, kTiny)
                 : m.few        ? EW_COMBINE(kMoveWaves, 8, 1, kPart)
                 : m.narrow     ? EW_COMBINE(1, 8, 1, kPart)
                 : a.top <= 2   ? m.each ? EW_COMBINE(kMoveWaves, 2, 4, kPart) : EW_COMBINE(1, 2, 4, kPart)
                 : m.each       ? EW_COMBINE(kMoveWaves, 4, 2, kPart)
                                : EW_COMBINE(1, 4, 2, kPart),
                 dim3(m.blocks, m.shares), kMoveBlock, 0, s, a, m.blocks);
#undef EW_COMBINE
}

hipError_t launch_experts_combine_grad(RowType t, const ExpertsMoveArgs &a, hipStream_t s,
                                       const char **path)
{
    const MoveSplit m = move_split(t, a, path);
#define EW_GRAD(W, C, U, FIT) EW_MOVE_OF(t, ew_experts_combine_grad_kernel, W, C, U, FIT)
    return start(m.tiny                 ? EW_GRAD(1, 8, 1, kTiny)
                 : m.narrow             ? EW_GRAD(1, 8, 1, kPart)
                 : m.few || a.top <= 2  ? m.each ? EW_GRAD(kMoveWaves, 2, 4, kPart) : EW_GRAD(1, 2, 4, kPart)
                 : m.each               ? EW_GRAD(kMoveWaves, 4, 2, kPart)
                                        : EW_GRAD(1, 4, 2, kPart),
                 dim3(m.blocks + a.experts * kPadBlocks, m.few ? (a.top + 1) / 2 : 1), kMoveBlock, 0, s, a,
                 m.blocks);
#undef EW_GRAD
}

}  // namespace ew
