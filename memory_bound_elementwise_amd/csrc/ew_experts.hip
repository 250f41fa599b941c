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
// ---------------------------------------------------------------------------

constexpr uint32_t kSortWaves = 4, kSortBlock = kSortWaves * 64;

// Lanes whose key equals this lane's; keys below 2^bits, live lanes only.
__device__ __forceinline__ uint64_t lanes_of(uint32_t key, bool live, uint32_t bits)
{
    uint64_t same = __ballot(live);
    for (uint32_t b = 0; b < bits; ++b) {
        const bool one = key >> b & 1u;
        const uint64_t ones = __ballot(one);
        same &= one ? ones : ~ones;
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

// Counts of a wave's entries [from, end) by expert, added to its counters.
__device__ __forceinline__ void count_entries(const ExpertsSortArgs &a, uint64_t from, uint64_t end,
                                              uint32_t bits, uint32_t *counter)
{
    const uint32_t lane = threadIdx.x % 64;
    for (uint64_t i = from; i < end; i += 64) {
        const uint32_t e = expert_of(a, i + lane, end);
        const uint64_t same = lanes_of(e, e < a.cols, bits);
        if (e < a.cols && (uint32_t)__builtin_ctzll(same) == lane)
            counter[e] += (uint32_t)__builtin_popcountll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// Rows of a wave's entries: counter[e] is the row of its next one of expert e.
__device__ __forceinline__ void place_entries(const ExpertsSortArgs &a, uint64_t from, uint64_t end,
                                              uint32_t bits, uint32_t *counter)
{
    const uint32_t lane = threadIdx.x % 64;
    for (uint64_t i = from; i < end; i += 64) {
        const uint32_t e = expert_of(a, i + lane, end);
        const bool live = e < a.cols;
        const uint64_t same = lanes_of(e, live, bits);
        const uint32_t first = live ? counter[e] : 0;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (live && (uint32_t)__builtin_ctzll(same) == lane)
            counter[e] = first + (uint32_t)__builtin_popcountll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const uint32_t row = first + (uint32_t)__builtin_popcountll(same & (((uint64_t)1 << lane) - 1));
        if (i + lane < end) {
            a.slot[i + lane] = live ? (int32_t)row : -1;
            if (live && a.source) a.source[row] = (int32_t)(i + lane);
        }
    }
}

// Inclusive sum over a block's threads; scratch: a value a wave.
template <uint32_t Waves>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *scratch)
{
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
    for (uint32_t d = 1; d < 64; d *= 2) {
        const uint32_t up = (uint32_t)__shfl_up((int)x, d);
        if (lane >= d) x += up;
    }
    __syncthreads();
    if (lane == 63) scratch[wave] = x;
    __syncthreads();
    for (uint32_t w = 0; w < wave; ++w) x += scratch[w];
    return x;
}

// One launch sorts what a block can (kOne), else every block adds up the
// counts of those before it (`totals`: a row of counts a block, by
// ew_experts_count_kernel).
// LDS: Waves counters an expert, then the experts' first rows.
template <uint32_t Waves, bool One>
__global__ void __launch_bounds__(Waves * 64) ew_experts_sort_kernel(ExpertsSortArgs a, uint32_t chunk,
                                                                    uint32_t bits,
                                                                    const uint32_t *totals)
{
    constexpr uint32_t kThreads = Waves * 64;
    extern __shared__ uint32_t counters[];
    __shared__ uint32_t scratch[Waves];
    const uint32_t experts = a.cols, wave = threadIdx.x / 64;
    uint32_t *const mine = counters + wave * experts;
    // the wave's own entries
    const uint64_t block_from = (uint64_t)blockIdx.x * chunk;
    const uint64_t block_end = block_from + chunk < a.rows ? block_from + chunk : a.rows;
    uint64_t from = block_from + (uint64_t)wave * (chunk / Waves);
    uint64_t end = from + chunk / Waves;
    from = from < block_end ? from : block_end;
    end = end < block_end ? end : block_end;
    for (uint32_t i = threadIdx.x; i < Waves * experts; i += kThreads) counters[i] = 0;
    __syncthreads();
    count_entries(a, from, end, bits, mine);
    __syncthreads();
    // the experts' rows: kThreads of them at a time
    uint32_t start = 0;
    for (uint32_t e0 = 0; e0 < experts; e0 += kThreads) {
        const uint32_t e = e0 + threadIdx.x;
        uint32_t before = 0, all = 0;
        if (e < experts) {
            if constexpr (One) {
                for (uint32_t w = 0; w < Waves; ++w) all += counters[w * experts + e];
            } else {
                for (uint32_t b = 0; b < gridDim.x; ++b) {
                    const uint32_t n = totals[(uint64_t)b * experts + e];
                    all += n;
                    before += b < blockIdx.x ? n : 0;
                }
            }
        }
        const uint32_t room = (all + a.align - 1) / a.align * a.align;
        const uint32_t after = start + block_scan<Waves>(room, scratch);
        if (e < experts) {
            const uint32_t first = after - room;
            uint32_t next = first + before;
            for (uint32_t w = 0; w < Waves; ++w) {
                const uint32_t n = counters[w * experts + e];
                counters[w * experts + e] = next;
                next += n;
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
        for (uint32_t w = 0; w < Waves; ++w) start += scratch[w];
        __syncthreads();
    }
    if (a.source)
        for (uint64_t r = start + (uint64_t)blockIdx.x * kThreads + threadIdx.x; r < a.source_rows;
             r += (uint64_t)gridDim.x * kThreads)
            a.source[r] = -1;
    place_entries(a, from, end, bits, mine);
}

// Counts of each block's entries by expert.
__global__ void __launch_bounds__(kSortBlock) ew_experts_count_kernel(ExpertsSortArgs a, uint32_t chunk,
                                                                     uint32_t bits, uint32_t *totals)
{
    extern __shared__ uint32_t counters[];
    const uint32_t experts = a.cols, wave = threadIdx.x / 64;
    const uint64_t block_from = (uint64_t)blockIdx.x * chunk;
    const uint64_t block_end = block_from + chunk < a.rows ? block_from + chunk : a.rows;
    uint64_t from = block_from + (uint64_t)wave * (chunk / kSortWaves);
    uint64_t end = from + chunk / kSortWaves;
    from = from < block_end ? from : block_end;
    end = end < block_end ? end : block_end;
    for (uint32_t i = threadIdx.x; i < kSortWaves * experts; i += kSortBlock) counters[i] = 0;
    __syncthreads();
    count_entries(a, from, end, bits, counters + wave * experts);
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < experts; e += kSortBlock) {
        uint32_t n = 0;
        for (uint32_t w = 0; w < kSortWaves; ++w) n += counters[w * experts + e];
        totals[(uint64_t)blockIdx.x * experts + e] = n;
    }
}

// ---------------------------------------------------------------------------
// Movement of rows.  Lanes threads of a block share a token and go along its
// columns 16 bytes at a time; the token's row is read once.
// ---------------------------------------------------------------------------

constexpr uint32_t kMoveBlock = 256;

// Zeros in the padding rows of expert e, by a block.
template <typename T>
__device__ __forceinline__ void clear_padding(const ExpertsMoveArgs &a, uint32_t e)
{
    constexpr uint32_t N = Vec<T>::N;
    const int64_t first = (int64_t)a.offsets[e] + a.counts[e], after = a.offsets[e + 1];
    const int64_t from = first < 0 ? 0 : first, to = after < a.places ? after : a.places;
    for (int64_t r = from; r < to; ++r) {
        T *const row = static_cast<T *>(a.out) + (uint64_t)r * a.out_stride;
        for (uint64_t at = threadIdx.x * N; at < a.cols; at += kMoveBlock * N)
            store_vec(row, a.cols, (uint32_t)at, u32x4{0, 0, 0, 0});
    }
}

// A token's slot j, or -1 where it names no row.
__device__ __forceinline__ int32_t place_of(const ExpertsMoveArgs &a, uint64_t t, uint32_t j)
{
    const int32_t s = a.slot[t * a.top + j];
    return (uint32_t)s < a.places ? s : -1;
}

template <typename T, uint32_t Lanes>
__global__ void __launch_bounds__(kMoveBlock) ew_experts_gather_kernel(ExpertsMoveArgs a, uint32_t blocks)
{
    constexpr uint32_t N = Vec<T>::N, kTokens = kMoveBlock / Lanes;
    if (blockIdx.x >= blocks) {
        if (blockIdx.y == 0) clear_padding<T>(a, blockIdx.x - blocks);
        return;
    }
    const uint32_t lane = threadIdx.x % Lanes;
    for (uint64_t t0 = (uint64_t)blockIdx.x * kTokens; t0 < a.rows; t0 += (uint64_t)blocks * kTokens) {
        const uint64_t t = t0 + threadIdx.x / Lanes;
        if (t >= a.rows) break;
        const T *const x = static_cast<const T *>(a.in) + t * a.in_stride;
        for (uint64_t at = (blockIdx.y * (uint64_t)Lanes + lane) * N; at < a.cols;
             at += (uint64_t)gridDim.y * Lanes * N) {
            const u32x4 v = settle<T>(load_vec<T, true>(x, a.cols, (uint32_t)at), a.cols, (uint32_t)at);
            for (uint32_t j = 0; j < a.top; ++j) {
                const int32_t s = place_of(a, t, j);
                if (s >= 0)
                    store_vec(static_cast<T *>(a.out) + (uint64_t)(uint32_t)s * a.out_stride, a.cols,
                              (uint32_t)at, v);
            }
        }
    }
}

template <typename T, uint32_t Lanes>
__global__ void __launch_bounds__(kMoveBlock) ew_experts_combine_kernel(ExpertsMoveArgs a, uint32_t blocks)
{
    constexpr uint32_t N = Vec<T>::N, kTokens = kMoveBlock / Lanes;
    using Wide = typename Vec<T>::wide;
    const uint32_t lane = threadIdx.x % Lanes;
    for (uint64_t t0 = (uint64_t)blockIdx.x * kTokens; t0 < a.rows; t0 += (uint64_t)blocks * kTokens) {
        const uint64_t t = t0 + threadIdx.x / Lanes;
        if (t >= a.rows) break;
        T *const y = static_cast<T *>(a.out) + t * a.out_stride;
        const T *const res = static_cast<const T *>(a.residual) + t * a.residual_stride;
        for (uint64_t at64 = (blockIdx.y * (uint64_t)Lanes + lane) * N; at64 < a.cols;
             at64 += (uint64_t)gridDim.y * Lanes * N) {
            const uint32_t at = (uint32_t)at64;
            Wide sum(0.0f);
            if (a.residual) sum = Vec<T>::widen(settle<T>(load_vec<T, true>(res, a.cols, at), a.cols, at));
            for (uint32_t j = 0; j < a.top; ++j) {
                const int32_t s = place_of(a, t, j);
                if (s < 0) continue;
                const T *const z = static_cast<const T *>(a.z) + (uint64_t)(uint32_t)s * a.z_stride;
                const Wide v = Vec<T>::widen(settle<T>(load_vec<T, true>(z, a.cols, at), a.cols, at));
                const float w = a.weights ? a.weights[t * a.top + j] : 1.0f;
#pragma unroll
                for (uint32_t k = 0; k < N; ++k) sum[k] = __builtin_fmaf(w, v[k], sum[k]);
            }
            store_vec(y, a.cols, at, Vec<T>::narrow(sum));
        }
    }
}

// dz and the weights' gradients: one choice after another, the token's dy
// again for each (from the caches).
template <typename T, uint32_t Lanes>
__global__ void __launch_bounds__(kMoveBlock) ew_experts_combine_grad_kernel(ExpertsMoveArgs a,
                                                                            uint32_t blocks)
{
    constexpr uint32_t N = Vec<T>::N, kTokens = kMoveBlock / Lanes;
    using Wide = typename Vec<T>::wide;
    __shared__ float scratch[2][kMoveBlock / 64];
    if (blockIdx.x >= blocks) {
        clear_padding<T>(a, blockIdx.x - blocks);
        return;
    }
    const uint32_t lane = threadIdx.x % Lanes;
    int set = 0;
    for (uint64_t t0 = (uint64_t)blockIdx.x * kTokens; t0 < a.rows; t0 += (uint64_t)blocks * kTokens) {
        const uint64_t t = t0 + threadIdx.x / Lanes;
        const bool live = t < a.rows;
        const T *const dy = static_cast<const T *>(a.in) + t * a.in_stride;
        for (uint32_t j = 0; j < a.top; ++j, set ^= 1) {
            const int32_t s = live ? place_of(a, t, j) : -1;
            float dot = 0.0f;
            if (s >= 0) {
                const T *const z = static_cast<const T *>(a.z) + (uint64_t)(uint32_t)s * a.z_stride;
                T *const dz = static_cast<T *>(a.out) + (uint64_t)(uint32_t)s * a.out_stride;
                const float w = a.weights[t * a.top + j];
                for (uint64_t at64 = lane * N; at64 < a.cols; at64 += Lanes * N) {
                    const uint32_t at = (uint32_t)at64;
                    const Wide g = Vec<T>::widen(settle<T>(load_vec<T, false>(dy, a.cols, at), a.cols, at));
                    const Wide v = Vec<T>::widen(settle<T>(load_vec<T, true>(z, a.cols, at), a.cols, at));
#pragma unroll
                    for (uint32_t k = 0; k < N; ++k) dot = __builtin_fmaf(g[k], v[k], dot);
                    store_vec(dz, a.cols, at, Vec<T>::narrow(w * g));
                }
            }
            if constexpr (Lanes <= 64) {
#pragma unroll
                for (uint32_t d = 1; d < Lanes; d *= 2) dot += __shfl_xor(dot, (int)d);
            } else {
                dot = block_reduce<Sum, kMoveBlock / 64>(dot, scratch[set]);
            }
            if (live && lane == 0) a.dweights[t * a.top + j] = dot;
        }
    }
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

// One block sorts up to this many entries.
constexpr uint64_t kOneSort = 8192;
// Blocks of a larger sorting: each adds up all the others' counts.
constexpr uint64_t kSortBlocks = 128;

size_t experts_sort_workspace(uint64_t entries, uint64_t experts)
{
    return entries <= kOneSort ? 0 : kSortBlocks * ((experts + 3) / 4 * 4) * sizeof(uint32_t);
}

hipError_t launch_experts_sort(RowType, const ExpertsSortArgs &a, hipStream_t s, const char **path)
{
    uint32_t bits = 0;
    while ((1u << bits) < a.cols) ++bits;
    if (a.rows <= kOneSort) {
        *path = "one block";
        // 32 KB of counters at most
        const uint32_t waves = a.cols <= 512 ? 16 : 8, block = waves * 64;
        const uint32_t chunk = (a.rows + block - 1) / block * block;
        return start(waves == 16 ? reinterpret_cast<const void *>(&ew_experts_sort_kernel<16, true>)
                                 : reinterpret_cast<const void *>(&ew_experts_sort_kernel<8, true>),
                     dim3(1), block, waves * a.cols * sizeof(uint32_t), s, a, chunk, bits,
                     (const uint32_t *)nullptr);
    }
    *path = "counts, then places";
    const uint64_t per = ((uint64_t)a.rows + kSortBlocks - 1) / kSortBlocks;
    const uint32_t chunk = (uint32_t)((per + kSortBlock - 1) / kSortBlock * kSortBlock);
    const uint32_t blocks = (a.rows + chunk - 1) / chunk;
    const size_t lds = kSortWaves * a.cols * sizeof(uint32_t);
    uint32_t *const totals = static_cast<uint32_t *>(a.workspace);
    const hipError_t e = start(reinterpret_cast<const void *>(&ew_experts_count_kernel), dim3(blocks),
                               kSortBlock, lds, s, a, chunk, bits, totals);
    if (e != hipSuccess) return e;
    return start(reinterpret_cast<const void *>(&ew_experts_sort_kernel<kSortWaves, false>), dim3(blocks),
                 kSortBlock, lds, s, a, chunk, bits, (const uint32_t *)totals);
}

// Lanes of a token: 16, 64 or the block.
#define EW_MOVE_KERNEL(t, K, lanes)                                                             \
    ((lanes) == 16   ? ((t) == kRowF32   ? reinterpret_cast<const void *>(&K<float, 16>)        \
                        : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16, 16>)     \
                                         : reinterpret_cast<const void *>(&K<__bf16, 16>))      \
     : (lanes) == 64 ? ((t) == kRowF32   ? reinterpret_cast<const void *>(&K<float, 64>)        \
                        : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16, 64>)     \
                                         : reinterpret_cast<const void *>(&K<__bf16, 64>))      \
                     : ((t) == kRowF32   ? reinterpret_cast<const void *>(&K<float, 256>)       \
                        : (t) == kRowF16 ? reinterpret_cast<const void *>(&K<_Float16, 256>)    \
                                         : reinterpret_cast<const void *>(&K<__bf16, 256>)))

static uint32_t move_lanes(uint32_t vectors) { return vectors <= 16 ? 16 : vectors <= 64 ? 64 : kMoveBlock; }

static uint32_t token_blocks(uint64_t rows, uint32_t lanes)
{
    const uint64_t per = kMoveBlock / lanes;
    return row_blocks((rows + per - 1) / per);
}

hipError_t launch_experts_gather(RowType t, const ExpertsMoveArgs &a, hipStream_t s, const char **path)
{
    *path = "by tokens";
    const uint32_t lanes = move_lanes(vectors_of(t, a.cols)), blocks = token_blocks(a.rows, lanes);
    return start(EW_MOVE_KERNEL(t, ew_experts_gather_kernel, lanes), dim3(blocks + a.experts), kMoveBlock,
                 0, s, a, blocks);
}

hipError_t launch_experts_combine(RowType t, const ExpertsMoveArgs &a, hipStream_t s, const char **path)
{
    *path = "by tokens";
    const uint32_t lanes = move_lanes(vectors_of(t, a.cols)), blocks = token_blocks(a.rows, lanes);
    return start(EW_MOVE_KERNEL(t, ew_experts_combine_kernel, lanes), dim3(blocks), kMoveBlock, 0, s, a,
                 blocks);
}

hipError_t launch_experts_combine_grad(RowType t, const ExpertsMoveArgs &a, hipStream_t s,
                                       const char **path)
{
    *path = "by tokens";
    const uint32_t lanes = move_lanes(vectors_of(t, a.cols)), blocks = token_blocks(a.rows, lanes);
    return start(EW_MOVE_KERNEL(t, ew_experts_combine_grad_kernel, lanes), dim3(blocks + a.experts),
                 kMoveBlock, 0, s, a, blocks);
}

}  // namespace ew
