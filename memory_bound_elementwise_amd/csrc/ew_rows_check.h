// ew_rows_check.h -- what the host API's files of the row operators
// (ew_rows_api.cpp, ew_train_api.cpp) share: the checks of buffers and sizes,
// and the launch with its log.  Not installed; not part of the C ABI.
#pragma once

#include "ew.h"
#include "ew_host.h"
#include "ew_rows_args.h"

#include <cmath>
#include <cstdio>

namespace ew {

// One buffer of a call: rows pieces of row_bytes, stride_bytes apart
// (contiguous buffers: one piece).
struct Span {
    const void *p;
    size_t align;          // element size
    uint64_t rows, row_bytes, stride_bytes;
    bool required;
};

inline uintptr_t addr(const Span &s) { return reinterpret_cast<uintptr_t>(s.p); }
inline bool live(const Span &s) { return s.p != nullptr && s.rows != 0 && s.row_bytes != 0; }
inline uint64_t extent(const Span &s) { return (s.rows - 1) * s.stride_bytes + s.row_bytes; }

inline Span matrix(const void *p, int es, size_t stride, size_t rows, size_t cols, bool required = true)
{
    // a single row's stride is never used
    return Span{p, (size_t)es, rows, (uint64_t)cols * (uint64_t)es,
                (rows > 1 ? (uint64_t)stride : (uint64_t)cols) * (uint64_t)es, required};
}

inline Span array(const void *p, int es, uint64_t n, bool required = true)
{
    return Span{p, (size_t)es, n ? 1u : 0u, n * (uint64_t)es, n * (uint64_t)es, required};
}

// Whether two buffers share a byte.  Equal strides: the pieces repeat with
// that period, so only the offset within it matters.  Different strides:
// whether their extents meet.
inline bool overlap(const Span &a, const Span &b)
{
    const uintptr_t alo = addr(a), blo = addr(b);
    if (alo >= blo + extent(b) || blo >= alo + extent(a)) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride_bytes == b.stride_bytes) {
        const uint64_t st = a.stride_bytes;
        const uint64_t d = blo >= alo ? (blo - alo) % st : (st - (alo - blo) % st) % st;
        return d < a.row_bytes || d + b.row_bytes > st;
    }
    return true;
}

inline bool same(const Span &a, const Span &b)
{
    return a.p == b.p && a.rows == b.rows && a.row_bytes == b.row_bytes &&
           a.stride_bytes == b.stride_bytes;
}

constexpr uint64_t kMaxDim = (uint64_t)1 << 31;
constexpr uint64_t kMaxBytes = (uint64_t)1 << 62;

// Null pointers, strides and address wrap, then alignment, then overlap: outs[i] may be exactly
// ins[j] where bit j of alias[i] is set, and never meets another output.
inline ew_status_t check(const Span *ins, int n_in, const Span *outs, int n_out, const unsigned *alias)
{
    const auto sizes_ok = [](const Span &s) {
        if (!s.p) return !s.required || s.rows == 0 || s.row_bytes == 0;
        if (!live(s)) return true;
        if (s.stride_bytes < s.row_bytes) return false;
        const unsigned __int128 bytes =
            (unsigned __int128)(s.rows - 1) * s.stride_bytes + s.row_bytes;
        return bytes < kMaxBytes && reinterpret_cast<uintptr_t>(s.p) <= UINTPTR_MAX - (uint64_t)bytes;
    };
    for (int i = 0; i < n_in; ++i)
        if (!sizes_ok(ins[i])) return EW_ERR_INVALID_ARG;
    for (int i = 0; i < n_out; ++i)
        if (!sizes_ok(outs[i])) return EW_ERR_INVALID_ARG;
    for (int i = 0; i < n_in; ++i)
        if (live(ins[i]) && addr(ins[i]) % ins[i].align) return EW_ERR_MISALIGNED;
    for (int i = 0; i < n_out; ++i)
        if (live(outs[i]) && addr(outs[i]) % outs[i].align) return EW_ERR_MISALIGNED;
    for (int i = 0; i < n_out; ++i) {
        if (!live(outs[i])) continue;
        for (int j = 0; j < n_in; ++j) {
            if (!live(ins[j]) || !overlap(outs[i], ins[j])) continue;
            if ((alias[i] >> j & 1u) && same(outs[i], ins[j])) continue;
            return EW_ERR_OVERLAP;
        }
        for (int j = 0; j < i; ++j)
            if (live(outs[j]) && overlap(outs[i], outs[j])) return EW_ERR_OVERLAP;
    }
    return EW_OK;
}

inline bool dims_ok(size_t rows, size_t cols) { return rows < kMaxDim && cols < kMaxDim; }

// A stride no element offset overflows 64 bits with (checked per span too).
inline bool stride_ok(size_t stride) { return stride < ((size_t)1 << 60); }

inline bool scale_ok(float scale) { return std::isfinite(scale) && scale > 0.0f; }

template <class Args>
ew_status_t launch(const char *op, RowType t, const Args &a, hipStream_t s,
                   hipError_t (*fn)(RowType, const Args &, hipStream_t, const char **))
{
    int cus = 0;
    const ew_status_t st = host_device(&cus);
    if (st != EW_OK) return st;
    const char *path = "";
    const hipError_t e = fn(t, a, s, &path);
    if (host_log_enabled()) {
        static const char *const names[] = {"f32", "f16", "bf16"};
        std::fprintf(stderr, "[ew] %s_%s rows=%u cols=%u path=%s\n", op, names[t], a.rows, a.cols,
                     path);
    }
    return e == hipSuccess ? EW_OK : host_fail(e);
}

}  // namespace ew
