// ew_rows_args.h -- the row operators' arguments and launchers, shared by
// their host API (ew_rows_api.cpp) and kernels (ew_norm.hip, ew_vocab.hip).
// Not installed; not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ew {

enum RowType : int { kRowF32 = 0, kRowF16, kRowBF16 };

constexpr int row_elem_size(RowType t) { return t == kRowF32 ? 4 : 2; }

// Strides are in elements.  A pointer that is optional and absent is null.
struct NormArgs {
    const void *x, *residual, *weight;
    void *y, *total;            // y: the type's elements, or e4m3 bytes
    float *rstd, *scales;       // scales != null: y is e4m3
    uint64_t x_stride, residual_stride, y_stride, total_stride;
    uint32_t rows, cols;
    uint32_t group, groups;     // columns per scale (cols for one a row), scales per row
    float eps;
};

struct NormGradArgs {
    const void *dy, *x, *weight, *dtotal;
    const float *rstd;
    void *dx;
    float *dweight, *partial;   // partial: sums of dweight over parts of the rows
    uint64_t dy_stride, x_stride, dtotal_stride, dx_stride;
    uint32_t rows, cols;
};

struct LogprobsArgs {
    const void *logits;
    const int64_t *targets;
    float *logp, *entropy, *lse, *top_logp;
    int64_t *top_ids;
    void *workspace;
    uint64_t stride;
    uint32_t rows, cols, top;
    float scale;
};

struct LogprobsGradArgs {
    const void *logits;
    const int64_t *targets;
    const float *lse, *entropy, *dlogp, *dentropy;
    void *dlogits;
    uint64_t stride, dlogits_stride;
    uint32_t rows, cols;
    float scale;
};

// Below it the difference of two logits may overflow though scale times it is
// an ordinary number.
constexpr float kTinyScale = 0x1p-64f;

// scale in two factors: the exact part that logits take before their
// difference is formed, and what the difference takes.
struct TeacherScale {
    float part, whole;
};
constexpr TeacherScale teacher_scale(float scale)
{
    return scale < kTinyScale ? TeacherScale{0.5f, 2.0f * scale} : TeacherScale{1.0f, scale};
}

struct DistillArgs {
    const void *logits;
    const float *teacher;
    const int64_t *ids;
    float *loss, *lse;
    void *workspace;
    uint64_t stride;
    uint32_t rows, cols, kept;
    float scale;
    TeacherScale by;
};

struct DistillGradArgs {
    const void *logits;
    const float *teacher;
    const int64_t *ids;
    const float *lse, *dloss;
    void *dlogits;
    uint64_t stride, dlogits_stride;
    uint32_t rows, cols, kept;
    float scale;
    TeacherScale by;
};

// Most alternatives a call ranks: one per lane of a wave.
constexpr uint32_t kTopMax = 64;

// Most kept entries of a row: the distillation's gradient holds a row's in LDS.
constexpr uint32_t kMaxKept = 1024;

// Workspace bytes: a function of the sizes alone.
size_t norm_grad_workspace(uint64_t rows, uint64_t cols);
size_t logprobs_workspace(uint64_t rows, uint64_t cols, uint64_t top);
size_t distill_workspace(uint64_t rows, uint64_t cols);

// Each launches its kernels on s; *path names what ran (for the log).
hipError_t launch_norm(RowType t, const NormArgs &a, hipStream_t s, const char **path);
hipError_t launch_norm_grad(RowType t, const NormGradArgs &a, hipStream_t s,
                            const char **path);
hipError_t launch_logprobs(RowType t, const LogprobsArgs &a, hipStream_t s,
                           const char **path);
hipError_t launch_logprobs_grad(RowType t, const LogprobsGradArgs &a, hipStream_t s,
                                const char **path);
hipError_t launch_distill(RowType t, const DistillArgs &a, hipStream_t s,
                          const char **path);
hipError_t launch_distill_grad(RowType t, const DistillGradArgs &a, hipStream_t s,
                               const char **path);

}  // namespace ew
