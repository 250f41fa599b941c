// ew_rows_args.h -- the row operators' arguments and launchers, shared by
// their host API (ew_rows_api.cpp) and kernels (ew_norm.hip, ew_vocab.hip,
// ew_layernorm.hip, ew_policy.hip, ew_experts.hip).  Not installed; not part of
// the C ABI.
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

struct LayerNormArgs {
    const void *x, *residual, *weight, *bias;
    void *y, *total;
    float *mean, *rstd;
    uint64_t x_stride, residual_stride, y_stride, total_stride;
    double by_cols;             // 1 / cols
    uint32_t rows, cols;
    float eps;
};

struct LayerNormGradArgs {
    const void *dy, *x, *weight, *dtotal;
    const float *mean, *rstd;
    void *dx;
    float *dweight, *dbias;
    void *workspace;
    uint64_t dy_stride, x_stride, dtotal_stride, dx_stride;
    uint32_t rows, cols;
};

// What the policy loss and its gradient read alike.
struct PolicyTokens {
    const float *logp, *old, *ref, *advantage;
    const uint8_t *mask;
    uint64_t logp_stride, old_stride, ref_stride, mask_stride;
    uint64_t advantage_stride;  // 0: one value a row
    double above, below;        // borders of logp - old
    float most, least;          // the ratios at them
    float kl;                   // 0: without its term in loss and gradient
};

struct PolicyLossArgs {
    PolicyTokens in;
    float *loss, *stats, *weights;
    void *workspace;
    uint32_t rows, cols;
    float scale;
    int mean;                   // an ew_mean_t
};

struct PolicyGradArgs {
    PolicyTokens in;
    const float *weights, *dloss;
    float *dlogp;
    uint64_t dlogp_stride;
    uint32_t rows, cols;
};

struct ExpertsSortArgs {
    const int64_t *ids;
    int32_t *slot, *offsets, *counts, *source;
    void *workspace;
    uint32_t align;
    uint32_t source_rows;       // ew_experts_rows()
    uint32_t rows, cols;        // entries, experts
};

// Rows from x (rows x cols) to slots of out, z (out_rows rows) to rows of y,
// or the gradient of that: in is x, z or dy, out is out, y or dz.
struct ExpertsMoveArgs {
    const void *in, *z, *residual;
    const int32_t *slot, *offsets, *counts;
    const float *weights;
    void *out;
    float *dweights;
    uint64_t in_stride, z_stride, residual_stride, out_stride;
    uint32_t top, experts;
    uint32_t places;            // rows that slots name: of out, z and dz
    uint32_t rows, cols;
};

// Most alternatives a call ranks: one per lane of a wave.
constexpr uint32_t kTopMax = 64;

// Most kept entries of a row: the distillation's gradient holds a row's in LDS.
constexpr uint32_t kMaxKept = 1024;

// Most experts of a sorting (the waves' counters lie in LDS), most of a token,
// and the largest multiple that an expert's first row is put at.
constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxChoices = 64;
constexpr uint32_t kMaxAlign = 1024;

// Workspace bytes: a function of the sizes alone.
size_t norm_grad_workspace(uint64_t rows, uint64_t cols);
size_t logprobs_workspace(uint64_t rows, uint64_t cols, uint64_t top);
size_t distill_workspace(uint64_t rows, uint64_t cols);

size_t layernorm_grad_workspace(uint64_t rows, uint64_t cols);
size_t policy_loss_workspace(uint64_t rows, uint64_t cols);
size_t experts_sort_workspace(uint64_t entries, uint64_t experts);

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
hipError_t launch_layernorm(RowType t, const LayerNormArgs &a, hipStream_t s, const char **path);
hipError_t launch_layernorm_grad(RowType t, const LayerNormGradArgs &a, hipStream_t s,
                                 const char **path);
hipError_t launch_policy_loss(RowType t, const PolicyLossArgs &a, hipStream_t s,
                              const char **path);
hipError_t launch_policy_grad(RowType t, const PolicyGradArgs &a, hipStream_t s,
                              const char **path);
hipError_t launch_experts_sort(RowType t, const ExpertsSortArgs &a, hipStream_t s,
                               const char **path);
hipError_t launch_experts_gather(RowType t, const ExpertsMoveArgs &a, hipStream_t s,
                                 const char **path);
hipError_t launch_experts_combine(RowType t, const ExpertsMoveArgs &a, hipStream_t s,
                                  const char **path);
hipError_t launch_experts_combine_grad(RowType t, const ExpertsMoveArgs &a, hipStream_t s,
                                       const char **path);

}  // namespace ew
