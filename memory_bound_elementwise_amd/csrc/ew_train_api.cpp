// ew_train_api.cpp -- host side of the layer norm, the policy loss and the
// movement of tokens to their experts: argument validation and the exported
// entry points (include/ew.h, "Row operators of language models").  Validation
// runs before any HIP call.

#include "ew_rows_check.h"

namespace ew {
namespace {

ew_status_t layernorm(RowType t, const void *x, size_t x_stride, const void *weight,
                      const void *bias, const void *residual, size_t residual_stride, void *y,
                      size_t y_stride, void *total, size_t total_stride, float *mean, float *rstd,
                      size_t rows, size_t cols, float eps, hipStream_t stream)
{
    if (rows == 0 || cols == 0) return EW_OK;
    if (!dims_ok(rows, cols) || !stride_ok(x_stride) || !stride_ok(y_stride) ||
        (residual && !stride_ok(residual_stride)) || (total && !stride_ok(total_stride)))
        return EW_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.0f || (total && !residual)) return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const Span ins[] = {matrix(x, es, x_stride, rows, cols),
                        matrix(residual, es, residual_stride, rows, cols, false),
                        array(weight, es, cols, false), array(bias, es, cols, false)};
    const Span outs[] = {matrix(y, es, y_stride, rows, cols),
                         matrix(total, es, total_stride, rows, cols, false),
                         array(mean, 4, rows, false), array(rstd, 4, rows, false)};
    // y may be x or residual, total too; y and total meeting is caught as two outputs
    const unsigned alias[] = {3u, 3u, 0u, 0u};
    const ew_status_t st = check(ins, 4, outs, 4, alias);
    if (st != EW_OK) return st;
    LayerNormArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.total = total;
    a.mean = mean;
    a.rstd = rstd;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.y_stride = y_stride;
    a.total_stride = total_stride;
    a.by_cols = 1.0 / (double)cols;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.eps = eps;
    return launch("layernorm", t, a, stream, launch_layernorm);
}

ew_status_t layernorm_grad(RowType t, const void *dy, size_t dy_stride, const void *x,
                           size_t x_stride, const void *weight, const float *mean,
                           const float *rstd, const void *dtotal, size_t dtotal_stride, void *dx,
                           size_t dx_stride, float *dweight, float *dbias, void *workspace,
                           size_t workspace_bytes, size_t rows, size_t cols, hipStream_t stream)
{
    const bool sums = dweight || dbias;
    if (cols == 0 || (rows == 0 && !sums)) return EW_OK;
    if (!dims_ok(rows, cols) || !stride_ok(dy_stride) || !stride_ok(x_stride) ||
        !stride_ok(dx_stride) || (dtotal && !stride_ok(dtotal_stride)))
        return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const size_t need = sums ? layernorm_grad_workspace(rows, cols) : 0;
    if (workspace_bytes < need) return EW_ERR_INVALID_ARG;
    const Span ins[] = {matrix(dy, es, dy_stride, rows, cols),
                        matrix(x, es, x_stride, rows, cols),
                        matrix(dtotal, es, dtotal_stride, rows, cols, false),
                        array(weight, es, rows ? cols : 0, false), array(mean, 4, rows),
                        array(rstd, 4, rows)};
    Span ws = array(workspace, 1, need);
    ws.align = 16;
    const Span outs[] = {matrix(dx, es, dx_stride, rows, cols), array(dweight, 4, cols, false),
                         array(dbias, 4, cols, false), ws};
    const unsigned alias[] = {7u, 0u, 0u, 0u};
    const ew_status_t st = check(ins, 6, outs, 4, alias);
    if (st != EW_OK) return st;
    LayerNormGradArgs a{};
    a.dy = dy;
    a.x = x;
    a.weight = weight;
    a.dtotal = dtotal;
    a.mean = mean;
    a.rstd = rstd;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.workspace = workspace;
    a.dy_stride = dy_stride;
    a.x_stride = x_stride;
    a.dtotal_stride = dtotal_stride;
    a.dx_stride = dx_stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    return launch("layernorm_grad", t, a, stream, launch_layernorm_grad);
}

// The matrices that a policy loss and its gradient read, and what they make of
// them.
constexpr int kPolicySpans = 5;
struct PolicyInputs {
    Span spans[kPolicySpans];
    PolicyTokens tokens;
};

// Fills in *p; whether the sizes, strides and numbers are valid.
bool policy_inputs(const float *logp, size_t logp_stride, const float *old_logp, size_t old_stride,
                   const float *ref_logp, size_t ref_stride, const float *advantage,
                   size_t advantage_stride, const uint8_t *mask, size_t mask_stride,
                   float clip_low, float clip_high, float kl, size_t rows, size_t cols,
                   PolicyInputs *p)
{
    if (!dims_ok(rows, cols) || !stride_ok(logp_stride) || !stride_ok(old_stride) ||
        (ref_logp && !stride_ok(ref_stride)) || !stride_ok(advantage_stride) ||
        (mask && !stride_ok(mask_stride)))
        return false;
    // a NaN fails each comparison
    if (!(clip_low >= 0.0f) || !(clip_high >= 0.0f) || !(kl >= 0.0f) || std::isinf(kl)) return false;
    p->spans[0] = matrix(logp, 4, logp_stride, rows, cols);
    p->spans[1] = matrix(old_logp, 4, old_stride, rows, cols);
    p->spans[2] = matrix(ref_logp, 4, ref_stride, rows, cols, false);
    p->spans[3] = advantage_stride ? matrix(advantage, 4, advantage_stride, rows, cols)
                                   : array(advantage, 4, cols ? rows : 0);
    p->spans[4] = matrix(mask, 1, mask_stride, rows, cols, false);
    PolicyTokens &t = p->tokens;
    t.logp = logp;
    t.old = old_logp;
    t.ref = ref_logp;
    t.advantage = advantage;
    t.mask = mask;
    t.logp_stride = logp_stride;
    t.old_stride = old_stride;
    t.ref_stride = ref_stride;
    t.mask_stride = mask_stride;
    t.advantage_stride = advantage_stride;
    t.above = std::log1p((double)clip_high);
    t.below = clip_low < 1.0f ? std::log1p(-(double)clip_low) : -(double)INFINITY;
    t.most = (float)(1.0 + (double)clip_high);
    t.least = (float)(1.0 - (double)clip_low);
    t.kl = kl;
    return true;
}

// Sizes of a movement of rows; offsets and counts come together.
bool move_ok(size_t rows, size_t cols, size_t places, size_t top, const int32_t *offsets,
             const int32_t *counts, size_t experts)
{
    if (!dims_ok(rows, cols) || places >= kMaxDim || top == 0 || top > kMaxChoices ||
        rows * top >= kMaxDim)
        return false;
    if (!offsets != !counts) return false;
    return !offsets || (experts != 0 && experts <= kMaxExperts);
}

ew_status_t experts_gather(RowType t, const void *x, size_t x_stride, const int32_t *slot,
                           size_t top, const int32_t *offsets, const int32_t *counts,
                           size_t experts, void *out, size_t out_stride, size_t out_rows,
                           size_t rows, size_t cols, hipStream_t stream)
{
    if (rows == 0 || cols == 0 || out_rows == 0) return EW_OK;
    if (!move_ok(rows, cols, out_rows, top, offsets, counts, experts) || !stride_ok(x_stride) ||
        !stride_ok(out_stride))
        return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const Span ins[] = {matrix(x, es, x_stride, rows, cols), array(slot, 4, rows * top),
                        array(offsets, 4, experts + 1, false), array(counts, 4, experts, false)};
    const Span outs[] = {matrix(out, es, out_stride, out_rows, cols)};
    const unsigned alias[] = {0u};
    const ew_status_t st = check(ins, 4, outs, 1, alias);
    if (st != EW_OK) return st;
    ExpertsMoveArgs a{};
    a.in = x;
    a.slot = slot;
    a.offsets = offsets;
    a.counts = counts;
    a.out = out;
    a.in_stride = x_stride;
    a.out_stride = out_stride;
    a.top = (uint32_t)top;
    a.experts = offsets ? (uint32_t)experts : 0;
    a.places = (uint32_t)out_rows;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    return launch("experts_gather", t, a, stream, launch_experts_gather);
}

ew_status_t experts_combine(RowType t, const void *z, size_t z_stride, size_t z_rows,
                            const int32_t *slot, size_t top, const float *weights,
                            const void *residual, size_t residual_stride, void *y,
                            size_t y_stride, size_t rows, size_t cols, hipStream_t stream)
{
    if (rows == 0 || cols == 0) return EW_OK;
    if (!move_ok(rows, cols, z_rows, top, nullptr, nullptr, 0) || !stride_ok(z_stride) ||
        (residual && !stride_ok(residual_stride)) || !stride_ok(y_stride))
        return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const Span ins[] = {matrix(residual, es, residual_stride, rows, cols, false),
                        matrix(z, es, z_stride, z_rows, cols), array(slot, 4, rows * top),
                        array(weights, 4, rows * top, false)};
    const Span outs[] = {matrix(y, es, y_stride, rows, cols)};
    const unsigned alias[] = {1u};
    const ew_status_t st = check(ins, 4, outs, 1, alias);
    if (st != EW_OK) return st;
    ExpertsMoveArgs a{};
    a.z = z;
    a.residual = residual;
    a.slot = slot;
    a.weights = weights;
    a.out = y;
    a.z_stride = z_stride;
    a.residual_stride = residual_stride;
    a.out_stride = y_stride;
    a.top = (uint32_t)top;
    a.places = (uint32_t)z_rows;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    return launch("experts_combine", t, a, stream, launch_experts_combine);
}

ew_status_t experts_combine_grad(RowType t, const void *dy, size_t dy_stride, const void *z,
                                 size_t z_stride, size_t z_rows, const int32_t *slot, size_t top,
                                 const float *weights, const int32_t *offsets,
                                 const int32_t *counts, size_t experts, void *dz,
                                 size_t dz_stride, float *dweights, size_t rows, size_t cols,
                                 hipStream_t stream)
{
    if (rows == 0) return EW_OK;
    if (!move_ok(rows, cols, z_rows, top, offsets, counts, experts) || !stride_ok(dy_stride) ||
        !stride_ok(z_stride) || !stride_ok(dz_stride))
        return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const Span ins[] = {matrix(z, es, z_stride, z_rows, cols), matrix(dy, es, dy_stride, rows, cols),
                        array(slot, 4, rows * top), array(weights, 4, rows * top),
                        array(offsets, 4, experts + 1, false), array(counts, 4, experts, false)};
    const Span outs[] = {matrix(dz, es, dz_stride, z_rows, cols), array(dweights, 4, rows * top)};
    const unsigned alias[] = {1u, 0u};
    const ew_status_t st = check(ins, 6, outs, 2, alias);
    if (st != EW_OK) return st;
    ExpertsMoveArgs a{};
    a.in = dy;
    a.z = z;
    a.slot = slot;
    a.offsets = offsets;
    a.counts = counts;
    a.weights = weights;
    a.out = dz;
    a.dweights = dweights;
    a.in_stride = dy_stride;
    a.z_stride = z_stride;
    a.out_stride = dz_stride;
    a.top = (uint32_t)top;
    a.experts = offsets ? (uint32_t)experts : 0;
    a.places = (uint32_t)z_rows;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    return launch("experts_combine_grad", t, a, stream, launch_experts_combine_grad);
}

}  // namespace
}  // namespace ew

using namespace ew;

extern "C" {

// The entry points of one element type: E the C type, X its suffix, T its
// RowType.
#define EW_TRAIN_ENTRY_POINTS(E, X, T)                                                            \
    ew_status_t ew_layernorm_##X(const E *x, size_t x_stride, const E *weight, const E *bias,     \
                                 const E *residual, size_t residual_stride, E *y,                 \
                                 size_t y_stride, E *total, size_t total_stride, float *mean,     \
                                 float *rstd, size_t rows, size_t cols, float eps,                \
                                 hipStream_t stream)                                              \
    {                                                                                             \
        return layernorm(T, x, x_stride, weight, bias, residual, residual_stride, y, y_stride,    \
                         total, total_stride, mean, rstd, rows, cols, eps, stream);               \
    }                                                                                             \
    ew_status_t ew_layernorm_grad_##X(const E *dy, size_t dy_stride, const E *x,                  \
                                      size_t x_stride, const E *weight, const float *mean,        \
                                      const float *rstd, const E *dtotal,                         \
                                      size_t dtotal_stride, E *dx, size_t dx_stride,              \
                                      float *dweight, float *dbias, void *workspace,              \
                                      size_t workspace_bytes, size_t rows, size_t cols,           \
                                      hipStream_t stream)                                         \
    {                                                                                             \
        return layernorm_grad(T, dy, dy_stride, x, x_stride, weight, mean, rstd, dtotal,          \
                              dtotal_stride, dx, dx_stride, dweight, dbias, workspace,            \
                              workspace_bytes, rows, cols, stream);                               \
    }                                                                                             \
    ew_status_t ew_experts_gather_##X(const E *x, size_t x_stride, const int32_t *slot,           \
                                      size_t top, const int32_t *offsets,                         \
                                      const int32_t *counts, size_t experts, E *out,              \
                                      size_t out_stride, size_t out_rows, size_t rows,            \
                                      size_t cols, hipStream_t stream)                            \
    {                                                                                             \
        return experts_gather(T, x, x_stride, slot, top, offsets, counts, experts, out,           \
                              out_stride, out_rows, rows, cols, stream);                          \
    }                                                                                             \
    ew_status_t ew_experts_combine_##X(const E *z, size_t z_stride, size_t z_rows,                \
                                       const int32_t *slot, size_t top, const float *weights,     \
                                       const E *residual, size_t residual_stride, E *y,           \
                                       size_t y_stride, size_t rows, size_t cols,                 \
                                       hipStream_t stream)                                        \
    {                                                                                             \
        return experts_combine(T, z, z_stride, z_rows, slot, top, weights, residual,              \
                               residual_stride, y, y_stride, rows, cols, stream);                 \
    }                                                                                             \
    ew_status_t ew_experts_combine_grad_##X(const E *dy, size_t dy_stride, const E *z,            \
                                            size_t z_stride, size_t z_rows,                       \
                                            const int32_t *slot, size_t top,                      \
                                            const float *weights, const int32_t *offsets,         \
                                            const int32_t *counts, size_t experts, E *dz,         \
                                            size_t dz_stride, float *dweights, size_t rows,       \
                                            size_t cols, hipStream_t stream)                      \
    {                                                                                             \
        return experts_combine_grad(T, dy, dy_stride, z, z_stride, z_rows, slot, top, weights,    \
                                    offsets, counts, experts, dz, dz_stride, dweights, rows,      \
                                    cols, stream);                                                \
    }

EW_TRAIN_ENTRY_POINTS(float, f32, kRowF32)
EW_TRAIN_ENTRY_POINTS(uint16_t, f16, kRowF16)
EW_TRAIN_ENTRY_POINTS(uint16_t, bf16, kRowBF16)
#undef EW_TRAIN_ENTRY_POINTS

// Sizes no call accepts need no workspace.
size_t ew_layernorm_grad_workspace(size_t rows, size_t cols)
{
    return dims_ok(rows, cols) ? layernorm_grad_workspace(rows, cols) : 0;
}

size_t ew_policy_loss_workspace(size_t rows, size_t cols)
{
    return dims_ok(rows, cols) ? policy_loss_workspace(rows, cols) : 0;
}

ew_status_t ew_policy_loss_f32(const float *logp, size_t logp_stride, const float *old_logp,
                               size_t old_stride, const float *ref_logp, size_t ref_stride,
                               const float *advantage, size_t advantage_stride,
                               const uint8_t *mask, size_t mask_stride, float *loss, float *stats,
                               float *weights, float clip_low, float clip_high, float kl,
                               float scale, int mean, void *workspace, size_t workspace_bytes,
                               size_t rows, size_t cols, hipStream_t stream)
{
    PolicyInputs p{};
    if (!policy_inputs(logp, logp_stride, old_logp, old_stride, ref_logp, ref_stride, advantage,
                       advantage_stride, mask, mask_stride, clip_low, clip_high, kl, rows, cols,
                       &p))
        return EW_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || mean < EW_MEAN_TOKENS || mean > EW_MEAN_NONE)
        return EW_ERR_INVALID_ARG;
    const size_t need = policy_loss_workspace(rows, cols);
    if (workspace_bytes < need) return EW_ERR_INVALID_ARG;
    Span ws = array(workspace, 1, need);
    ws.align = 16;
    const Span outs[] = {array(loss, 4, 1), array(stats, 4, 4, false),
                         array(weights, 4, rows, false), ws};
    const unsigned alias[4] = {};
    const ew_status_t st = check(p.spans, kPolicySpans, outs, 4, alias);
    if (st != EW_OK) return st;
    PolicyLossArgs a{};
    a.in = p.tokens;
    a.loss = loss;
    a.stats = stats;
    a.weights = weights;
    a.workspace = workspace;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.scale = scale;
    a.mean = mean;
    return launch("policy_loss", kRowF32, a, stream, launch_policy_loss);
}

ew_status_t ew_policy_loss_grad_f32(const float *logp, size_t logp_stride, const float *old_logp,
                                    size_t old_stride, const float *ref_logp, size_t ref_stride,
                                    const float *advantage, size_t advantage_stride,
                                    const uint8_t *mask, size_t mask_stride,
                                    const float *weights, const float *dloss, float *dlogp,
                                    size_t dlogp_stride, float clip_low, float clip_high,
                                    float kl, size_t rows, size_t cols, hipStream_t stream)
{
    if (rows == 0 || cols == 0) return EW_OK;
    PolicyInputs p{};
    if (!policy_inputs(logp, logp_stride, old_logp, old_stride, ref_logp, ref_stride, advantage,
                       advantage_stride, mask, mask_stride, clip_low, clip_high, kl, rows, cols,
                       &p) ||
        !stride_ok(dlogp_stride))
        return EW_ERR_INVALID_ARG;
    const Span ins[] = {p.spans[0], p.spans[1], p.spans[2], p.spans[3], p.spans[4],
                        array(weights, 4, rows), array(dloss, 4, 1, false)};
    const Span outs[] = {matrix(dlogp, 4, dlogp_stride, rows, cols)};
    // dlogp may be a matrix of a value a token
    const unsigned alias[] = {advantage_stride ? 15u : 7u};
    const ew_status_t st = check(ins, 7, outs, 1, alias);
    if (st != EW_OK) return st;
    PolicyGradArgs a{};
    a.in = p.tokens;
    a.weights = weights;
    a.dloss = dloss;
    a.dlogp = dlogp;
    a.dlogp_stride = dlogp_stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    return launch("policy_loss_grad", kRowF32, a, stream, launch_policy_grad);
}

size_t ew_experts_rows(size_t entries, size_t experts, size_t align)
{
    if (entries >= kMaxDim || experts == 0 || experts > kMaxExperts || align == 0 ||
        align > kMaxAlign)
        return SIZE_MAX;
    const size_t some = entries < experts ? entries : experts;
    const size_t rows = (entries + some * (align - 1) + align - 1) / align * align;
    return rows < kMaxDim ? rows : SIZE_MAX;
}

size_t ew_experts_sort_workspace(size_t entries, size_t experts)
{
    return entries < kMaxDim && experts <= kMaxExperts ? experts_sort_workspace(entries, experts)
                                                       : 0;
}

ew_status_t ew_experts_sort(const int64_t *ids, size_t entries, size_t experts, size_t align,
                            int32_t *slot, int32_t *offsets, int32_t *counts, int32_t *source,
                            void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const size_t rows = ew_experts_rows(entries, experts, align);
    if (rows == SIZE_MAX) return EW_ERR_INVALID_ARG;
    const size_t need = experts_sort_workspace(entries, experts);
    if (workspace_bytes < need) return EW_ERR_INVALID_ARG;
    const Span ins[] = {array(ids, 8, entries)};
    Span ws = array(workspace, 1, need);
    ws.align = 16;
    const Span outs[] = {array(slot, 4, entries), array(offsets, 4, experts + 1),
                         array(counts, 4, experts, false), array(source, 4, rows, false), ws};
    const unsigned alias[5] = {};
    const ew_status_t st = check(ins, 1, outs, 5, alias);
    if (st != EW_OK) return st;
    ExpertsSortArgs a{};
    a.ids = ids;
    a.slot = slot;
    a.offsets = offsets;
    a.counts = counts;
    a.source = source;
    a.workspace = workspace;
    a.align = (uint32_t)align;
    a.source_rows = (uint32_t)rows;
    a.rows = (uint32_t)entries;
    a.cols = (uint32_t)experts;
    return launch("experts_sort", kRowF32, a, stream, launch_experts_sort);
}

}  // extern "C"
