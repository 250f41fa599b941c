// ew_rows_api.cpp -- host side of the row operators: argument validation and
// the exported entry points (include/ew.h, "Row operators of language
// models").  Validation runs before any HIP call.

#include "ew.h"
#include "ew_rows_check.h"

namespace ew {
namespace {

ew_status_t rmsnorm(RowType t, const void *x, size_t x_stride, const void *weight,
                    const void *residual, size_t residual_stride, void *y, size_t y_stride,
                    float *scales, size_t group, bool e4m3, void *total, size_t total_stride,
                    float *rstd, size_t rows, size_t cols, float eps, hipStream_t stream)
{
    if (rows == 0 || cols == 0) return EW_OK;
    if (!dims_ok(rows, cols) || !stride_ok(x_stride) || !stride_ok(y_stride) ||
        (residual && !stride_ok(residual_stride)) || (total && !stride_ok(total_stride)))
        return EW_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.0f || (total && !residual)) return EW_ERR_INVALID_ARG;
    if (e4m3 && group != 0 && group != 16 && group != 32 && group != 64 && group != 128 &&
        group != 256)
        return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const size_t per = group ? group : cols, groups = (cols + per - 1) / per;
    const Span ins[] = {matrix(x, es, x_stride, rows, cols),
                        matrix(residual, es, residual_stride, rows, cols, false),
                        array(weight, es, cols)};
    const Span outs[] = {matrix(y, e4m3 ? 1 : es, y_stride, rows, cols),
                         matrix(total, es, total_stride, rows, cols, false),
                         array(rstd, 4, rows, false),
                         array(scales, 4, e4m3 ? rows * groups : 0, e4m3)};
    // y may be x or residual, total too; y and total meeting is caught as two outputs
    const unsigned alias[] = {e4m3 ? 0u : 3u, 3u, 0u, 0u};
    const ew_status_t st = check(ins, 3, outs, 4, alias);
    if (st != EW_OK) return st;
    NormArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.y = y;
    a.total = total;
    a.rstd = rstd;
    a.scales = e4m3 ? scales : nullptr;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.y_stride = y_stride;
    a.total_stride = total_stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.group = (uint32_t)per;
    a.groups = (uint32_t)groups;
    a.eps = eps;
    return launch(e4m3 ? "rmsnorm_e4m3" : "rmsnorm", t, a, stream, launch_norm);
}

ew_status_t rmsnorm_grad(RowType t, const void *dy, size_t dy_stride, const void *x,
                         size_t x_stride, const void *weight, const float *rstd,
                         const void *dtotal, size_t dtotal_stride, void *dx, size_t dx_stride,
                         float *dweight, void *workspace, size_t workspace_bytes, size_t rows,
                         size_t cols, hipStream_t stream)
{
    if (cols == 0 || (rows == 0 && !dweight)) return EW_OK;
    if (!dims_ok(rows, cols) || !stride_ok(dy_stride) || !stride_ok(x_stride) ||
        !stride_ok(dx_stride) || (dtotal && !stride_ok(dtotal_stride)))
        return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const size_t need = dweight ? norm_grad_workspace(rows, cols) : 0;
    if (workspace_bytes < need) return EW_ERR_INVALID_ARG;
    const Span ins[] = {matrix(dy, es, dy_stride, rows, cols),
                        matrix(x, es, x_stride, rows, cols),
                        matrix(dtotal, es, dtotal_stride, rows, cols, false),
                        array(weight, es, rows ? cols : 0), array(rstd, 4, rows)};
    Span ws = array(workspace, 1, need);
    ws.align = 16;
    const Span outs[] = {matrix(dx, es, dx_stride, rows, cols), array(dweight, 4, cols, false), ws};
    const unsigned alias[] = {7u, 0u, 0u};
    const ew_status_t st = check(ins, 5, outs, 3, alias);
    if (st != EW_OK) return st;
    NormGradArgs a{};
    a.dy = dy;
    a.x = x;
    a.weight = weight;
    a.dtotal = dtotal;
    a.rstd = rstd;
    a.dx = dx;
    a.dweight = dweight;
    a.partial = static_cast<float *>(workspace);
    a.dy_stride = dy_stride;
    a.x_stride = x_stride;
    a.dtotal_stride = dtotal_stride;
    a.dx_stride = dx_stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    return launch("rmsnorm_grad", t, a, stream, launch_norm_grad);
}

ew_status_t logprobs(RowType t, const void *logits, size_t stride, const int64_t *targets,
                     float *logp, float *entropy, float *lse, float *top_logp, int64_t *top_ids,
                     size_t top, float scale, void *workspace, size_t workspace_bytes,
                     size_t rows, size_t cols, hipStream_t stream)
{
    if (rows == 0) return EW_OK;
    if (!dims_ok(rows, cols) || !stride_ok(stride) || !scale_ok(scale)) return EW_ERR_INVALID_ARG;
    if (top > kTopMax || top > cols) return EW_ERR_INVALID_ARG;
    if (!top_logp != !top_ids) return EW_ERR_INVALID_ARG;
    const size_t need = logprobs_workspace(rows, cols, top);
    if (workspace_bytes < need) return EW_ERR_INVALID_ARG;
    const Span ins[] = {matrix(logits, row_elem_size(t), stride, rows, cols),
                        array(targets, 8, rows)};
    Span ws = array(workspace, 1, need);
    ws.align = 16;
    const Span outs[] = {array(logp, 4, rows), array(entropy, 4, rows, false),
                         array(lse, 4, rows, false), array(top_logp, 4, rows * top),
                         array(top_ids, 8, rows * top), ws};
    const unsigned alias[6] = {};
    const ew_status_t st = check(ins, 2, outs, 6, alias);
    if (st != EW_OK) return st;
    LogprobsArgs a{};
    a.logits = logits;
    a.targets = targets;
    a.logp = logp;
    a.entropy = entropy;
    a.lse = lse;
    a.top_logp = top_logp;
    a.top_ids = top_ids;
    a.workspace = workspace;
    a.stride = stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.top = (uint32_t)top;
    a.scale = scale;
    return launch("logprobs", t, a, stream, launch_logprobs);
}

ew_status_t logprobs_grad(RowType t, const void *logits, size_t stride, const int64_t *targets,
                          const float *lse, const float *entropy, const float *dlogp,
                          const float *dentropy, void *dlogits, size_t dlogits_stride,
                          float scale, size_t rows, size_t cols, hipStream_t stream)
{
    if (rows == 0 || cols == 0) return EW_OK;
    if (!dims_ok(rows, cols) || !stride_ok(stride) || !stride_ok(dlogits_stride) ||
        !scale_ok(scale))
        return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const Span ins[] = {matrix(logits, es, stride, rows, cols), array(targets, 8, rows),
                        array(lse, 4, rows), array(dlogp, 4, rows),
                        array(dentropy, 4, rows, false),
                        array(entropy, 4, rows, dentropy != nullptr)};
    const Span outs[] = {matrix(dlogits, es, dlogits_stride, rows, cols)};
    const unsigned alias[] = {1u};
    const ew_status_t st = check(ins, 6, outs, 1, alias);
    if (st != EW_OK) return st;
    LogprobsGradArgs a{};
    a.logits = logits;
    a.targets = targets;
    a.lse = lse;
    a.entropy = entropy;
    a.dlogp = dlogp;
    a.dentropy = dentropy;
    a.dlogits = dlogits;
    a.stride = stride;
    a.dlogits_stride = dlogits_stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.scale = scale;
    return launch("logprobs_grad", t, a, stream, launch_logprobs_grad);
}

ew_status_t distill(RowType t, const void *logits, size_t stride, const float *teacher,
                    const int64_t *ids, size_t kept, float *loss, float *lse, float scale,
                    void *workspace, size_t workspace_bytes, size_t rows, size_t cols,
                    hipStream_t stream)
{
    if (rows == 0) return EW_OK;
    if (!dims_ok(rows, cols) || !stride_ok(stride) || !scale_ok(scale) || kept > kMaxKept)
        return EW_ERR_INVALID_ARG;
    const size_t need = distill_workspace(rows, cols);
    if (workspace_bytes < need) return EW_ERR_INVALID_ARG;
    const Span ins[] = {matrix(logits, row_elem_size(t), stride, rows, cols),
                        array(teacher, 4, rows * kept), array(ids, 8, rows * kept)};
    Span ws = array(workspace, 1, need);
    ws.align = 16;
    const Span outs[] = {array(loss, 4, rows), array(lse, 4, rows, false), ws};
    const unsigned alias[3] = {};
    const ew_status_t st = check(ins, 3, outs, 3, alias);
    if (st != EW_OK) return st;
    DistillArgs a{};
    a.logits = logits;
    a.teacher = teacher;
    a.ids = ids;
    a.loss = loss;
    a.lse = lse;
    a.workspace = workspace;
    a.stride = stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.kept = (uint32_t)kept;
    a.scale = scale;
    a.by = teacher_scale(scale);
    return launch("distill", t, a, stream, launch_distill);
}

ew_status_t distill_grad(RowType t, const void *logits, size_t stride, const float *teacher,
                         const int64_t *ids, size_t kept, const float *lse, const float *dloss,
                         void *dlogits, size_t dlogits_stride, float scale, size_t rows,
                         size_t cols, hipStream_t stream)
{
    if (rows == 0 || cols == 0) return EW_OK;
    if (!dims_ok(rows, cols) || !stride_ok(stride) || !stride_ok(dlogits_stride) ||
        !scale_ok(scale) || kept > kMaxKept)
        return EW_ERR_INVALID_ARG;
    const int es = row_elem_size(t);
    const Span ins[] = {matrix(logits, es, stride, rows, cols), array(teacher, 4, rows * kept),
                        array(ids, 8, rows * kept), array(lse, 4, rows), array(dloss, 4, rows)};
    const Span outs[] = {matrix(dlogits, es, dlogits_stride, rows, cols)};
    const unsigned alias[] = {1u};
    const ew_status_t st = check(ins, 5, outs, 1, alias);
    if (st != EW_OK) return st;
    DistillGradArgs a{};
    a.logits = logits;
    a.teacher = teacher;
    a.ids = ids;
    a.lse = lse;
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.stride = stride;
    a.dlogits_stride = dlogits_stride;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.kept = (uint32_t)kept;
    a.scale = scale;
    a.by = teacher_scale(scale);
    return launch("distill_grad", t, a, stream, launch_distill_grad);
}

}  // namespace
}  // namespace ew

using namespace ew;

extern "C" {

// The entry points of one element type: E the C type, X its suffix, T its
// RowType.
#define EW_ROW_ENTRY_POINTS(E, X, T)                                                             \
    ew_status_t ew_rmsnorm_##X(const E *x, size_t x_stride, const E *weight, const E *residual,  \
                               size_t residual_stride, E *y, size_t y_stride, E *total,          \
                               size_t total_stride, float *rstd, size_t rows, size_t cols,       \
                               float eps, hipStream_t stream)                                    \
    {                                                                                            \
        return rmsnorm(T, x, x_stride, weight, residual, residual_stride, y, y_stride, nullptr,  \
                       0, false, total, total_stride, rstd, rows, cols, eps, stream);            \
    }                                                                                            \
    ew_status_t ew_rmsnorm_e4m3_##X(const E *x, size_t x_stride, const E *weight,                \
                                    const E *residual, size_t residual_stride, uint8_t *q,       \
                                    size_t q_stride, float *scales, size_t group, E *total,      \
                                    size_t total_stride, float *rstd, size_t rows, size_t cols,  \
                                    float eps, hipStream_t stream)                               \
    {                                                                                            \
        return rmsnorm(T, x, x_stride, weight, residual, residual_stride, q, q_stride, scales,   \
                       group, true, total, total_stride, rstd, rows, cols, eps, stream);         \
    }                                                                                            \
    ew_status_t ew_rmsnorm_grad_##X(const E *dy, size_t dy_stride, const E *x, size_t x_stride,  \
                                    const E *weight, const float *rstd, const E *dtotal,         \
                                    size_t dtotal_stride, E *dx, size_t dx_stride,               \
                                    float *dweight, void *workspace, size_t workspace_bytes,     \
                                    size_t rows, size_t cols, hipStream_t stream)                \
    {                                                                                            \
        return rmsnorm_grad(T, dy, dy_stride, x, x_stride, weight, rstd, dtotal, dtotal_stride,  \
                            dx, dx_stride, dweight, workspace, workspace_bytes, rows, cols,      \
                            stream);                                                             \
    }                                                                                            \
    ew_status_t ew_logprobs_##X(const E *logits, size_t stride, const int64_t *targets,          \
                                float *logp, float *entropy, float *lse, float *top_logp,        \
                                int64_t *top_ids, size_t top, float scale, void *workspace,      \
                                size_t workspace_bytes, size_t rows, size_t cols,                \
                                hipStream_t stream)                                              \
    {                                                                                            \
        return logprobs(T, logits, stride, targets, logp, entropy, lse, top_logp, top_ids, top,  \
                        scale, workspace, workspace_bytes, rows, cols, stream);                  \
    }                                                                                            \
    ew_status_t ew_logprobs_grad_##X(const E *logits, size_t stride, const int64_t *targets,     \
                                     const float *lse, const float *entropy, const float *dlogp, \
                                     const float *dentropy, E *dlogits, size_t dlogits_stride,   \
                                     float scale, size_t rows, size_t cols, hipStream_t stream)  \
    {                                                                                            \
        return logprobs_grad(T, logits, stride, targets, lse, entropy, dlogp, dentropy, dlogits, \
                             dlogits_stride, scale, rows, cols, stream);                         \
    }                                                                                            \
    ew_status_t ew_distill_##X(const E *logits, size_t stride, const float *teacher,             \
                               const int64_t *ids, size_t kept, float *loss, float *lse,         \
                               float scale, void *workspace, size_t workspace_bytes,             \
                               size_t rows, size_t cols, hipStream_t stream)                     \
    {                                                                                            \
        return distill(T, logits, stride, teacher, ids, kept, loss, lse, scale, workspace,       \
                       workspace_bytes, rows, cols, stream);                                     \
    }                                                                                            \
    ew_status_t ew_distill_grad_##X(const E *logits, size_t stride, const float *teacher,        \
                                    const int64_t *ids, size_t kept, const float *lse,           \
                                    const float *dloss, E *dlogits, size_t dlogits_stride,       \
                                    float scale, size_t rows, size_t cols, hipStream_t stream)   \
    {                                                                                            \
        return distill_grad(T, logits, stride, teacher, ids, kept, lse, dloss, dlogits,          \
                            dlogits_stride, scale, rows, cols, stream);                          \
    }

EW_ROW_ENTRY_POINTS(float, f32, kRowF32)
EW_ROW_ENTRY_POINTS(uint16_t, f16, kRowF16)
EW_ROW_ENTRY_POINTS(uint16_t, bf16, kRowBF16)
#undef EW_ROW_ENTRY_POINTS

// Sizes no call accepts need no workspace.
size_t ew_rmsnorm_grad_workspace(size_t rows, size_t cols)
{
    return dims_ok(rows, cols) ? norm_grad_workspace(rows, cols) : 0;
}

size_t ew_logprobs_workspace(size_t rows, size_t cols, size_t top)
{
    return dims_ok(rows, cols) && top <= kTopMax ? logprobs_workspace(rows, cols, top) : 0;
}

size_t ew_distill_workspace(size_t rows, size_t cols)
{
    return dims_ok(rows, cols) ? distill_workspace(rows, cols) : 0;
}

}  // extern "C"
