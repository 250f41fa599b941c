/*
 * ew.h -- C ABI of libew, streaming elementwise kernels for AMD Instinct
 * MI355X (gfx950).
 *
 * Plain C: no C++ or torch types.  Every operation takes device pointers, an
 * element count n and a HIP stream, validates its arguments on the host,
 * launches one kernel asynchronously on that stream (ew_batch: one per
 * EW_BATCH_MAX items; ew_batch_run: one for any number; the row operators:
 * up to three) and returns a status.
 *
 * Pages cited (by title and section):
 *   [HyperAI]   HyperAI article on optimising the Elementwise operator
 *               (hyper.ai/ko/news/49090)
 *   [EwOps]     "逐元素操作算子 / Element-wise 算子优化" (517adam.github.io)
 *   [Puzzle31]  Mojo GPU Puzzles, "Puzzle 31: occupancy optimisation"
 *               (puzzles.modular.com)
 *   [PerfNotes] GPU-performance lecture notes (cyqw.cn/news/898472)
 *   [GEMM-9.3]  "9.3 project: GEMM optimisation step by step" (amittech.dev)
 *
 * Conventions shared by every operation
 * -------------------------------------
 * Memory      The caller owns every buffer (device memory, e.g. allocated by
 *             torch).  The library never allocates or frees device memory
 *             and keeps no pointer after the call returns (ew_batch and
 *             ew_batch_build alone take transient host memory for their
 *             overlap check).
 * Layout      One-dimensional, contiguous, n elements (the row operators'
 *             matrices: see their section).  Pointers need only
 *             element alignment (4 bytes for fp32, 2 bytes for 16-bit data);
 *             16-byte alignment is NOT required: the library peels a scalar
 *             head so that the output's body is 16-byte aligned, streams the
 *             body with 16-byte vector accesses, and finishes a scalar tail.
 * Streams     Asynchronous on `stream` (0 = the null stream).  The library
 *             never synchronises.  A kernel fault surfaces at the caller's
 *             next synchronisation, not here.
 * n == 0      Returns EW_OK without launching anything (pointers unchecked).
 * Aliasing    An output may be exactly the same pointer as an input where the
 *             operation says so; any other overlap between an output range
 *             and an input range returns EW_ERR_OVERLAP.
 * Errors      Checked in this order, before any HIP call: null pointer or an
 *             invalid size/stride (EW_ERR_INVALID_ARG), element misalignment
 *             (EW_ERR_MISALIGNED), overlap (EW_ERR_OVERLAP).  Then: no HIP
 *             device (EW_ERR_NO_DEVICE), a failed launch (EW_ERR_HIP; the
 *             hipError_t is kept for ew_last_hip_error()).  Nothing aborts.
 * Logging     With the environment variable EW_LOG set (to anything but ""
 *             or "0") every launch prints its plan -- op, n, head, vectors,
 *             tail, grid, block, unroll and the kernel path -- as one line on
 *             stderr.  Read once per process.
 * Numerics    IEEE-754 round-to-nearest-even, subnormals preserved (no
 *             flush-to-zero).  NaN results are NaN; their payload is not part
 *             of the contract for arithmetic operations.  Copy and gather
 *             move bit patterns unchanged.
 * Threads     All functions are thread-safe.
 */
#ifndef EW_H_
#define EW_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The HIP runtime declares hipStream_t the same way; repeating an identical
 * typedef is valid C11 and C++. */
typedef struct ihipStream_t *hipStream_t;

typedef enum ew_status {
    EW_OK = 0,
    EW_ERR_INVALID_ARG = -1, /* null pointer, size overflow, zero stride, unknown op name */
    EW_ERR_MISALIGNED = -2,  /* pointer not aligned to its element size */
    EW_ERR_OVERLAP = -3,     /* output partially overlaps an input */
    EW_ERR_NO_DEVICE = -4,   /* no HIP device is usable */
    EW_ERR_HIP = -5,         /* a HIP runtime call failed; see ew_last_hip_error() */
    EW_ERR_TOO_LARGE = -6    /* a batch table larger than EW_BATCH_SCRATCH_BYTES */
} ew_status_t;

/* ------------------------------------------------------------------------ */
/* Operations                                                                */
/* ------------------------------------------------------------------------ */

/* c[i] = a[i] + b[i] in binary32, i < n.
 * [HyperAI] "Version 1: FP32 baseline" and "Version 2: FP32x4 vectorisation";
 * [EwOps] section 二, template code and optimisation points 2-3 (grid-stride
 * loop, float4 body with a scalar tail).
 * a, b: inputs (device, 4-byte aligned).  c: output (device, 4-byte aligned);
 * c may equal a or b exactly. */
ew_status_t ew_add_f32(const float *a, const float *b, float *c, size_t n,
                       hipStream_t stream);

/* c[i] = rne16(widen(a[i]) + widen(b[i])) on binary16 data passed as raw
 * uint16_t bit patterns: each pair is widened exactly to binary32, added
 * once, and the sum rounded to binary16, nearest-even.  This equals the
 * correctly rounded binary16 sum.
 * [HyperAI] "Version 3: FP16 baseline" (half add per element) and
 * "Version 6: FP16x8 pack" (eight halves per 128-bit access).
 * Pointers 2-byte aligned; c may equal a or b exactly. */
ew_status_t ew_add_f16(const uint16_t *a, const uint16_t *b, uint16_t *c,
                       size_t n, hipStream_t stream);

/* The same as ew_add_f16 for bfloat16 bit patterns: widen, add in binary32,
 * round to bfloat16 nearest-even.  (The pages treat binary16; bfloat16 takes
 * the same rule.)  Pointers 2-byte aligned; c may equal a or b exactly. */
ew_status_t ew_add_bf16(const uint16_t *a, const uint16_t *b, uint16_t *c,
                        size_t n, hipStream_t stream);

/* In place: y[i] = fma(alpha, x[i], y[i]), one rounding per element.
 * [Puzzle31] overview: single-precision alpha times x plus y.
 * x: input, y: input and output (both 4-byte aligned); x may equal y
 * exactly. */
ew_status_t ew_saxpy_f32(float alpha, const float *x, float *y, size_t n,
                         hipStream_t stream);

/* y[i] = maximum(x[i], +0) in the IEEE 754-2019 sense: x > 0 gives x, a NaN
 * gives a NaN, everything else (negative, -0, -inf) gives +0.
 * [PerfNotes] section 5.2, ReLU as a memory-bound example.
 * x: input, y: output (4-byte aligned); y may equal x exactly. */
ew_status_t ew_relu_f32(const float *x, float *y, size_t n, hipStream_t stream);

/* x[i] = maximum(x[i], +0) in place, with the result of ew_relu_f32, but
 * storing only what changes: an element that is already >= 0 (or a NaN)
 * costs a read and no write ([PerfNotes] section 5.2, the ReLU intensity
 * example, its second case).  Stores are decided per aligned 64-byte span:
 * a span holding at least one element to clear is written whole, any other
 * span is left untouched (a partial span is never written: on MI355X that
 * costs more than writing it whole).  The body is aligned to 64 bytes by a
 * scalar head of up to 15 elements.  x: 4-byte aligned.  Errors as for
 * ew_relu_f32.  On data whose every element is already >= 0 it moves half
 * the bytes of ew_relu_f32(x, x).  When to prefer ew_relu_f32(x, x): data
 * with mixed signs.  On normal(0, 1) data almost every 64-byte span holds a
 * negative element, so nearly every span is written and the call moves the
 * same bytes as ew_relu_f32(x, x) (measured on MI355X: 1.33 x the bytes it
 * must move, and a few per cent slower than ew_relu_f32(x, x)). */
ew_status_t ew_relu_inplace_f32(float *x, size_t n, hipStream_t stream);

/* out[i] = in[i], bit patterns unchanged (NaN payloads included).
 * [PerfNotes] section 3.2, the coalesced copy kernel.
 * out == in is allowed and launches nothing. */
ew_status_t ew_copy_f32(const float *in, float *out, size_t n,
                        hipStream_t stream);

/* out[i] = in[(stride * i) mod n], bit patterns unchanged; the index product
 * is reduced exactly for every stride (no 32- or 64-bit wrap-around).
 * [PerfNotes] section 3.2, the non-coalesced copy kernel reads in[idx*2 % n].
 * Reads are strided; writes are contiguous.  stride 0 -> EW_ERR_INVALID_ARG.
 * in and out must not overlap at all. */
ew_status_t ew_gather_f32(const float *in, float *out, size_t n, size_t stride,
                          hipStream_t stream);

/* The same result as ew_gather_f32 -- out[i] = in[(stride * i) mod n], bits
 * unchanged -- computed the way the non-coalesced copy kernel of [PerfNotes]
 * section 3.2 computes it: every output element loads its own input element
 * (4-byte loads, index stepped per lane), whatever the stride, with none of
 * ew_gather_f32's reuse (no replicated segments, no pass decomposition, no
 * tiled transposition, no contiguous-span path).  For stride 2 on even n it reads the input twice
 * (outputs i and i + n/2 read the same element).  It is the baseline against
 * which the cost of strided reads is measured ([PerfNotes] 3.3).  Arguments,
 * errors and launch rows ("gather_walk_f32") as for ew_gather_f32; stride 1
 * also walks (no redirection to the copy). */
ew_status_t ew_gather_walk_f32(const float *in, float *out, size_t n, size_t stride,
                               hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Strided views                                                            */
/* ------------------------------------------------------------------------ */

/* A strided 2-D view copied to a contiguous row-major array, bit patterns
 * unchanged: out[r*cols + c] = in[r*stride_r + c*stride_c] for r < rows,
 * c < cols.  Strides are in elements and signed (zero and negative strides
 * are allowed); `in` points at element (0, 0) of the view.  A 1-D strided
 * view (PyTorch x[::s]) is rows = 1, stride_c = s; a submatrix has
 * stride_c = 1; a transposed view has stride_r = 1.
 * [PerfNotes] 3.4 (non-contiguous tensors show up as strides) and 3.1-3.2
 * (coalesced versus strided reads).
 * Paths: rows == 1 with stride_c == 2 reads contiguous 16-byte spans and
 * keeps the even elements; rows == 1 with 3 <= stride_c <= 32 reads the
 * view's span contiguously (staged through LDS) and keeps one element in
 * stride_c; stride_c == 1 reads whole 16-byte row segments;
 * stride_r == 1 moves 128 x 128 tiles through LDS so that both reads and
 * writes are coalesced; otherwise one 4-byte load per element.  out is written with 16-byte
 * stores after a scalar head.
 * Errors: rows or cols 0 -> EW_OK; null pointers, rows*cols overflow, or a
 * view reaching outside the address space -> EW_ERR_INVALID_ARG; in or out
 * not 4-byte aligned -> EW_ERR_MISALIGNED; any overlap between out and the
 * span of elements the view touches -> EW_ERR_OVERLAP. */
ew_status_t ew_copy2d_f32(const float *in, int64_t stride_r, int64_t stride_c,
                          float *out, size_t rows, size_t cols, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* SAXPY and ReLU on 16-bit data                                             */
/* ------------------------------------------------------------------------ */
/* The operator template of [EwOps] section 二 (only the middle operation
 * changes) applied to the 16-bit formats of [HyperAI] Stage 2.  Data are raw
 * uint16_t bit patterns, pointers 2-byte aligned, 8 lanes per 16-byte vector. */

/* In place: y[i] = rne16(fma(alpha, widen(x[i]), widen(y[i]))): x and y are
 * widened exactly, one binary32 fused multiply-add with the binary32 alpha,
 * then one round-to-nearest-even to binary16.  x may equal y. */
ew_status_t ew_saxpy_f16(float alpha, const uint16_t *x, uint16_t *y, size_t n,
                         hipStream_t stream);

/* The same for bfloat16. */
ew_status_t ew_saxpy_bf16(float alpha, const uint16_t *x, uint16_t *y, size_t n,
                          hipStream_t stream);

/* y[i] = maximum(x[i], +0) on binary16 / bfloat16: x's bits when x > 0 or x
 * is a NaN, else +0 (no rounding).  y may equal x. */
ew_status_t ew_relu_f16(const uint16_t *x, uint16_t *y, size_t n, hipStream_t stream);
ew_status_t ew_relu_bf16(const uint16_t *x, uint16_t *y, size_t n, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Scalar-broadcast and unary maps, in every format                          */
/* ------------------------------------------------------------------------ */
/* More instances of [EwOps] section 二's template (index, bounds check and
 * store fixed; only the middle operation replaced): y[i] = f(x[i]), one
 * input stream and one output stream, 8 bytes per fp32 element and 4 per
 * 16-bit element.  fp32: f is one binary32 operation rounded to nearest-
 * even.  _f16 / _bf16: x is widened exactly to binary32, f is applied in
 * binary32 (with the binary32 alpha), and the result is rounded once to the
 * 16-bit format, nearest-even -- the rule of the 16-bit add ([HyperAI]
 * Stage 2).  Data are raw bit patterns for the 16-bit formats; pointers
 * need element alignment.  y may equal x (in place); any other overlap is
 * EW_ERR_OVERLAP.  NaN results are NaN (payload not part of the contract)
 * except for abs, which moves bits. */

/* Scalar broadcast, multiply: y[i] = alpha * x[i]. */
ew_status_t ew_scale_f32(float alpha, const float *x, float *y, size_t n, hipStream_t stream);
ew_status_t ew_scale_f16(float alpha, const uint16_t *x, uint16_t *y, size_t n,
                         hipStream_t stream);
ew_status_t ew_scale_bf16(float alpha, const uint16_t *x, uint16_t *y, size_t n,
                          hipStream_t stream);

/* Scalar broadcast, add: y[i] = x[i] + alpha. */
ew_status_t ew_add_scalar_f32(float alpha, const float *x, float *y, size_t n,
                              hipStream_t stream);
ew_status_t ew_add_scalar_f16(float alpha, const uint16_t *x, uint16_t *y, size_t n,
                              hipStream_t stream);
ew_status_t ew_add_scalar_bf16(float alpha, const uint16_t *x, uint16_t *y, size_t n,
                               hipStream_t stream);

/* Unary: y[i] = sqrt(x[i]), correctly rounded in binary32 (sqrt(-0) = -0,
 * negative inputs give NaN); the 16-bit forms round that binary32 root to
 * the 16-bit format, which equals the correctly rounded 16-bit root. */
ew_status_t ew_sqrt_f32(const float *x, float *y, size_t n, hipStream_t stream);
ew_status_t ew_sqrt_f16(const uint16_t *x, uint16_t *y, size_t n, hipStream_t stream);
ew_status_t ew_sqrt_bf16(const uint16_t *x, uint16_t *y, size_t n, hipStream_t stream);

/* Unary: y[i] = |x[i]|, the sign bit cleared and every other bit (NaN
 * payloads included) unchanged. */
ew_status_t ew_abs_f32(const float *x, float *y, size_t n, hipStream_t stream);
ew_status_t ew_abs_f16(const uint16_t *x, uint16_t *y, size_t n, hipStream_t stream);
ew_status_t ew_abs_bf16(const uint16_t *x, uint16_t *y, size_t n, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Batched calls: many small arrays, one launch                              */
/* ------------------------------------------------------------------------ */
/* [HyperAI] Stage 3: at the smallest size every kernel version takes the
 * same few microseconds -- the launch, not the memory.  Many small arrays
 * each cost that floor through the single-array entry points; a batched call
 * runs up to EW_BATCH_MAX of them per kernel launch. */

#define EW_BATCH_MAX 96

/* One operand set: the pointers of the single call, in ew_make_plan's
 * order.  out = c (add), y (saxpy, in place), y (ReLU, maps), out (copy).
 * in0 = a (add) or x.  in1 = b (add); ignored for the one-input operations
 * and for SAXPY, whose second input is out itself. */
typedef struct ew_batch_item {
    void *out;
    const void *in0;
    const void *in1;
    size_t n;
} ew_batch_item_t;

/* Runs count independent instances of one streaming operation -- any of
 * "add_f32", "add_f16", "add_bf16", "saxpy_f32", "relu_f32", "copy_f32",
 * "add_relu_f32", "saxpy_relu_f32", "saxpy_f16", "saxpy_bf16", "relu_f16",
 * "relu_bf16" and the scale / add_scalar / sqrt / abs maps -- each with the
 * result its single call would give, in ceil(items / EW_BATCH_MAX) kernel
 * launches on `stream` (items with n == 0 are skipped).  alpha is used by
 * the SAXPY, scale and add-scalar operations and ignored otherwise.  items:
 * a host array, read during the call only.
 * Errors: an unknown or non-batchable op name, items == NULL with count >
 * 0, or host memory for the overlap check (about 72 bytes per item) not
 * available -> EW_ERR_INVALID_ARG; each item is validated like its single call
 * (first failing item's status); an item's output range intersecting any
 * range of another item -> EW_ERR_OVERLAP (the items run concurrently; reads
 * of shared inputs are fine).  count == 0 or all n == 0 -> EW_OK, no launch.
 * The launch shape is the table's row of the operation for the total element
 * count (unroll at most 4). */
ew_status_t ew_batch(const char *op, float alpha, const ew_batch_item_t *items,
                     size_t count, hipStream_t stream);

/* Batched calls with the item table in device memory: one kernel launch for
 * any number of items.  The library builds the table image on the host
 * (ew_batch_build, into memory the caller provides), the caller places it in
 * device memory (any copy; it may be reused for every call on the same
 * items), and ew_batch_run launches one kernel that reads it.  This is the
 * form to use for many items and for repeated calls on the same arrays; it
 * also suits graph capture (ew_batch_run makes no copy and allocates
 * nothing).
 *
 * ew_batch_plan_t describes a built table; fill it only through
 * ew_batch_build.  The launch shape is the table's row of the operation for
 * the total element count (unroll at most 4); the grid is min(blocks_per_cu
 * * CU count, tiles). */
typedef struct ew_batch_plan {
    int32_t op;             /* operation (library-internal number) */
    int32_t block;          /* threads per block */
    int32_t unroll;         /* 16-byte vectors per lane per tile */
    int32_t blocks_per_cu;  /* grid cap per compute unit */
    uint64_t items;         /* records in the table: the items with n > 0 */
    uint64_t tiles;         /* tiles of all items together (one block each) */
    uint64_t bytes;         /* size of the table image, a multiple of 8 */
    uint64_t total_n;       /* elements of all items together */
} ew_batch_plan_t;

/* Validates items exactly as ew_batch does (same operations, same errors)
 * and fills *plan.  With table == NULL it only sizes the image (plan->bytes)
 * and returns EW_OK; otherwise it writes the image -- plan->items records of
 * 40 bytes (in0, in1, out, n, first tile), then one 32-bit item index per
 * tile, zero padded to plan->bytes -- into `table` (host memory, 8-byte
 * aligned, table_bytes >= plan->bytes; EW_ERR_INVALID_ARG if smaller,
 * EW_ERR_MISALIGNED if not 8-byte aligned).  No device is needed.  The
 * image holds the items' device pointers: it stays valid while those
 * buffers do. */
ew_status_t ew_batch_build(const char *op, const ew_batch_item_t *items, size_t count,
                           void *table, size_t table_bytes, ew_batch_plan_t *plan);

/* Runs a built table in one kernel launch on `stream`: the result of
 * ew_batch on the same items and alpha.  table: device memory (8-byte
 * aligned) holding exactly the plan->bytes bytes that ew_batch_build wrote
 * for this plan; the kernel trusts its pointers as every entry point trusts
 * its buffers, so a table that was changed or built for other buffers is
 * undefined behaviour.  The plan's fields are checked for consistency
 * (EW_ERR_INVALID_ARG).  plan->tiles == 0 (no item with n > 0) -> EW_OK, no
 * launch.  Calls on different streams may share one table (it is only
 * read). */
ew_status_t ew_batch_run(const ew_batch_plan_t *plan, float alpha, const void *table,
                         hipStream_t stream);

/* For callers that cannot allocate device memory (no hipMalloc of their own
 * for the table: code that must not allocate, allocation-free serving
 * loops): ew_batch_run with the table image taken from host memory and
 * placed by the library in a static device array of EW_BATCH_SCRATCH_BYTES
 * that it holds on each GPU it runs on until the process ends.  The call
 * allocates nothing.  It waits for `stream` (earlier work may still read
 * the array), copies the plan->bytes bytes of table_host (the image
 * ew_batch_build wrote, in host memory) into the array on the current
 * device, waits for the copy, and launches the kernel asynchronously;
 * table_host may be reused when the call returns.  Because it waits, it
 * cannot be captured into a graph (ew_batch_run with a caller-owned device
 * table can).  Every call on one GPU shares that GPU's array, which keeps
 * the last call's table: calls that overlap on one GPU -- on different
 * streams, or from several threads -- race; calls on one stream do not.
 * plan->bytes > EW_BATCH_SCRATCH_BYTES -> EW_ERR_TOO_LARGE (use
 * ew_batch_run); other errors as for ew_batch_run. */
#define EW_BATCH_SCRATCH_BYTES (256 * 1024)
ew_status_t ew_batch_run_static(const ew_batch_plan_t *plan, float alpha, const void *table_host,
                                hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Fused chains: one pass over memory instead of two                         */
/* ------------------------------------------------------------------------ */
/* An epilogue fused into the producing kernel saves a full pass through HBM
 * ([GEMM-9.3] "what comes next": bias and ReLU inside the same kernel;
 * [PerfNotes] 5.3: fusion raises the arithmetic intensity of memory-bound
 * work).  Each result is rounded exactly as the unfused sequence would round
 * it, so the fused and unfused paths agree bit for bit. */

/* c[i] = maximum(a[i] + b[i], +0): the binary32 sum, then the ReLU of
 * ew_relu_f32.  12 bytes per element, where ew_add_f32 followed by
 * ew_relu_f32 moves 20.  Pointers 4-byte aligned; c may equal a or b. */
ew_status_t ew_add_relu_f32(const float *a, const float *b, float *c, size_t n,
                            hipStream_t stream);

/* In place: y[i] = maximum(fma(alpha, x[i], y[i]), +0).  x may equal y. */
ew_status_t ew_saxpy_relu_f32(float alpha, const float *x, float *y, size_t n,
                              hipStream_t stream);

/* y[r*cols + c] = maximum(x[r*cols + c] + bias[c], +0) for a row-major
 * rows x cols matrix: the bias row is broadcast down the rows (a bias-and-
 * activation epilogue).  x, y: rows*cols elements (y may equal x); bias: cols
 * elements, must not overlap y.  rows or cols 0 -> EW_OK.  Errors as for the
 * other operations; the bias pointer is checked after x and y. */
ew_status_t ew_bias_relu_f32(const float *x, const float *bias, float *y,
                             size_t rows, size_t cols, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Row operators of language models                                          */
/* ------------------------------------------------------------------------ */
/* Operations that reduce along the rows of a matrix: the RMS norm with the
 * residual's addition (plain and 8-bit output, gradient), log probabilities
 * of given tokens (entropy, top alternatives, gradient), distillation from
 * a teacher's top logits (gradient), the layer norm (gradient) and a clipped
 * policy loss (gradient); and the movement of rows to the experts that their
 * tokens are sent to, and back (gradient).  Each has an f32, an f16 and a bf16
 * form, but the policy loss, whose log probabilities are binary32, and the
 * sorting; 16-bit data are raw uint16_t bit patterns.
 *
 * Matrices    rows x cols, row-major, columns contiguous; row r starts
 *             r * stride elements after the pointer (stride in elements, at
 *             least cols; ignored for a single row).  Pointers and strides
 *             need only element alignment; rows that start on 16-byte
 *             boundaries are fastest.  Vectors and per-row outputs are
 *             contiguous.
 * Sizes       rows and cols below 2^31; offsets are 64-bit.  rows == 0
 *             returns EW_OK without a launch (the gradients of the norms
 *             still clear dweight and dbias, the policy loss and the sorting
 *             write their results).  cols == 0 returns EW_OK without a
 *             launch for the norms and the movement of rows; a row of logits
 *             or of log probabilities without columns is a row whose mask
 *             leaves nothing.
 * Optional    A pointer documented as optional may be NULL.
 * Workspace   Device memory of the caller's, 16-byte aligned, of at least the
 *             bytes the _workspace function gives (EW_ERR_INVALID_ARG if
 *             fewer are passed); its contents before the call do not matter
 *             and nothing is kept in it.  0 bytes: it may be NULL.
 * Aliasing    An output may be exactly an input matrix (same pointer and
 *             stride) where the operation says so.  Views of one buffer that
 *             interleave without sharing an element (equal strides, disjoint
 *             columns) do not overlap.  Any other overlap of an output with
 *             an input or another output returns EW_ERR_OVERLAP.
 * Arithmetic  In binary32 (sums, statistics and gradients too), 16-bit data
 *             widened exactly, each result rounded once to its type, nearest
 *             even.  No atomics: a call repeated on the same device gives the
 *             same bits.
 * Launches    One to three kernels on the stream; nothing synchronises or
 *             allocates, so calls can be captured in a HIP graph.
 * Errors      As above, in the same order. */

/* total = round(x + residual), rstd = 1 / sqrt(mean(total^2) + eps),
 * y = round(total * rstd * weight), row by row.  The norm is that of the
 * rounded total, which is what a later layer reads back.
 * residual    optional: without it total is x itself
 * total       optional, requires residual: the rounded sum
 * rstd        optional, rows values: what the gradient needs
 * eps         >= 0 and finite
 * total may be exactly x or residual (the usual update in place); y may be
 * exactly x or residual unless total is that one. */
ew_status_t ew_rmsnorm_f32(const float *x, size_t x_stride, const float *weight,
                           const float *residual, size_t residual_stride, float *y,
                           size_t y_stride, float *total, size_t total_stride, float *rstd,
                           size_t rows, size_t cols, float eps, hipStream_t stream);
ew_status_t ew_rmsnorm_f16(const uint16_t *x, size_t x_stride, const uint16_t *weight,
                           const uint16_t *residual, size_t residual_stride, uint16_t *y,
                           size_t y_stride, uint16_t *total, size_t total_stride, float *rstd,
                           size_t rows, size_t cols, float eps, hipStream_t stream);
ew_status_t ew_rmsnorm_bf16(const uint16_t *x, size_t x_stride, const uint16_t *weight,
                            const uint16_t *residual, size_t residual_stride, uint16_t *y,
                            size_t y_stride, uint16_t *total, size_t total_stride, float *rstd,
                            size_t rows, size_t cols, float eps, hipStream_t stream);

/* The same norm with an 8-bit output: each group of columns of a row has
 * scale = max(max |y| / 448, 2^-126) over its unrounded y, and
 * q = e4m3(y / scale) (OCP e4m3fn, nearest even, largest value 448).  A NaN
 * in a group makes its scale NaN.
 * group       columns per scale: 16, 32, 64, 128 or 256 (the last group of a
 *             row may be shorter), or 0 for one scale a row
 * q           rows x cols bytes, row stride q_stride
 * scales      rows x ceil(cols / group) floats (rows x 1 for group 0) */
ew_status_t ew_rmsnorm_e4m3_f32(const float *x, size_t x_stride, const float *weight,
                                const float *residual, size_t residual_stride, uint8_t *q,
                                size_t q_stride, float *scales, size_t group, float *total,
                                size_t total_stride, float *rstd, size_t rows, size_t cols,
                                float eps, hipStream_t stream);
ew_status_t ew_rmsnorm_e4m3_f16(const uint16_t *x, size_t x_stride, const uint16_t *weight,
                                const uint16_t *residual, size_t residual_stride, uint8_t *q,
                                size_t q_stride, float *scales, size_t group, uint16_t *total,
                                size_t total_stride, float *rstd, size_t rows, size_t cols,
                                float eps, hipStream_t stream);
ew_status_t ew_rmsnorm_e4m3_bf16(const uint16_t *x, size_t x_stride, const uint16_t *weight,
                                 const uint16_t *residual, size_t residual_stride, uint8_t *q,
                                 size_t q_stride, float *scales, size_t group, uint16_t *total,
                                 size_t total_stride, float *rstd, size_t rows, size_t cols,
                                 float eps, hipStream_t stream);

/* The norm's gradient.  x is the normed matrix (the forward call's total),
 * rstd its statistic, dy the gradient of y and dtotal (optional) that of
 * total; with n = cols, per row
 *   dx = round(rstd*weight*dy - x*(rstd^3/n)*sum(x*weight*dy) + dtotal)
 * (the gradient of the forward call's x and of its residual alike), and
 *   dweight[c] = sum over rows of dy*x*rstd, in binary32 (optional).
 * dx may be exactly dy, x or dtotal.  The workspace is needed for dweight
 * only (without dweight it may be NULL). */
size_t ew_rmsnorm_grad_workspace(size_t rows, size_t cols);
ew_status_t ew_rmsnorm_grad_f32(const float *dy, size_t dy_stride, const float *x,
                                size_t x_stride, const float *weight, const float *rstd,
                                const float *dtotal, size_t dtotal_stride, float *dx,
                                size_t dx_stride, float *dweight, void *workspace,
                                size_t workspace_bytes, size_t rows, size_t cols,
                                hipStream_t stream);
ew_status_t ew_rmsnorm_grad_f16(const uint16_t *dy, size_t dy_stride, const uint16_t *x,
                                size_t x_stride, const uint16_t *weight, const float *rstd,
                                const uint16_t *dtotal, size_t dtotal_stride, uint16_t *dx,
                                size_t dx_stride, float *dweight, void *workspace,
                                size_t workspace_bytes, size_t rows, size_t cols,
                                hipStream_t stream);
ew_status_t ew_rmsnorm_grad_bf16(const uint16_t *dy, size_t dy_stride, const uint16_t *x,
                                 size_t x_stride, const uint16_t *weight, const float *rstd,
                                 const uint16_t *dtotal, size_t dtotal_stride, uint16_t *dx,
                                 size_t dx_stride, float *dweight, void *workspace,
                                 size_t workspace_bytes, size_t rows, size_t cols,
                                 hipStream_t stream);

/* Log probabilities of given tokens.  With s = scale * logits in binary32
 * (scale finite and > 0: the reciprocal of a temperature), per row
 *   lse     = log(sum exp(s))                           (optional)
 *   logp    = s[target] - lse; 0 where target is outside [0, cols), as for
 *             the padding positions of a batch
 *   entropy = -sum p log p, p = exp(s - lse)            (optional)
 *   top_ids, top_logp: the `top` most likely columns, most likely first,
 *             ties to the lowest column, and their s - lse; rows x top
 *             values, both or neither; top <= min(64, cols).
 * A logit whose s is -inf is masked: p = 0 and nothing of it enters the sums.
 * (A type's lowest value is a number: where its s is finite a row of nothing
 * else is an even one.)  A row whose mask leaves nothing has lse = -inf,
 * entropy 0, logp -inf (0 without a target) and top_logp -inf.  A row that
 * holds a NaN or a scaled logit of +inf has NaN in lse, entropy, top_logp and
 * the logp of a given target.  For the ranking a NaN counts as -inf, so
 * top_ids always holds `top` different columns. */
size_t ew_logprobs_workspace(size_t rows, size_t cols, size_t top);
ew_status_t ew_logprobs_f32(const float *logits, size_t stride, const int64_t *targets,
                            float *logp, float *entropy, float *lse, float *top_logp,
                            int64_t *top_ids, size_t top, float scale, void *workspace,
                            size_t workspace_bytes, size_t rows, size_t cols,
                            hipStream_t stream);
ew_status_t ew_logprobs_f16(const uint16_t *logits, size_t stride, const int64_t *targets,
                            float *logp, float *entropy, float *lse, float *top_logp,
                            int64_t *top_ids, size_t top, float scale, void *workspace,
                            size_t workspace_bytes, size_t rows, size_t cols,
                            hipStream_t stream);
ew_status_t ew_logprobs_bf16(const uint16_t *logits, size_t stride, const int64_t *targets,
                             float *logp, float *entropy, float *lse, float *top_logp,
                             int64_t *top_ids, size_t top, float scale, void *workspace,
                             size_t workspace_bytes, size_t rows, size_t cols,
                             hipStream_t stream);

/* Their gradient, from the forward call's lse (and entropy):
 *   dlogits[c] = round(scale * (dlogp * (1[c == target] - p)
 *                               - dentropy * p * (s - lse + entropy)))
 * with no dlogp term in a row without a target; 0 where s is -inf (whatever
 * dlogp and dentropy are, infinite or NaN too) and in a row whose mask leaves
 * nothing (lse = -inf).  A p below 2^-126 counts as 0.  dentropy is optional,
 * entropy required with it.  dlogits may be exactly logits. */
ew_status_t ew_logprobs_grad_f32(const float *logits, size_t stride, const int64_t *targets,
                                 const float *lse, const float *entropy, const float *dlogp,
                                 const float *dentropy, float *dlogits, size_t dlogits_stride,
                                 float scale, size_t rows, size_t cols, hipStream_t stream);
ew_status_t ew_logprobs_grad_f16(const uint16_t *logits, size_t stride, const int64_t *targets,
                                 const float *lse, const float *entropy, const float *dlogp,
                                 const float *dentropy, uint16_t *dlogits,
                                 size_t dlogits_stride, float scale, size_t rows, size_t cols,
                                 hipStream_t stream);
ew_status_t ew_logprobs_grad_bf16(const uint16_t *logits, size_t stride, const int64_t *targets,
                                  const float *lse, const float *entropy, const float *dlogp,
                                  const float *dentropy, uint16_t *dlogits,
                                  size_t dlogits_stride, float scale, size_t rows, size_t cols,
                                  hipStream_t stream);

/* Distillation from a teacher's `kept` top logits: teacher and ids are
 * rows x kept.  An entry whose id is outside [0, cols), or whose scaled
 * teacher logit is -inf, is dropped; t is the softmax of scale * teacher over
 * the entries that remain (NaN if one of them is a NaN or +inf),
 * and with s and lse as for the log probabilities
 *   loss = sum t * (log t - (s[id] - lse))
 * per row: 0 if no entry remains; entries whose t underflows (below 2^-126)
 * add nothing; +inf if another entry meets a masked logit.  A column named twice counts twice.
 * lse is optional.  scale is finite and > 0, kept <= 1024. */
size_t ew_distill_workspace(size_t rows, size_t cols);
ew_status_t ew_distill_f32(const float *logits, size_t stride, const float *teacher,
                           const int64_t *ids, size_t kept, float *loss, float *lse, float scale,
                           void *workspace, size_t workspace_bytes, size_t rows, size_t cols,
                           hipStream_t stream);
ew_status_t ew_distill_f16(const uint16_t *logits, size_t stride, const float *teacher,
                           const int64_t *ids, size_t kept, float *loss, float *lse, float scale,
                           void *workspace, size_t workspace_bytes, size_t rows, size_t cols,
                           hipStream_t stream);
ew_status_t ew_distill_bf16(const uint16_t *logits, size_t stride, const float *teacher,
                            const int64_t *ids, size_t kept, float *loss, float *lse, float scale,
                            void *workspace, size_t workspace_bytes, size_t rows, size_t cols,
                            hipStream_t stream);

/* Its gradient, from the forward call's lse:
 *   dlogits[c] = round(scale * dloss * (p - sum of t over entries naming c))
 * and 0 where s is -inf (whatever dloss is), in a row without a kept entry
 * and in a row whose mask leaves nothing.  A p or t below 2^-126 counts as 0.
 * dlogits may be exactly logits. */
ew_status_t ew_distill_grad_f32(const float *logits, size_t stride, const float *teacher,
                                const int64_t *ids, size_t kept, const float *lse,
                                const float *dloss, float *dlogits, size_t dlogits_stride,
                                float scale, size_t rows, size_t cols, hipStream_t stream);
ew_status_t ew_distill_grad_f16(const uint16_t *logits, size_t stride, const float *teacher,
                                const int64_t *ids, size_t kept, const float *lse,
                                const float *dloss, uint16_t *dlogits, size_t dlogits_stride,
                                float scale, size_t rows, size_t cols, hipStream_t stream);
ew_status_t ew_distill_grad_bf16(const uint16_t *logits, size_t stride, const float *teacher,
                                 const int64_t *ids, size_t kept, const float *lse,
                                 const float *dloss, uint16_t *dlogits, size_t dlogits_stride,
                                 float scale, size_t rows, size_t cols, hipStream_t stream);

/* Layer norm, row by row, with n = cols:
 *   total = round(x + residual), mean = sum(total) / n,
 *   rstd = 1 / sqrt(sum((total - mean)^2) / n + eps),
 *   y = round((total - mean) * rstd * weight + bias).
 * Differences are taken from the row's mean to 24 bits of the difference,
 * however far the row lies from 0: a row of equal values has y = bias exactly
 * (for eps > 0).  The numbers of total may be of any size, also where their
 * differences or the squares of these leave binary32 (rstd does for eps = 0 and
 * a standard deviation below 2^-128).  A row that holds a NaN or an infinity has
 * NaN in mean, rstd and y.
 * weight, bias  each optional: 1 and 0 where absent
 * residual      optional: without it total is x itself
 * total         optional, requires residual: the rounded sum
 * mean, rstd    optional, rows values each: what the gradient needs
 * eps           >= 0 and finite
 * total may be exactly x or residual; y may be exactly x or residual unless
 * total is that one. */
ew_status_t ew_layernorm_f32(const float *x, size_t x_stride, const float *weight,
                             const float *bias, const float *residual, size_t residual_stride,
                             float *y, size_t y_stride, float *total, size_t total_stride,
                             float *mean, float *rstd, size_t rows, size_t cols, float eps,
                             hipStream_t stream);
ew_status_t ew_layernorm_f16(const uint16_t *x, size_t x_stride, const uint16_t *weight,
                             const uint16_t *bias, const uint16_t *residual, size_t residual_stride,
                             uint16_t *y, size_t y_stride, uint16_t *total, size_t total_stride,
                             float *mean, float *rstd, size_t rows, size_t cols, float eps,
                             hipStream_t stream);
ew_status_t ew_layernorm_bf16(const uint16_t *x, size_t x_stride, const uint16_t *weight,
                              const uint16_t *bias, const uint16_t *residual,
                              size_t residual_stride, uint16_t *y, size_t y_stride, uint16_t *total,
                              size_t total_stride, float *mean, float *rstd, size_t rows,
                              size_t cols, float eps, hipStream_t stream);

/* The layer norm's gradient.  x is the normed matrix (the forward call's
 * total), mean and rstd its statistics, dy the gradient of y and dtotal
 * (optional) that of total; with h = (x - mean) * rstd and g = dy * weight
 * (weight optional), per row
 *   dx = round(rstd * (g - sum(g) / n - h * sum(g * h) / n) + dtotal)
 * (the gradient of the forward call's x and of its residual alike), and
 *   dweight[c] = sum over rows of dy * h, dbias[c] = sum over rows of dy,
 * in binary32, each optional.  mean is taken as given, rounded to binary32; of
 * rows whose mean is more than 2^12 standard deviations (1 / rstd) from 0, where
 * that rounding is up to 2^-12 of one and more, h is about the row's own mean,
 * sum(x) / n.  dx may be exactly dy, x or dtotal.  The workspace is needed for
 * dweight and dbias only (without both it may be NULL). */
size_t ew_layernorm_grad_workspace(size_t rows, size_t cols);
ew_status_t ew_layernorm_grad_f32(const float *dy, size_t dy_stride, const float *x,
                                  size_t x_stride, const float *weight, const float *mean,
                                  const float *rstd, const float *dtotal, size_t dtotal_stride,
                                  float *dx, size_t dx_stride, float *dweight, float *dbias,
                                  void *workspace, size_t workspace_bytes, size_t rows, size_t cols,
                                  hipStream_t stream);
ew_status_t ew_layernorm_grad_f16(const uint16_t *dy, size_t dy_stride, const uint16_t *x,
                                  size_t x_stride, const uint16_t *weight, const float *mean,
                                  const float *rstd, const uint16_t *dtotal, size_t dtotal_stride,
                                  uint16_t *dx, size_t dx_stride, float *dweight, float *dbias,
                                  void *workspace, size_t workspace_bytes, size_t rows, size_t cols,
                                  hipStream_t stream);
ew_status_t ew_layernorm_grad_bf16(const uint16_t *dy, size_t dy_stride, const uint16_t *x,
                                   size_t x_stride, const uint16_t *weight, const float *mean,
                                   const float *rstd, const uint16_t *dtotal, size_t dtotal_stride,
                                   uint16_t *dx, size_t dx_stride, float *dweight, float *dbias,
                                   void *workspace, size_t workspace_bytes, size_t rows,
                                   size_t cols, hipStream_t stream);

/* How the policy loss weighs its tokens: by the number of counted tokens of
 * the batch; by that of each sequence, and the number of sequences that have
 * any; or not at all. */
typedef enum ew_mean {
    EW_MEAN_TOKENS = 0,
    EW_MEAN_SEQUENCES = 1,
    EW_MEAN_NONE = 2
} ew_mean_t;

/* Clipped policy loss with a KL term, over the tokens of `rows` sequences of
 * at most `cols`.  Of a counted token, with x = logp - old_logp, r = exp(x),
 * a its advantage and d = ref_logp - logp,
 *   gain = min(r * a, clip(r, 1 - clip_low, 1 + clip_high) * a)
 *   k    = exp(d) - d - 1       (0 without ref_logp)
 * and, w being the weight of its sequence's tokens (scale / number of counted
 * tokens of the batch, scale / (number of counted tokens of the sequence *
 * number of sequences that have any), or scale),
 *   loss = sum w * (kl * k - gain).
 * Which side of a border r lies on is decided exactly (x against the border's
 * logarithm, in binary64); r, k and each gain are binary32, r and exp(d) off by
 * about |x| and |d| times 2^-24 of themselves; sums are binary64.  Where r is past
 * binary32 (x above 88.7) it is infinite, but a token of advantage 0 adds 0.  A
 * batch or sequence whose mask leaves nothing adds nothing, whatever lies in its
 * masked places: its weights are 0, and a loss of no tokens is 0.
 * ref_logp    optional; kl weighs its term, which is left out where kl is 0
 * advantage   a matrix, or with advantage_stride 0 one value a sequence
 * mask        optional, rows x cols bytes with a stride of its own: tokens
 *             whose byte is not 0 count; without it all do
 * loss        one value
 * stats       optional, four values: -sum w * gain, sum w * k, the fraction
 *             of counted tokens whose gain is the clipped one, and the mean of
 *             old_logp - logp over counted tokens
 * weights     optional, rows values: w (0 for a sequence of no counted
 *             tokens), which the gradient needs
 * clip_low, clip_high   >= 0, infinity for no clip on that side
 * kl          >= 0 and finite; scale finite
 * mean        an ew_mean_t */
size_t ew_policy_loss_workspace(size_t rows, size_t cols);
ew_status_t ew_policy_loss_f32(const float *logp, size_t logp_stride, const float *old_logp,
                               size_t old_stride, const float *ref_logp, size_t ref_stride,
                               const float *advantage, size_t advantage_stride,
                               const uint8_t *mask, size_t mask_stride, float *loss, float *stats,
                               float *weights, float clip_low, float clip_high, float kl,
                               float scale, int mean, void *workspace,
                               size_t workspace_bytes, size_t rows, size_t cols,
                               hipStream_t stream);

/* Its gradient by logp, from the forward call's weights:
 *   dlogp = dloss * w * (-(clipped ? 0 : r * a) - kl * (exp(d) - 1))
 * for counted tokens, 0 for the others.  dloss is one value on the device
 * (optional: 1).  dlogp may be exactly one of the matrices it is computed
 * from. */
ew_status_t ew_policy_loss_grad_f32(const float *logp, size_t logp_stride, const float *old_logp,
                                    size_t old_stride, const float *ref_logp, size_t ref_stride,
                                    const float *advantage, size_t advantage_stride,
                                    const uint8_t *mask, size_t mask_stride,
                                    const float *weights, const float *dloss, float *dlogp,
                                    size_t dlogp_stride, float clip_low, float clip_high,
                                    float kl, size_t rows, size_t cols, hipStream_t stream);

/* Sorting of entries (a token's choices of experts, in the tokens' order) by
 * expert: entries of expert e get consecutive rows from offsets[e] on, in
 * their own order; offsets[e] is a multiple of align.  An entry whose id is
 * outside [0, experts) is dropped.
 * slot        entries values: the row of each entry, -1 for a dropped one
 * offsets     experts + 1 values: each expert's first row, and the end of the
 *             last expert's rows
 * counts      optional, experts values: entries of each expert (the rows from
 *             offsets[e] + counts[e] to offsets[e + 1] are padding)
 * source      optional, ew_experts_rows() values: the entry of each row, -1
 *             for a row without one
 * experts and align in [1, 1024], ew_experts_rows() < 2^31 (it is the rows
 * that any ids of these sizes fit in: entries + min(entries, experts) *
 * (align - 1), rounded up to a multiple of align; SIZE_MAX for sizes no call
 * accepts). */
size_t ew_experts_rows(size_t entries, size_t experts, size_t align);
size_t ew_experts_sort_workspace(size_t entries, size_t experts);
ew_status_t ew_experts_sort(const int64_t *ids, size_t entries, size_t experts, size_t align,
                            int32_t *slot, int32_t *offsets, int32_t *counts, int32_t *source,
                            void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Rows of x to the places of their entries: out[slot[t * top + j]] = x[t] for
 * t < rows, j < top.  Entries whose slot is outside [0, out_rows) are dropped;
 * the others' slots differ.  With offsets and counts (both or neither) the
 * padding rows of each of `experts` experts become 0; all other rows of out
 * stay as they are.  top in [1, 64].  The gradient of x is
 * ew_experts_combine_* of that of out, without weights. */
ew_status_t ew_experts_gather_f32(const float *x, size_t x_stride, const int32_t *slot, size_t top,
                                  const int32_t *offsets, const int32_t *counts, size_t experts,
                                  float *out, size_t out_stride, size_t out_rows, size_t rows,
                                  size_t cols, hipStream_t stream);
ew_status_t ew_experts_gather_f16(const uint16_t *x, size_t x_stride, const int32_t *slot,
                                  size_t top, const int32_t *offsets, const int32_t *counts,
                                  size_t experts, uint16_t *out, size_t out_stride, size_t out_rows,
                                  size_t rows, size_t cols, hipStream_t stream);
ew_status_t ew_experts_gather_bf16(const uint16_t *x, size_t x_stride, const int32_t *slot,
                                   size_t top, const int32_t *offsets, const int32_t *counts,
                                   size_t experts, uint16_t *out, size_t out_stride,
                                   size_t out_rows, size_t rows, size_t cols, hipStream_t stream);

/* Rows of z back to their tokens, weighed:
 *   y[t] = round(residual[t] + sum over j of weights[t * top + j] *
 *                z[slot[t * top + j]])
 * in the order of j, without the entries whose slot is outside [0, z_rows).
 * weights (rows x top values) are 1 where absent, residual is 0.  y may be
 * exactly residual. */
ew_status_t ew_experts_combine_f32(const float *z, size_t z_stride, size_t z_rows,
                                   const int32_t *slot, size_t top, const float *weights,
                                   const float *residual, size_t residual_stride, float *y,
                                   size_t y_stride, size_t rows, size_t cols, hipStream_t stream);
ew_status_t ew_experts_combine_f16(const uint16_t *z, size_t z_stride, size_t z_rows,
                                   const int32_t *slot, size_t top, const float *weights,
                                   const uint16_t *residual, size_t residual_stride, uint16_t *y,
                                   size_t y_stride, size_t rows, size_t cols, hipStream_t stream);
ew_status_t ew_experts_combine_bf16(const uint16_t *z, size_t z_stride, size_t z_rows,
                                    const int32_t *slot, size_t top, const float *weights,
                                    const uint16_t *residual, size_t residual_stride, uint16_t *y,
                                    size_t y_stride, size_t rows, size_t cols, hipStream_t stream);

/* The gradient of that by z and the weights, from the gradient dy of y (which
 * is that of residual too):
 *   dz[slot[t * top + j]] = round(weights[t * top + j] * dy[t])
 *   dweights[t * top + j] = sum over columns of dy[t] * z[slot[t * top + j]]
 * (0 where the entry is dropped).  The kept entries' slots differ.  Padding
 * rows and other rows of dz (z_rows, as z) are treated as ew_experts_gather_*
 * treats out's.  dz may be exactly z. */
ew_status_t ew_experts_combine_grad_f32(const float *dy, size_t dy_stride, const float *z,
                                        size_t z_stride, size_t z_rows, const int32_t *slot,
                                        size_t top, const float *weights, const int32_t *offsets,
                                        const int32_t *counts, size_t experts, float *dz,
                                        size_t dz_stride, float *dweights, size_t rows, size_t cols,
                                        hipStream_t stream);
ew_status_t ew_experts_combine_grad_f16(const uint16_t *dy, size_t dy_stride, const uint16_t *z,
                                        size_t z_stride, size_t z_rows, const int32_t *slot,
                                        size_t top, const float *weights, const int32_t *offsets,
                                        const int32_t *counts, size_t experts, uint16_t *dz,
                                        size_t dz_stride, float *dweights, size_t rows, size_t cols,
                                        hipStream_t stream);
ew_status_t ew_experts_combine_grad_bf16(const uint16_t *dy, size_t dy_stride, const uint16_t *z,
                                         size_t z_stride, size_t z_rows, const int32_t *slot,
                                         size_t top, const float *weights, const int32_t *offsets,
                                         const int32_t *counts, size_t experts, uint16_t *dz,
                                         size_t dz_stride, float *dweights, size_t rows,
                                         size_t cols, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Status, launch configuration and planning                                */
/* ------------------------------------------------------------------------ */

/* Static string for a status code (never NULL). */
const char *ew_status_string(ew_status_t status);

/* The hipError_t behind the most recent EW_ERR_HIP on the calling thread
 * (0 if none). */
int ew_last_hip_error(void);

/* Library ABI version (incremented on any incompatible change). */
int ew_abi_version(void);

/* Launch configuration, per operation name ("add_f32", "add_f16",
 * "add_bf16", "saxpy_f32", "relu_f32", "copy_f32", "gather_f32",
 * "gather_walk_f32", "add_relu_f32", "saxpy_relu_f32", "bias_relu_f32",
 * "saxpy_f16", "saxpy_bf16", "relu_f16", "relu_bf16", "copy2d_f32",
 * "relu_inplace_f32", "scale_f32", "scale_f16", "scale_bf16",
 * "add_scalar_f32", "add_scalar_f16", "add_scalar_bf16", "sqrt_f32",
 * "sqrt_f16", "sqrt_bf16", "abs_f32", "abs_f16", "abs_bf16").
 * A launch is `grid` blocks of `block` threads; each block walks tiles of
 * block * unroll 16-byte vectors with a grid stride, and the grid is
 * min(blocks_per_cu * CU count, number of tiles) ([EwOps] section 二,
 * optimisation point 2: a grid sized to the processor count times a small
 * factor).  block: a multiple of 64 in [64, 1024]; blocks_per_cu in
 * [1, 1024]; unroll in {1, 2, 4, 8}.  Out of range or unknown op ->
 * EW_ERR_INVALID_ARG.
 *
 * The table holds, per operation, rows for size classes (see
 * ew_set_launch_row); the compiled-in rows were tuned on MI355X. */

/* One launch configuration for every size of `op`: replaces all of op's
 * rows with one row applying to every n. */
ew_status_t ew_set_launch_config(const char *op, int block, int blocks_per_cu, int unroll);

/* The launch the next call of `op` with n elements would make on the
 * current device, for pointers 16-byte aligned (as device allocations are):
 * threads per block, grid (0 when n == 0: no launch) and unroll.  For the
 * gather this is the index walk's grid (ew_gather_walk_f32, or
 * ew_gather_f32 at a stride that takes the walk); ew_make_gather_plan gives
 * the grid for a given stride.  Needs a device: EW_ERR_NO_DEVICE without
 * one. */
ew_status_t ew_get_launch_config(const char *op, size_t n, int *block, int *grid, int *unroll);

/* Size classes: a row applies to every n >= min_n up to the next row's
 * min_n; setting a row with an existing min_n replaces it (at most 16 rows
 * per operation, else EW_ERR_INVALID_ARG). */
ew_status_t ew_set_launch_row(const char *op, size_t min_n, int block, int blocks_per_cu,
                              int unroll);

/* The row that applies to n (no device needed). */
ew_status_t ew_get_launch_row(const char *op, size_t n, int *block, int *blocks_per_cu,
                              int *unroll);

/* Restore the compiled-in table (tuned on MI355X). */
void ew_reset_launch_config(void);

/* Read rows "op min_n block blocks_per_cu unroll" (one per line, '#'
 * comments) from a text file and apply them with ew_set_launch_row.
 * EW_ERR_INVALID_ARG on an unreadable file or a malformed row (rows before
 * it stay applied). */
ew_status_t ew_load_launch_table(const char *path);

/* The host-side plan of one call: how the n elements split into a scalar
 * head, a body of 16-byte vectors and a scalar tail, and how the body is
 * launched.  Pure arithmetic on the pointer values -- nothing is touched and
 * no device is needed (pass cu_count explicitly).
 *   head       elements before the output reaches 16-byte alignment
 *              ((16 - out mod 16) mod 16) / element size, capped at n
 *              (64-byte alignment, 64 in place of 16, for relu_inplace_f32)
 *   vectors    16-byte vectors in the body, floor((n - head) / vec_elems)
 *   tail       n - head - vectors * vec_elems  (< vec_elems)
 *   in_coaligned[k]  1 if input k's body start is 16-byte aligned too
 *              (then it is read with aligned 16-byte loads; otherwise with
 *              4- or 2-byte aligned 16-byte loads); unused inputs report 1
 *   tiles      ceil(vectors / (block * unroll))
 *   grid       min(blocks_per_cu * cu_count, tiles), at least 1 when n > 0
 *   segment, reps, passes   n, 1 and 1, except for the gather
 *              (ew_make_gather_plan)
 *   path       the kernel path (ew_path_t): EW_PATH_STREAM, or
 *              EW_PATH_GATHER_WALK for "gather_walk_f32"
 * Validation is the same as the operation's (in1 is ignored for one-input
 * ops; for saxpy in0 = x and out = y). */
/* Which kernel path a plan launches. */
typedef enum ew_path {
    EW_PATH_STREAM = 0,          /* the streaming kernel: head / 16-byte body / tail */
    EW_PATH_COPY = 1,            /* a gather with stride 1 mod n: the contiguous copy */
    EW_PATH_GATHER_WALK = 2,     /* per-output index walk (reps equal segments) */
    EW_PATH_GATHER_SPANS = 3,    /* stride 2: contiguous 16-byte loads, even elements kept */
    EW_PATH_GATHER_PASSES = 4,   /* stride 2..32: spans staged through LDS, runs written */
    EW_PATH_VIEW_ROWS = 5,       /* strided view, rows contiguous */
    EW_PATH_VIEW_TRANSPOSE = 6,  /* strided view, 128 x 128 tiles through LDS */
    EW_PATH_VIEW_GENERIC = 7,    /* strided view, one 4-byte load per element */
    EW_PATH_GATHER_TILES = 8     /* stride > 32: rows of `stride` elements transposed
                                    through LDS, each column written as a run */
} ew_path_t;

typedef struct ew_plan {
    size_t n;
    size_t head;
    size_t vectors;
    size_t tail;
    size_t tiles;
    int vec_elems;
    int elem_size;
    int in_coaligned[2];
    int block;
    int blocks_per_cu;
    int unroll;
    int grid;
    size_t segment;
    int reps;
    int passes;
    int path;               /* an ew_path_t */
} ew_plan_t;

ew_status_t ew_make_plan(const char *op, const void *out, const void *in0,
                         const void *in1, size_t n, int cu_count,
                         ew_plan_t *plan);

/* The gather's plan.  Let s = stride mod n and g = gcd(s, n): output
 * elements i and i + n/g read the same input element, so the output
 * consists of reps = g equal segments of segment = n/g elements, and the
 * kernels compute one segment and store each value g times, so that each
 * input line is fetched once rather than g times.
 * s == 1 (or n == 1): the contiguous copy (path EW_PATH_COPY, the copy's
 * plan).  s == 2 with g == 2 and n/2 a multiple of 4: a kernel that reads the
 * input with contiguous 16-byte loads (EW_PATH_GATHER_SPANS; head / vectors
 * / tail describe one segment).
 * Otherwise 2 <= s <= 32 (EW_PATH_GATHER_PASSES): with s' = s/g, a segment
 * splits into passes = s' contiguous runs: run k holds the i with
 * floor(s'*i / segment) == k and reads every s-th input element from an
 * offset g*r that differs per run (0 <= r < s'), so slot m of all runs reads
 * from the s consecutive elements s*m .. s*m + s - 1.  The kernel reads the
 * input once, contiguously (staged through LDS), and writes the runs;
 * vectors = groups of four slots of the longest run (ceil(segment / s')),
 * head = tail = 0, block = 256 and unroll = 1 whatever the table says (its
 * blocks_per_cu still caps the grid; the kernel's own LDS reservation limits
 * how many of its blocks share a compute unit).
 * Otherwise, for s > 32 with s' = s/g >= 2, g < 32, at least 128 rows
 * (ceil(n / s) >= 128), s' < 2^32 and s' * (n/g) < 2^64
 * (EW_PATH_GATHER_TILES): the input viewed as rows of s elements,
 * A[m][c] = in[s*m + c], is transposed through LDS: column g*r of A is one
 * run of a segment (passes = s', clamped to INT_MAX; the run of column g*r
 * is the k-th with k = (-r * (n/g)^-1) mod s'), written from output
 * ceil(k * segment / s') on.  block = 1024, unroll = 1, one block per tile
 * (tiles: for s < 68 bands of floor(16384 / s) rounded down to a multiple
 * of 4 whole rows, kept one word apart in LDS when s is a multiple of 4,
 * else 128 x 128 tiles while A has fewer than 1024 rows and
 * 256 rows x 64 columns from there on), the grid capped at the table's
 * blocks_per_cu per compute unit, vectors = ceil(segment / 4),
 * head = tail = 0.
 * Otherwise (s == 0, or a large stride outside those bounds) the per-output
 * index walk (EW_PATH_GATHER_WALK), on one segment when n/g is a multiple of
 * 4 and 2 <= g <= 8 or n/g >= 2^14 (else segment = n and reps = 1);
 * passes = 1.
 * Same validation as ew_gather_f32. */
ew_status_t ew_make_gather_plan(const void *out, const void *in, size_t n,
                                size_t stride, int cu_count, ew_plan_t *plan);

/* The plan of ew_copy2d_f32 with these arguments: its path (x[::2] ->
 * EW_PATH_GATHER_SPANS, x[::s] with s = 3..32 -> EW_PATH_GATHER_PASSES with
 * passes = 1 (one run), stride_c == 1 -> EW_PATH_VIEW_ROWS, stride_r == 1 ->
 * EW_PATH_VIEW_TRANSPOSE, else EW_PATH_VIEW_GENERIC) and the launch it makes
 * (block, grid, unroll as launched; a kernel with a fixed block shape reports
 * that shape; tiles counts 128 x 128 tiles for the transpose).  No device is
 * needed.  Same validation as ew_copy2d_f32. */
ew_status_t ew_make_copy2d_plan(const void *in, int64_t stride_r, int64_t stride_c,
                                const void *out, size_t rows, size_t cols, int cu_count,
                                ew_plan_t *plan);

#ifdef __cplusplus
}
#endif

#endif /* EW_H_ */
