/* ew_rows_fuzz.c -- randomised calls of the row operators' entry points with
 * fabricated device addresses, for a library whose host code is built with
 * sanitizers.  With no GPU visible every call that passes validation ends
 * with EW_ERR_NO_DEVICE, so nothing is launched; a workspace function must
 * not depend on anything but its sizes.
 *
 *   ew_rows_fuzz CALLS SEED
 *
 * Prints the number of each status; exits 1 on a status the header does not
 * define, or on EW_ERR_HIP. */
#include "ew.h"

#include <math.h>
#include <stdio.h>
#include <stdlib.h>

static uint64_t state;

static uint64_t rnd(void)
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}

static size_t size_value(void)
{
    static const size_t odd[] = {0, 1, 2, 63, 64, 65, 4096, 16384, 49152, 49153, (size_t)1 << 31,
                                 ((size_t)1 << 31) - 1, (size_t)1 << 60, SIZE_MAX, SIZE_MAX / 2};
    return rnd() % 3 ? 1 + rnd() % 5000 : odd[rnd() % (sizeof odd / sizeof odd[0])];
}

static size_t stride_value(size_t cols)
{
    return rnd() % 4 ? cols + rnd() % 9 : size_value();
}

/* mostly distinct, aligned addresses; sometimes null, shared, odd or high */
static void *address(unsigned k)
{
    const uint64_t r = rnd() % 40;
    if (r == 0) return NULL;
    if (r == 1) return (void *)(uintptr_t)(UINT64_MAX - rnd() % 4096);
    uintptr_t a = 0x7f0000000000u + ((uintptr_t)(r == 2 ? 0 : k) << 40);
    if (r == 3) a += 1 + rnd() % 15;
    return (void *)a;
}

static float scalar(void)
{
    static const float odd[] = {0.0f, -1.0f, INFINITY, -INFINITY, NAN, 1e-38f, 3e38f};
    return rnd() % 4 ? 0.5f : odd[rnd() % (sizeof odd / sizeof odd[0])];
}

static long counts[16];
static int failures;

static void note(ew_status_t st)
{
    const int s = -(int)st;
    if (s < 0 || s > 6 || st == EW_ERR_HIP) ++failures;
    else ++counts[s];
}

#define P(k) address(k)
#define ONE_TYPE(E, X)                                                                            \
    static void call_##X(void)                                                                    \
    {                                                                                             \
        const size_t rows = size_value(), cols = size_value(), k = size_value();                  \
        const size_t ws = rnd() % 4 ? (size_t)1 << 40 : size_value();                             \
        switch (rnd() % 7) {                                                                      \
        case 0:                                                                                   \
            note(ew_rmsnorm_##X(P(1), stride_value(cols), P(2), P(3), stride_value(cols), P(4),   \
                                stride_value(cols), P(5), stride_value(cols), P(6), rows, cols,   \
                                scalar(), NULL));                                                 \
            break;                                                                                \
        case 1:                                                                                   \
            note(ew_rmsnorm_e4m3_##X(P(1), stride_value(cols), P(2), P(3), stride_value(cols),    \
                                     P(4), stride_value(cols), P(7),                              \
                                     rnd() % 2 ? (size_t)16 << rnd() % 5 : size_value(), P(5),    \
                                     stride_value(cols), P(6), rows, cols, scalar(), NULL));      \
            break;                                                                                \
        case 2:                                                                                   \
            note(ew_rmsnorm_grad_##X(P(1), stride_value(cols), P(2), stride_value(cols), P(3),    \
                                     P(4), P(5), stride_value(cols), P(6), stride_value(cols),    \
                                     P(7), P(8), ws, rows, cols, NULL));                          \
            break;                                                                                \
        case 3:                                                                                   \
            note(ew_logprobs_##X(P(1), stride_value(cols), P(2), P(3), P(4), P(5), P(6), P(7),    \
                                 rnd() % 2 ? rnd() % 65 : k, scalar(), P(8), ws, rows, cols,      \
                                 NULL));                                                          \
            break;                                                                                \
        case 4:                                                                                   \
            note(ew_logprobs_grad_##X(P(1), stride_value(cols), P(2), P(3), P(4), P(5), P(6),     \
                                      P(7), stride_value(cols), scalar(), rows, cols, NULL));     \
            break;                                                                                \
        case 5:                                                                                   \
            note(ew_distill_##X(P(1), stride_value(cols), P(2), P(3), rnd() % 2 ? rnd() % 99 : k, \
                                P(4), P(5), scalar(), P(6), ws, rows, cols, NULL));               \
            break;                                                                                \
        default:                                                                                  \
            note(ew_distill_grad_##X(P(1), stride_value(cols), P(2), P(3),                        \
                                     rnd() % 2 ? rnd() % 99 : k, P(4), P(5), P(6),                \
                                     stride_value(cols), scalar(), rows, cols, NULL));            \
        }                                                                                         \
        if (ew_logprobs_workspace(rows, cols, k) < ew_logprobs_workspace(rows, cols, 0) &&        \
            k <= 64)                                                                              \
            ++failures;                                                                           \
        if (ew_rmsnorm_grad_workspace(rows, cols) % 4 || ew_distill_workspace(rows, cols) % 16)   \
            ++failures;                                                                           \
    }

ONE_TYPE(float, f32)
ONE_TYPE(uint16_t, f16)
ONE_TYPE(uint16_t, bf16)

int main(int argc, char **argv)
{
    if (argc < 3) return 2;
    const long calls = atol(argv[1]);
    state = strtoull(argv[2], NULL, 10) * 0x9e3779b97f4a7c15u + 1;
    int block, grid, unroll;
    if (ew_get_launch_config("add_f32", 1000, &block, &grid, &unroll) != EW_ERR_NO_DEVICE) {
        printf("a GPU is visible: fabricated addresses must not reach it\n");
        return 77;
    }
    for (long i = 0; i < calls; ++i) {
        switch (rnd() % 3) {
        case 0: call_f32(); break;
        case 1: call_f16(); break;
        default: call_bf16();
        }
    }
    printf("%ld calls, %d failures; OK %ld, INVALID_ARG %ld, MISALIGNED %ld, OVERLAP %ld, "
           "NO_DEVICE %ld\n",
           calls, failures, counts[0], counts[1], counts[2], counts[3], counts[4]);
    return failures ? 1 : 0;
}
