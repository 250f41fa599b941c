/* ew_train_fuzz.c -- randomised calls of the entry points of the layer norm, the
 * policy loss and the movement of rows to experts with fabricated device
 * addresses, for a library whose host code is built with sanitizers.  With no GPU visible every call that passes validation ends
 * with EW_ERR_NO_DEVICE, so nothing is launched; a workspace function must
 * not depend on anything but its sizes.
 *
 *   ew_train_fuzz CALLS SEED
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
#define S(cols) stride_value(cols)
#define ONE_TYPE(E, X)                                                                            \
    static void call_##X(void)                                                                    \
    {                                                                                             \
        const size_t rows = size_value(), cols = size_value();                                    \
        const size_t top = rnd() % 4 ? 1 + rnd() % 66 : size_value();                             \
        const size_t places = size_value(), experts = rnd() % 4 ? rnd() % 1100 : size_value();    \
        const size_t ws = rnd() % 4 ? (size_t)1 << 40 : size_value();                             \
        const int pads = rnd() % 3 != 0;                                                          \
        switch (rnd() % 5) {                                                                      \
        case 0:                                                                                   \
            note(ew_layernorm_##X(P(1), S(cols), P(2), P(3), P(4), S(cols), P(5), S(cols), P(6),  \
                                  S(cols), P(7), P(8), rows, cols, scalar(), NULL));              \
            break;                                                                                \
        case 1:                                                                                   \
            note(ew_layernorm_grad_##X(P(1), S(cols), P(2), S(cols), P(3), P(4), P(5), P(6),      \
                                       S(cols), P(7), S(cols), P(8), P(9), P(10), ws, rows, cols, \
                                       NULL));                                                    \
            break;                                                                                \
        case 2:                                                                                   \
            note(ew_experts_gather_##X(P(1), S(cols), P(2), top, pads ? P(3) : NULL,              \
                                       pads ? P(4) : NULL, experts, P(5), S(cols), places, rows,  \
                                       cols, NULL));                                              \
            break;                                                                                \
        case 3:                                                                                   \
            note(ew_experts_combine_##X(P(1), S(cols), places, P(2), top, P(3), P(4), S(cols),    \
                                        P(5), S(cols), rows, cols, NULL));                        \
            break;                                                                                \
        default:                                                                                  \
            note(ew_experts_combine_grad_##X(P(1), S(cols), P(2), S(cols), places, P(3), top,     \
                                             P(4), pads ? P(5) : NULL, pads ? P(6) : NULL,        \
                                             experts, P(7), S(cols), P(8), rows, cols, NULL));    \
        }                                                                                         \
    }

ONE_TYPE(float, f32)
ONE_TYPE(uint16_t, f16)
ONE_TYPE(uint16_t, bf16)

static void call_others(void)
{
    const size_t rows = size_value(), cols = size_value(), align = size_value();
    const size_t experts = rnd() % 4 ? rnd() % 1100 : size_value();
    const size_t ws = rnd() % 4 ? (size_t)1 << 40 : size_value();
    const size_t each = rnd() % 2 ? 0 : S(cols);
    switch (rnd() % 3) {
    case 0:
        note(ew_policy_loss_f32(P(1), S(cols), P(2), S(cols), P(3), S(cols), P(4), each, P(5),
                                S(cols), P(6), P(7), P(8), scalar(), scalar(), scalar(), scalar(),
                                (int)(rnd() % 5) - 1, P(9), ws, rows, cols, NULL));
        break;
    case 1:
        note(ew_policy_loss_grad_f32(P(1), S(cols), P(2), S(cols), P(3), S(cols), P(4), each, P(5),
                                     S(cols), P(6), P(7), P(8), S(cols), scalar(), scalar(),
                                     scalar(), rows, cols, NULL));
        break;
    default:
        note(ew_experts_sort(P(1), rows, experts, rnd() % 2 ? 1 + rnd() % 1024 : align, P(2), P(3),
                             P(4), P(5), P(6), ws, NULL));
    }
    if (ew_layernorm_grad_workspace(rows, cols) % 16 || ew_policy_loss_workspace(rows, cols) % 16 ||
        ew_experts_sort_workspace(rows, experts) % 16)
        ++failures;
    const size_t places = ew_experts_rows(rows, experts, align);
    if (places != SIZE_MAX && (places < rows || places % align || places >= (size_t)1 << 31))
        ++failures;
}

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
        switch (rnd() % 5) {
        case 0: call_f32(); break;
        case 1: call_f16(); break;
        case 2: call_bf16(); break;
        default: call_others();
        }
    }
    printf("%ld calls, %d failures; OK %ld, INVALID_ARG %ld, MISALIGNED %ld, OVERLAP %ld, "
           "NO_DEVICE %ld\n",
           calls, failures, counts[0], counts[1], counts[2], counts[3], counts[4]);
    return failures ? 1 : 0;
}
