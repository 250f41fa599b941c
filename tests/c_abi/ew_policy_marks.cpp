// counted_tokens() (ew_policy_marks.h) byte by byte, under the sanitizer of
// undefined behaviour: a lane past the last token has skip 4 and more.
#include <cstdint>
#include <cstdio>

#include "ew_policy_marks.h"

int main()
{
    const uint32_t bytes[] = {0, 1, 2, 0x7f, 0x80, 0x81, 0xff};
    const uint32_t past[] = {4, 5, 7, 8, 31, 32, 1000, 0x7fffffffu, 0xffffffffu};
    int wrong = 0;
    for (uint32_t a : bytes)
        for (uint32_t b : bytes)
            for (uint32_t c : bytes)
                for (uint32_t d : bytes)
                    for (uint32_t skip = 0; skip < 4; ++skip) {
                        const uint32_t byte[] = {a, b, c, d};
                        uint32_t want = 0;
                        for (uint32_t j = skip; j < 4; ++j)
                            if (byte[j]) want |= 0x80u << 8 * j;
                        wrong += ew::counted_tokens(a | b << 8 | c << 16 | d << 24, skip) != want;
                    }
    for (uint32_t skip : past) wrong += ew::counted_tokens(0, skip) != 0;
    std::printf("%d wrong\n", wrong);
    return wrong != 0;
}
