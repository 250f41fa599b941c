// ew_policy_marks.h -- which of four neighbouring tokens count, from their mask's
// bytes (ew_policy.hip; its test compiles it for the host).  Not installed; not
// part of the C ABI.
#pragma once

#include <stdint.h>

namespace ew {

// Bit 8 j + 7: byte j of mark is not 0 and j >= skip.  A lane without tokens has
// mark 0, and skip may then be any number; else it is below 4.
constexpr uint32_t counted_tokens(uint32_t mark, uint32_t skip)
{
    if (mark == 0) return 0;
    const uint32_t counted = (((mark & 0x7f7f7f7fu) + 0x7f7f7f7fu) | mark) & 0x80808080u;
    return counted >> 8 * skip << 8 * skip;
}

}  // namespace ew
