// Grid of the kernels that walk over rows of one alignment class (host only).
#pragma once

#include <cstdint>

namespace ddp {

// CTAs for `need` pieces of work of which a CTA takes every grid-th: a multiple of 8 where it takes more than one, so
// that the rows it takes lie alike on a grid of up to 8 elements, whatever their pitch.  From a wave's CTAs upwards: a
// part of a GPU may hold fewer than 8.
inline int alike_grid(int wave, int64_t need) {
    const int64_t up = (static_cast<int64_t>(wave) + 7) / 8 * 8;
    return static_cast<int>(up < need ? up : need);
}

}  // namespace ddp
