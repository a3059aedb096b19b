// 16-byte accesses at the elements' own alignment (gfx950 allows them in global
// memory), for rows that may start anywhere.
#pragma once

#include "../gdr_device.h"

namespace gdr {

template <typename TIO> struct Wide;
template <> struct Wide<bf16> { typedef u32x4 __attribute__((aligned(2))) T; };
template <> struct Wide<float> { typedef u32x4 __attribute__((aligned(4))) T; };

}  // namespace gdr
