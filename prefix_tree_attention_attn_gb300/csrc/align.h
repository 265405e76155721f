// Checks of addresses at the C entries.
#pragma once

#include <cstdint>

namespace treeattn {

// Whether an address is a multiple of a power of two.
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace treeattn
