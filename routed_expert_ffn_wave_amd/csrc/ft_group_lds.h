// LDS of a group list (ft_groups.h), for the kernels and for the host code that chooses among them.
#pragma once
#include <stddef.h>

namespace ftk {

// LDS bytes of a group list for E experts: slot, row0, cnt and item0 arrays of E + 2 ints each, and
// a few ints of scratch, rounded up to 16 bytes.
constexpr size_t group_lds_bytes(int E) { return (((size_t)4 * (E + 2) + 4) * 4 + 15) & ~(size_t)15; }

}  // namespace ftk
