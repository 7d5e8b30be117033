// Launchers of the 16-bit operators (layer norm, rotary positions, linear).
// The entry points beside them validate; these only launch.
#pragma once

#include "svdq_internal.h"

namespace svdq {

// Rotary frequencies as fractions of a turn (times 2^64) and each pair's
// axis; passed to the kernel by value.
struct RopeTurns {
  uint64_t turn[SVDQ_ROPE_MAX_PAIRS];
  uint8_t axis[SVDQ_ROPE_MAX_PAIRS];
  int pairs, axes;
};

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of `ld` elements of `esize` bytes start on 16-byte boundaries.
inline bool rows_aligned16(const void* p, int ld, int esize) {
  return is_aligned16(p) && ((long long)ld * esize) % 16 == 0;
}

inline int dtype_size(int dtype) { return dtype == SVDQ_DTYPE_F32 ? 4 : 2; }

}  // namespace svdq
