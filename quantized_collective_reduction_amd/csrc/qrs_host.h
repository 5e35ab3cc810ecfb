// Shared by the host sources of the C ABI: status and message of a call, and
// the pointer checks. Not installed; callers use include/qrs.h.
#pragma once

#include <stdint.h>

#include "qrs.h"

namespace qrs {

// Records the message qrs_last_error returns to this thread, and returns s.
qrs_status fail(qrs_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Clears the message and returns QRS_OK.
qrs_status ok();

const char* last_error();

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

}  // namespace qrs
