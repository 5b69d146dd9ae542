// Host-side helpers that the library's translation units share (definitions in gdn_api.cu).
#pragma once

#include <cstdint>

#include "gdn.h"

namespace gdn {

// Bit of the device error word: a block-table entry or a sequence length outside the paged cache.
constexpr unsigned kErrPages = 4u;

// Records a printf-style message as the calling thread's last error and returns `st`.
gdn_status fail(gdn_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Forgets the calling thread's last error (every entry point does so first).
void clear_error();

// Device address of the current device's error word; nullptr with *st set when the look-up fails.
unsigned* err_word_ptr(gdn_status* st);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace gdn
