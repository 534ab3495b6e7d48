// rope_error.h -- the error record behind rope_last_error_message(), shared
// by the library's host files.
#pragma once
#include "rope_partial.h"

namespace rope {

// Record a message for the calling thread and return `st`.
rope_status_t fail(rope_status_t st, const char* fmt, ...);

// Every entry point starts with no message.
void clear_error();

// Byte ranges [a, a + na) and [b, b + nb) share a byte.
bool overlaps(const void* a, int64_t na, const void* b, int64_t nb);

}  // namespace rope
