// rope_pages.h -- what the host hands to the kernels that deal out pages of the cache
// and take them back.  Not part of the public ABI.
#pragma once
#include <stdint.h>

#include "fast_div.h"
#include "rope_step.h"

namespace rope {

struct PagesArgs {
    int32_t* kv_len;
    const int32_t* n;  // grow: new tokens; trim: lengths that are kept
    int32_t* table;
    int64_t table_stride;
    int32_t* free_pages;  // grow: only read
    int32_t* free_count;
    int32_t* q_start;
    int64_t* slots;
    int32_t* positions;  // or null
    int32_t* granted;    // or null
    int64_t T;
    int32_t R, max_pages, max_len, capacity;
    FastDiv div_page;
};

rope_status_t launch_grow(const PagesArgs& args, rope_stream_t stream, const char** err);
rope_status_t launch_trim(const PagesArgs& args, rope_stream_t stream, const char** err);

}  // namespace rope
