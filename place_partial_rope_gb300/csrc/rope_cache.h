// rope_cache.h -- what the host hands to the kernels that write and read the
// paged cache.  Not part of the public ABI.
#pragma once
#include <stdint.h>

#include "fast_div.h"
#include "rope_serving.h"

namespace rope {

constexpr int kCacheThreads = 128;

// The keys or the values of a call: dense rows (token, head) on one side,
// cache rows (page, token of the page, head) and their scales on the other.
struct CacheSide {
    char* rows;                          // dense, bytes
    int64_t row_tok, row_head;           // bytes
    char* codes;                         // cache, bytes
    int64_t page, tok, head;             // bytes
    float* scale;                        // null for a 16-bit cache
    int64_t s_page, s_tok, s_head;       // elements
    int32_t dim;
};

struct CacheArgs {
    CacheSide side[2];    // keys, values
    const int64_t* slots;
    const char* cos;      // rows of the rotation (write only; null: none)
    const char* sin;
    int64_t cos_tok, sin_tok;  // bytes
    int64_t page_size;
    uint64_t total;       // pages * page_size
    FastDiv div_rows;     // rows of one token: heads, or 2 * heads with values
    FastDiv div_page;     // used when total < 2^32
    uint32_t rows;        // rows of this launch
    int32_t heads;
    int32_t first;        // the side that the first `heads` rows of a token are
    int32_t start, half;  // slice start and half its length
    bool half_mode;
};

struct CachePlan {
    int dtype;      // rope_dtype_t of the dense rows
    int store;      // rope_cache_dtype_t
    int vec;        // elements per access: 16 (reading codes), 8 or 1
    int lanes;      // lanes per row, a power of two <= 32
    int chunks;     // accesses per lane
    bool turn;      // the rotation's partner and cos/sin come as whole accesses
};

rope_status_t launch_cache_write(const CachePlan& plan, const CacheArgs& args, rope_stream_t stream,
                                 const char** err);
rope_status_t launch_cache_read(const CachePlan& plan, const CacheArgs& args, rope_stream_t stream,
                                const char** err);

}  // namespace rope
