// rope_pages_host.cpp -- the C ABI entry points of include/rope_step.h for the pages of
// the cache: argument checks and the launches.  No CUDA call is made for a rejected
// call.
#include <initializer_list>

#include "rope_check.h"
#include "rope_pages.h"

namespace rope {
namespace {

constexpr int64_t kInt = (int64_t(1) << 31) - 1;

struct Range {
    const void* p;
    int64_t n;
};

// What both calls take; fills the sizes of `a`.
rope_status_t check_pages(PagesArgs* a, int64_t R, int64_t max_pages, int64_t stride, int64_t capacity,
                          int64_t page_size) {
    if (R < 0 || R >= (1 << 24)) return fail(ROPE_ERR_INVALID, "R=%lld requests", (long long)R);
    if (page_size < 1 || page_size > kInt)
        return fail(ROPE_ERR_INVALID, "page_size=%lld must be positive", (long long)page_size);
    if (max_pages < 0 || max_pages > kInt / page_size)
        return fail(ROPE_ERR_INVALID, "%lld pages of %lld tokens a request exceed 2^31 rows", (long long)max_pages,
                    (long long)page_size);
    if (stride < 0 || (R > 1 && stride < max_pages) || stride > kMaxSize)
        return fail(ROPE_ERR_INVALID, "page_table_stride %lld is less than max_pages %lld", (long long)stride,
                    (long long)max_pages);
    if (capacity < 0 || capacity > kInt)
        return fail(ROPE_ERR_INVALID, "free_capacity=%lld must be >= 0 and below 2^31", (long long)capacity);
    a->table_stride = stride;
    a->R = static_cast<int32_t>(R);
    a->max_pages = static_cast<int32_t>(max_pages);
    a->max_len = static_cast<int32_t>(max_pages * page_size);
    a->capacity = static_cast<int32_t>(capacity);
    a->div_page = FastDiv::make(static_cast<uint32_t>(page_size));
    return ROPE_OK;
}

int64_t table_bytes(const PagesArgs& a) {
    return a.R && a.max_pages ? ((a.R - 1) * a.table_stride + a.max_pages) * 4 : 0;
}

// The first `writes` of the ranges share a byte with another.
bool meet(const Range* r, int writes, int n) {
    for (int i = 0; i < writes; ++i)
        for (int j = i + 1; j < n; ++j)
            if (r[i].p && r[j].p && r[i].n && r[j].n && overlaps(r[i].p, r[i].n, r[j].p, r[j].n)) return true;
    return false;
}

rope_status_t grow(int32_t* kv_len, const int32_t* n, int64_t R, int32_t* table, int64_t max_pages, int64_t stride,
                   const int32_t* free_pages, int64_t capacity, int32_t* free_count, int64_t page_size,
                   int32_t* q_start, int64_t* slots, int32_t* positions, int64_t T, int32_t* granted,
                   rope_stream_t stream) {
    clear_error();
    PagesArgs a{};
    const rope_status_t st = check_pages(&a, R, max_pages, stride, capacity, page_size);
    if (st != ROPE_OK) return st;
    if (T < 0 || T > kInt) return fail(ROPE_ERR_INVALID, "T=%lld tokens", (long long)T);
    if ((R && (!kv_len || !n)) || !free_count || !q_start || (T && !slots))
        return fail(ROPE_ERR_NULLPTR, "kv_len, n, free_count, q_start or slots is null");
    if ((R && max_pages && !table) || (capacity && !free_pages))
        return fail(ROPE_ERR_NULLPTR, "page_table or free_pages is null");
    for (const void* p : {static_cast<const void*>(kv_len), static_cast<const void*>(n), static_cast<const void*>(table),
                          static_cast<const void*>(free_pages), static_cast<const void*>(free_count),
                          static_cast<const void*>(q_start), static_cast<const void*>(positions),
                          static_cast<const void*>(granted)})
        if (!aligned(p, 4)) return fail(ROPE_ERR_INVALID, "pointers must be aligned to their elements");
    if (!aligned(slots, 8)) return fail(ROPE_ERR_INVALID, "slots must be aligned to its elements");
    const Range r[] = {{kv_len, R * 4}, {table, table_bytes(a)}, {free_count, 4}, {q_start, (R + 1) * 4},
                       {slots, T * 8}, {positions, T * 4}, {granted, R * 4}, {n, R * 4}, {free_pages, capacity * 4}};
    if (meet(r, 7, 9)) return fail(ROPE_ERR_INVALID, "what is written must not overlap anything else");
    a.kv_len = kv_len;
    a.n = n;
    a.table = table;
    a.free_pages = const_cast<int32_t*>(free_pages);
    a.free_count = free_count;
    a.q_start = q_start;
    a.slots = slots;
    a.positions = positions;
    a.granted = granted;
    a.T = T;
    const char* err = nullptr;
    return launch_grow(a, stream, &err) == ROPE_OK ? ROPE_OK : fail(ROPE_ERR_CUDA, "%s", err);
}

rope_status_t trim(int32_t* kv_len, const int32_t* new_len, int64_t R, int32_t* table, int64_t max_pages,
                   int64_t stride, int32_t* free_pages, int64_t capacity, int32_t* free_count, int64_t page_size,
                   rope_stream_t stream) {
    clear_error();
    PagesArgs a{};
    const rope_status_t st = check_pages(&a, R, max_pages, stride, capacity, page_size);
    if (st != ROPE_OK) return st;
    if (R == 0) return ROPE_OK;
    if (!kv_len || !new_len || !free_count) return fail(ROPE_ERR_NULLPTR, "kv_len, new_len or free_count is null");
    if ((max_pages && !table) || (capacity && !free_pages))
        return fail(ROPE_ERR_NULLPTR, "page_table or free_pages is null");
    for (const void* p : {static_cast<const void*>(kv_len), static_cast<const void*>(new_len),
                          static_cast<const void*>(table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_count)})
        if (!aligned(p, 4)) return fail(ROPE_ERR_INVALID, "pointers must be aligned to their elements");
    const Range r[] = {{kv_len, R * 4}, {table, table_bytes(a)}, {free_count, 4}, {free_pages, capacity * 4},
                       {new_len, R * 4}};
    if (meet(r, 4, 5)) return fail(ROPE_ERR_INVALID, "what is written must not overlap anything else");
    a.kv_len = kv_len;
    a.n = new_len;
    a.table = table;
    a.free_pages = free_pages;
    a.free_count = free_count;
    const char* err = nullptr;
    return launch_trim(a, stream, &err) == ROPE_OK ? ROPE_OK : fail(ROPE_ERR_CUDA, "%s", err);
}

}  // namespace
}  // namespace rope

extern "C" {

rope_status_t rope_partial_cache_grow(int32_t* kv_len, const int32_t* n, int64_t R,
                                      int32_t* page_table, int64_t max_pages,
                                      int64_t page_table_stride, const int32_t* free_pages,
                                      int64_t free_capacity, int32_t* free_count, int64_t page_size,
                                      int32_t* q_start, int64_t* slots, int32_t* positions,
                                      int64_t T, int32_t* granted, rope_stream_t stream) {
    return rope::grow(kv_len, n, R, page_table, max_pages, page_table_stride, free_pages, free_capacity, free_count,
                      page_size, q_start, slots, positions, T, granted, stream);
}

rope_status_t rope_partial_cache_trim(int32_t* kv_len, const int32_t* new_len, int64_t R,
                                      int32_t* page_table, int64_t max_pages,
                                      int64_t page_table_stride, int32_t* free_pages,
                                      int64_t free_capacity, int32_t* free_count, int64_t page_size,
                                      rope_stream_t stream) {
    return rope::trim(kv_len, new_len, R, page_table, max_pages, page_table_stride, free_pages, free_capacity,
                      free_count, page_size, stream);
}

}  // extern "C"
