// Index arithmetic of the suffix and decode operators: tiles of packed sequences, places in a
// paged cache.  Plain functions of integers, so that host code can include and test them.
#pragma once
#include <stdint.h>

#ifdef __HIP__
#define GDN_HD __host__ __device__ inline __attribute__((always_inline))
#else
#define GDN_HD static inline
#endif

namespace gdn {

// Packed sequences are cut into tiles of `tile` rows each (`mul` rows per token).  Sequence n
// owns the tile indices from first_tile(n) = floor(cu[n] mul / tile) + n, which leaves every
// sequence, an empty one too, at least ceil(rows / tile) and at least one index; their number
// is known on the host as floor(T mul / tile) + n_seqs without reading cu.
GDN_HD int64_t first_tile(int32_t at, int n, int mul, int tile) { return (int64_t)at * mul / tile + n; }

// Whether [b, e) is a range of the packed tokens.
GDN_HD bool range_ok(int32_t b, int32_t e, int64_t total) { return b >= 0 && e >= b && e <= total; }

// Whether a sequence may have kv cached tokens.
GDN_HD bool kv_ok(int32_t kv, int32_t max_kv, int32_t page_size, int32_t max_pages) {
    return kv >= 0 && kv <= max_kv && ((int64_t)kv + page_size - 1) / page_size <= max_pages;
}

// Element offset of a page's token in the caches (head 0), or -1 with `bad` set for no page.
GDN_HD int64_t page_offset(int32_t page, int32_t token, int32_t n_pages, int64_t page_stride, int64_t token_stride, bool &bad) {
    if (page < 0 || page >= n_pages) {
        bad = true;
        return -1;
    }
    return (int64_t)page * page_stride + (int64_t)token * token_stride;
}
// The same for cached token j of a sequence.  j is in [0, kv) of a kv that passed kv_ok, so the
// block table is read in bounds.
GDN_HD int64_t cache_offset(const int32_t *table, int32_t j, int32_t page_size, int32_t n_pages, int64_t page_stride,
                            int64_t token_stride, bool &bad) {
    return page_offset(table[j / page_size], j % page_size, n_pages, page_stride, token_stride, bad);
}

}  // namespace gdn
