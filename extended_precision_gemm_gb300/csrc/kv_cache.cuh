// kv_cache.cuh -- the paged 4-bit key/value cache as the kernels see it.
//
// A row is what one token has of one head, keys or values: `width` codes (the head
// dimension filled up to 64, 128 or 256 with zeros), width / block scale bytes and
// an exponent byte.  Rows lie in the order (page, k or v, head, token of the page).
// A value is
//   mxfp4: code * 2^(byte - 127); the exponent is the row's largest byte - 127;
//   nvfp4: code * E4M3(byte) * 2^exponent.
#pragma once

#include <cstdint>

#include "launch.cuh"
#include "mx4.cuh"

namespace ddg {

inline int cache_width(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

#ifdef __CUDACC__

// Row number of token `offset` of a page.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int64_t page, int kv, int head, int offset) {
    return ((page * 2 + kv) * c.heads + head) * (int64_t)c.page_size + offset;
}

// The page of a sequence's token, -1 where the table has none in the cache.
__device__ __forceinline__ int page_of(const CacheView& c, const BatchView& b, int sequence, int position) {
    const int i = position >> c.page_shift;
    if (position < 0 || i >= b.table_pages) return -1;
    const int p = b.table[(int64_t)sequence * b.ld_table + i];
    return p >= 0 && p < c.pages ? p : -1;
}

// A sequence's tokens; any negative number as -1, so that no position behind it overflows.
__device__ __forceinline__ int length_of(const BatchView& b, int sequence) { return max(b.lengths[sequence], -1); }

// What a call's token is: its sequence (-1 for a token of none), position, and page (-1
// where it has none in the cache).
struct Place {
    int sequence, position, page;
};
// `starts`: those of the batch, here or in shared memory.
__device__ __forceinline__ Place place_of(const CacheView& c, const BatchView& b, const int32_t* starts, int64_t t) {
    int low = 0, high = b.batch;  // the number of sequences that end at or before t is in [low, high]
    while (low < high) {
        const int mid = (low + high) / 2;
        if (starts[mid + 1] <= t) low = mid + 1;
        else high = mid;
    }
    if (low >= b.batch || starts[low] > t) return {-1, -1, -1};
    const int position = length_of(b, low) - (starts[low + 1] - (int)t);
    return {low, position, page_of(c, b, low, position)};
}

#endif  // __CUDACC__

}  // namespace ddg
