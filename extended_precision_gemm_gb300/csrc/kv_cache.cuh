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

// What a call's token is: its sequence and position, -1 for a token of none.
struct Place {
    int sequence;
    int position;
};

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

// The sequence of token t, found by a whole block: the number of sequences that
// end at or before t.
__device__ __forceinline__ Place place_of(const BatchView& b, int64_t t) {
    int count = 0;
    for (int i = 0; i < b.batch; i += blockDim.x) {
        const int s = i + (int)threadIdx.x;
        count += __syncthreads_count(s < b.batch && b.starts[s + 1] <= t);
    }
    if (count >= b.batch || b.starts[count] > t) return {-1, -1};
    return {count, b.lengths[count] - (b.starts[count + 1] - (int)t)};
}

#endif  // __CUDACC__

}  // namespace ddg
