// attend.cuh -- what the kernels of attention over the 4-bit cache share: which
// tokens a query sees, and the partial results of work split over a long cache.
//
// o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m) over the tokens j that a query sees,
// with s_j = scale log2(e) q.k_j.  A cache row's value is its codes and block scales
// (exact in 16-bit floating point) times 2^r, r the row's exponent: it joins s_j as
// a factor for keys, and for values the weight is 2^((s_j - m) + (r_j - R)) with a
// reference R of its own, so rows of any size meet in range; R is relative to m, as a
// sum of both would lose it where scores are 2^24 and more.  A part of the sum is
// (m, R, l, o): l = sum 2^(s - m), o = sum 2^((s - m) + (r - R)) (codes times scales).
#pragma once

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "kv_cache.cuh"

namespace ddg {

struct CutItem;
// A launch of the kernels below.
struct AttendArgs {
    CacheView c;
    BatchView b;
    const void* q;
    void* out;
    int64_t qt, qh, ot, oh;  // strides of tokens and heads
    int heads, group;        // of queries; queries a key/value head
    int window, sinks;       // window 0: none
    float scale;             // log2(e) times the scale of scores
    bool vec_q, vec_out;
    int64_t above, upto;  // sequences of so many rows (tokens times queries a key/value head) are taken, the others left out
    int step;             // 0, or see first_tile
    int splits;    // attend_tile.cu: most parts of a row; attend.cu: CTAs, or (together) CTAs of a cluster
    bool together;
    float4* part;  // (m, R, l, 1 if any token is seen) of a part: by split and row (token, query head), or by CTA (attend.cu)
    float* sums;   // its o, `width` elements
    CutItem* cuts;  // attend.cu: one for each CTA

    __host__ __device__ bool takes(int64_t tokens) const { return tokens * group > above && tokens * group <= upto; }
    // The number of the first tile of `columns` rows of sequence i, which starts at token `start`.  Its rows' own tiles
    // have one more at most than start's difference gives: each sequence has a number more for it or, where only those
    // of more than `above` rows are taken and the others are the most, every `step` tokens have, the fewest of such a
    // sequence.  Numbers that are left over are of no tile.
    __host__ __device__ int64_t first_tile(int i, int start, int columns) const {
        return (int64_t)start * group / columns + (step > 0 ? (unsigned)start / (unsigned)step : i);
    }
    int64_t tiles(int columns) const { return first_tile((int)b.batch, (int)b.tokens, columns); }
};

#ifdef __CUDACC__

namespace {

__device__ __forceinline__ float minus_infinity() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ float not_a_number() { return __uint_as_float(0x7fc00000u); }

// 2^x by one instruction (2^-22; 0 below 2^-126).
__device__ __forceinline__ float power2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_of(float a, float b) {  // a in the low half
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A reference that may be minus infinity (nothing seen yet) as a number to subtract.
__device__ __forceinline__ float reference(float m) { return m == minus_infinity() ? 0.0f : m; }

// Query tokens [first, last] of a sequence, at positions p0 .. p1: the groups of 16
// tokens that any of them sees, those of the sinks and then those from `low` on.
struct Groups {
    int sink, low, count;
};
// Beyond the page table the list goes on as far only as makes every query that lies there see a token without a page:
// to the first group that the table does not reach, and with a window so far that each of an item's queries (of up to
// 256 positions in a row) has the begin of its own window in the list: p - window is less than 16 low + 271.
__device__ __forceinline__ Groups groups_of(const CacheView& c, const BatchView& b, int p0, int p1, int window, int sinks) {
    Groups g{0, 0, 0};
    if (p1 < 0) return g;
    int64_t most = (int64_t)b.table_pages * c.page_size / 16 + 1;
    if (window > 0) {
        if (p0 >= window) g.low = (p0 - window + 1) / 16;
        g.sink = min((int)(((unsigned)min(sinks, p1 + 1) + 15u) / 16u), g.low);
        most = max(most, (int64_t)g.low + 17);
    }
    g.count = g.sink + (int)min((int64_t)p1 / 16 + 1, most) - g.low;
    return g;
}
// Parts of tiles of 128 tokens that an item is cut into (attend_tile.cu): of four tiles at least.
__device__ __forceinline__ int parts_of(int tiles, int most) { return max(1, min(most, (tiles + 3) / 4)); }
__device__ __forceinline__ int group_token(const Groups& g, int i) { return (i < g.sink ? i : i - g.sink + g.low) * 16; }

__device__ __forceinline__ bool sees(int p, int j, int window, int sinks) {
    return j <= p && (window == 0 || j > p - window || j < sinks);
}

// Work items are tiles of `columns` (query token, head of the group) pairs of one
// sequence and key/value head, numbered by first_tile.
struct Item {
    int sequence, column, columns, first_token, tokens, length;
};
// The last sequence b with first(b) <= t, found by a whole warp, where first does not
// fall; -1 if there is none.
template <class F>
__device__ __forceinline__ int search(const BatchView& b, int64_t t, F first) {
    const int lane = threadIdx.x & 31;
    int low = 0, high = b.batch;  // the answer is in [low, high)
    bool none = b.batch <= 0;
    while (!none && (high - low > 1 || low == 0)) {
        const int stride = (high - low + 31) / 32;
        const int i = low + lane * stride;
        const bool at = i < high && first(i) <= t;
        const int n = __popc(__ballot_sync(~0u, at));
        none = n == 0;
        low += none ? 0 : (n - 1) * stride;
        high = min(high, low + stride);
        if (stride == 1) break;
    }
    return none ? -1 : low;
}
// Tile t's part of the batch.
__device__ __forceinline__ Item item_of(const AttendArgs& a, int64_t t, int columns) {
    const Item nothing{-1, 0, 0, 0, 0, 0};
    const BatchView& b = a.b;
    const int s = search(b, t, [&](int i) { return a.first_tile(i, b.starts[i], columns); });
    if (s < 0) return nothing;
    const int64_t s0 = b.starts[s], s1 = b.starts[s + 1];
    const int64_t column = (t - a.first_tile(s, (int)s0, columns)) * columns;
    if (s0 < 0 || s1 > b.tokens || !a.takes(s1 - s0) || column < 0 || column >= (s1 - s0) * a.group) return nothing;
    return Item{s, (int)column, (int)min((int64_t)columns, (s1 - s0) * a.group - column), (int)s0, (int)(s1 - s0), length_of(b, s)};
}

// A part's R as one of the reference m (its own is m_of_part, and m is no less).
__device__ __forceinline__ float relative(float R, float m_of_part, float m) { return R + (m_of_part - reference(m)); }
// (m, R) becomes that of two parts: where every weight has its place in range.
__device__ __forceinline__ void join_references(float& m, float& R, float other_m, float other_R) {
    const float top = fmaxf(m, other_m);
    R = fmaxf(relative(R, m, top), relative(other_R, other_m, top));
    m = top;
}

// How a row's sums become its output: times x twice (half of the exponent each),
// over l; 0 where no token is seen.
struct Finish {
    float x, inverse;
};
__device__ __forceinline__ Finish finish_of(float R, float l, float lift, bool any) {
    if (!any) return Finish{0.0f, 0.0f};
    return Finish{power2(0.5f * (reference(R) - lift)), 1.0f / l};
}
// Elements d .. d + 3 of an output row.
template <typename T>
__device__ __forceinline__ void store4(T* out, int d, int dim, bool vec, const Finish& z, const float (&y)[4]) {
    T t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = from_float<T>(z.inverse == 0.0f && z.x == 0.0f ? 0.0f : y[i] * z.x * z.x * z.inverse);
    if (vec && d + 4 <= dim) {
        uint2 w;
        memcpy(&w, t, 8);
        *reinterpret_cast<uint2*>(out + d) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d + i < dim) out[d + i] = t[i];
    }
}

}  // namespace

#endif  // __CUDACC__

cudaError_t launch_attend_columns(const AttendArgs& a, int type, cudaStream_t st);
// Sets `together` and `splits` for that launch; rows of its workspace unless together: (part, sums) of two cut items of
// each CTA.
void plan_attend_columns(AttendArgs& a, int type);
inline int64_t attend_columns_rows(int ctas) { return 2LL * 8 * ctas; }
// What a CTA says of the item that it begins and others end (0 columns: none): further CTAs, place of its columns,
// the position of its sequence's first query.
struct CutItem {
    int columns, others, first_token, column, head, before;
};
// The same for many queries, by tiles of 128 rows on the tensor cores.
cudaError_t launch_attend_tile(const AttendArgs& a, int type, cudaStream_t st);
int attend_tile_parts(const AttendArgs& a);
// The outputs from the parts of each row; lift: the exponent by which the sums are too
// large.
cudaError_t launch_attend_join(const AttendArgs& a, int type, float lift, cudaStream_t st);

}  // namespace ddg
