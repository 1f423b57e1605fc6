// attend.cu -- attention over the 4-bit cache for few queries, and the sum of parts.
//
// Few queries of a key/value head (a token's group of heads, a few proposed tokens)
// read the whole cache: the floor is its bytes.  A warp takes 32 tokens a round, two
// groups of 16 that are independent of each other, copied to its own part of shared
// memory one or two rounds ahead (cp.async; no block waits for another warp), and makes
// mma.sync fragments of them: scores as S^T = K Q^T (16 tokens by 8 queries), the sum as
// O^T = V^T P^T, so that 8 queries fill an instruction that 16 rows of queries would
// leave half empty, and the codes of a row are contiguous in a thread.  (tcgen05 wants
// its operands in shared memory and 128 rows: each 4-bit row would be written there in
// 16 bits and read again, four times its bytes, for a product that uses 8 of the
// columns.)
//
// All groups of all (8 columns, key/value head) items in a row are cut into equal runs, one
// for each CTA that the SMs hold: lengths may differ as they like.  An item that a run's
// end cuts leaves parts, which join_cut_kernel adds.
//
// Measured (bfloat16): 64 sequences of 100 to 8192 tokens, 8 heads of 128, 8 queries each,
// mxfp4: 103 us for 291 MB (2.8 TB/s); one of 131071, nvfp4: 48 us for 153 MB, 41 of them
// here.  Bound by issue and the latency of its own instructions: a group takes 370
// instructions, of which 140 run at half rate (conversions of codes, products with
// scales, movmatrix), by 12 warps an SM (161 registers).  A fourth CTA costs more
// instructions than its warps give, whole rows of codes at a time and 16 tokens a round
// took 53 us where this form took 47.
//
// The codes become 16-bit floating point by one conversion for two, the block's
// scale one packed multiplication for two, exactly: E4M3 times E2M1 has 6 bits;
// mxfp4 scales are relative to the row's largest, times 2^13, exact down to a block 2^36
// below it and 0 from 2^38 on: what a channel of its own may show, for an output's elements
// sum one block of each token.  Queries are scaled by a power of two into the range of 16
// bits; what they lose is 2^-36 of their row's largest.  Weights are rounded to 16 bits
// (11 significant) for bfloat16 outputs, and what that leaves enters the sum too for
// float16 ones, whose own rounding is as small.  (22 bits for bfloat16 too: 108 and 51 us
// for 103 and 48, and the error against 64 bits the same 0.0017, the output's rounding.)
#include <algorithm>
#include <atomic>

#include "async_copy.cuh"
#include "attend.cuh"

namespace ddg {
namespace {

constexpr int kWarps = 4;
constexpr float kLag = 8.0f;    // references follow when they are exceeded by more than 2^8
constexpr float kLift = 7.0f;   // weights are up to 2^(8 + 7), below the largest float16
constexpr int kMxLift = 13;     // mxfp4 scales relative to the row's largest, times 2^13

__device__ __forceinline__ float low_half(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float high_half(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
// Byte i of w, two codes, as two halves.
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
    uint32_t h;
    if constexpr (I == 0) asm("{.reg .b8 t0, t1, t2, t3; mov.b32 {t0, t1, t2, t3}, %1; cvt.rn.f16x2.e2m1x2 %0, t0;}" : "=r"(h) : "r"(w));
    if constexpr (I == 1) asm("{.reg .b8 t0, t1, t2, t3; mov.b32 {t0, t1, t2, t3}, %1; cvt.rn.f16x2.e2m1x2 %0, t1;}" : "=r"(h) : "r"(w));
    if constexpr (I == 2) asm("{.reg .b8 t0, t1, t2, t3; mov.b32 {t0, t1, t2, t3}, %1; cvt.rn.f16x2.e2m1x2 %0, t2;}" : "=r"(h) : "r"(w));
    if constexpr (I == 3) asm("{.reg .b8 t0, t1, t2, t3; mov.b32 {t0, t1, t2, t3}, %1; cvt.rn.f16x2.e2m1x2 %0, t3;}" : "=r"(h) : "r"(w));
    return h;
}

__device__ __forceinline__ bool half_is_nan(uint32_t h) { return (h & 0x7fffu) > 0x7c00u; }

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int N, int I = 0, class F>
__device__ __forceinline__ void static_for(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        static_for<N, I + 1>(f);
    }
}

template <int N>  // N words of shared memory, aligned to their size up to 16 bytes
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    }
}
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void close_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A group of 16 tokens on its way: a warp copies it to shared memory one or two rounds
// ahead, and a lane (r, c) = (lane / 4, lane % 4) reads of keys a quarter c of tokens r
// and r + 8, of values the eighth r of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9.  Two
// tokens' values are followed by 32 bytes of nothing: their readers are on different
// banks then.
template <int WIDTH, int FMT>
struct Stage {
    static constexpr int KW = WIDTH / 32, VW = WIDTH / 64;                 // words of codes of a token
    static constexpr int BLOCK = mx4_block(FMT), BLOCKS = WIDTH / BLOCK;
    static constexpr int KB = WIDTH / 4 / BLOCK > 0 ? WIDTH / 4 / BLOCK : 1;  // blocks a lane's codes touch
    static constexpr int VB = WIDTH / 8 / BLOCK > 0 ? WIDTH / 8 / BLOCK : 1;
    static constexpr int ROW = WIDTH / 2;                                  // bytes of codes
    static constexpr int V0 = 16 * ROW, S0 = V0 + 16 * ROW + 8 * 32;       // values' codes, scales of keys and values
    static constexpr int E0 = S0 + 32 * BLOCKS, BYTES = E0 + 32;           // exponents of keys and values
    static constexpr int PIECES = 2 * BLOCKS + 2;                          // of scales and exponents, 16 bytes each
    static constexpr int STAGES = WIDTH == 256 ? 2 : 3;                    // of two groups, which a round takes together

    // The lane's places in the first group of 16 rows of the cache.
    struct Base {
        const uint8_t *k, *v, *small[(PIECES + 31) / 32];
        uint32_t small_stride[(PIECES + 31) / 32];  // of a group of rows
    };
    static __device__ __forceinline__ Base base_of(const CacheView& c, int lane) {
        Base b;
        const int64_t values = (int64_t)c.heads * (c.page_size / 16);  // from a key to its value, in groups of 16 rows
        b.k = c.codes + lane * 16;
        b.v = b.k + values * (16 * ROW);
#pragma unroll
        for (int i = 0; i < (PIECES + 31) / 32; ++i) {
            const int piece = lane + 32 * i;
            const bool exponent = piece >= 2 * BLOCKS;
            const int kv = exponent ? piece - 2 * BLOCKS : piece / BLOCKS;
            b.small_stride[i] = exponent ? 16 : 16 * BLOCKS;
            b.small[i] = (exponent ? reinterpret_cast<const uint8_t*>(c.exponents) : c.scales + piece % BLOCKS * 16) + (kv ? values * b.small_stride[i] : 0);
        }
        return b;
    }
    // row: of the group's keys, in 16s; negative: no page, nothing is copied.
    static __device__ __forceinline__ void copy(const Base& b, int row, uint32_t to, int lane) {
        if (row >= 0) {
            const uint8_t *k = b.k + (uint64_t)(uint32_t)row * (16 * ROW), *v = b.v + (uint64_t)(uint32_t)row * (16 * ROW);
#pragma unroll
            for (int i = 0; i < 16 * ROW / 512; ++i) {
                const int at = i * 512 + lane * 16;
                copy16(to + at, k + i * 512);
                copy16(to + V0 + at + at / (2 * ROW) * 32, v + i * 512);
            }
#pragma unroll
            for (int i = 0; i < (PIECES + 31) / 32; ++i)
                if (lane + 32 * i < PIECES) copy16(to + S0 + (lane + 32 * i) * 16, b.small[i] + (uint64_t)(uint32_t)row * b.small_stride[i]);
        }
    }
};

// The scale bytes of N blocks of a row with exponent e as halves, each in both halves
// of a word.
template <int FMT, int N>
__device__ __forceinline__ void half_scales(const uint8_t* bytes, int e, uint32_t (&h)[N]) {
#pragma unroll
    for (int b = 0; b < N; b += 2) {
        const uint32_t two = N == 1 ? bytes[0] : *reinterpret_cast<const uint16_t*>(bytes + b);
        if (FMT == kNvfp4) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)two));
            h[b] = __byte_perm(h2, h2, 0x1010);
            if (b + 1 < N) h[b + 1] = __byte_perm(h2, h2, 0x3232);
        } else {
            const auto half = [&](uint32_t byte) {
                // at most 2^kMxLift, which is what the row's own exponent gives its largest: bytes that do not belong
                // together, of rows that no token has, stay finite (their weight is 0, and 0 times infinity is NaN)
                const float power = exp2_int(min(max((int)byte - e - 127 + kMxLift, -30), kMxLift));
                return byte == 255u ? 0x7fff7fffu : half2_of(power, power);
            };
            h[b] = half(two & 0xffu);
            if (b + 1 < N) h[b + 1] = half(two >> 8);
        }
    }
}
__device__ __forceinline__ uint32_t both_low(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }

// ---- how the work is dealt out ----
//
// An item is a tile of 8 columns of a sequence with one key/value head; its cost is
// the number of its groups of 16 tokens (at least one).  The items of all sequences in
// turn, their groups one after the other, are cut into equal runs, one for each CTA,
// so that lengths do not matter.  An item that one CTA does as a whole is written by
// it; of a cut one each CTA leaves a part: the one that begins it in its second slot,
// the others in their first.
struct Cut {
    int64_t total;   // groups of all items
    int64_t ctas;    // that work: at least kLeast groups each
    __device__ __forceinline__ int64_t first(int64_t cta) const { return total * cta / ctas; }
    // the CTA that has group g
    __device__ __forceinline__ int64_t owner(int64_t g) const { return ((g + 1) * ctas - 1) / total; }
};
constexpr int kLeast = 8;
__device__ __forceinline__ Cut cut_of(int64_t total, int ctas) {
    return Cut{total, max((int64_t)1, min((int64_t)ctas, total / kLeast))};
}

struct Sequence {
    int first_token, tokens, length;
};
__device__ __forceinline__ Sequence sequence_at(const AttendArgs& a, int i) {
    const int s0 = a.b.starts[i], s1 = a.b.starts[i + 1];
    if (s0 < 0 || s1 > a.b.tokens || s1 <= s0 || !a.takes(s1 - s0)) return Sequence{0, 0, 0};
    return Sequence{s0, s1 - s0, length_of(a.b, i)};
}
// The groups of tile `ct` of 8 columns, and (with count at least 1) its cost.
__device__ __forceinline__ Groups tile_groups(const AttendArgs& a, const Sequence& s, int ct) {
    const int before = s.length - s.tokens;
    const int64_t last = min((int64_t)s.tokens * a.group, (int64_t)(ct + 1) * 8) - 1;
    Groups g = groups_of(a.c, a.b, before + (int)((int64_t)ct * 8 / a.group), before + (int)(last / a.group), a.window, a.sinks);
    g.count = max(g.count, 1);
    return g;
}
__device__ __forceinline__ int tiles_of(const AttendArgs& a, const Sequence& s) { return (int)(((int64_t)s.tokens * a.group + 7) / 8); }
__device__ __forceinline__ int64_t cost_of(const AttendArgs& a, const Sequence& s) {
    int64_t n = 0;
    for (int ct = 0; ct < tiles_of(a, s); ++ct) n += tile_groups(a, s, ct).count;
    return n;
}

__device__ __forceinline__ float read_cluster(uint32_t local, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(local, rank)) : "memory");
    return v;
}

// One CTA: its run of groups, item by item; of an item's groups the warps take pairs in
// turn.  TOGETHER: instead a cluster of a.splits CTAs for each item, each with its share
// of the groups, whose parts are summed through distributed shared memory; for short
// sequences, where the second launch would take as long as the first.
template <typename T, int WIDTH, int FMT, bool TOGETHER>
__global__ void __launch_bounds__(kWarps * 32, WIDTH == 256 ? 2 : WIDTH == 128 ? 3 : 4) attend_columns_kernel(const AttendArgs a) {
    using G = Stage<WIDTH, FMT>;
    constexpr int KS = WIDTH / 16;  // MMAs along the head
    constexpr bool REST = std::is_same_v<T, __half>;
    constexpr int ROW = WIDTH + 4;  // a column's sums in shared memory
    constexpr int kStages = G::STAGES, kAhead = kStages - 1;
    extern __shared__ __align__(16) uint8_t shared[];  // [warp][stage], and [warp][8][ROW] floats behind an item's last group
    float* const sums = reinterpret_cast<float*>(shared);
    __shared__ float s_m[kWarps][8], s_R[kWarps][8], s_l[kWarps][8];
    __shared__ int64_t scan[kWarps];
    __shared__ int64_t found_before;
    __shared__ int found;
    __shared__ Sequence found_sequence;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane / 4, c = lane % 4;

    int64_t total = 0, ctas = 0, run = 0, run_end = 0, start = 0;  // run: groups from the item's first on; start: of the sequence's
    int b, ct = 0, head, g0;
    Sequence seq;
    Groups groups;
    const uint32_t rank = TOGETHER ? blockIdx.y : 0;
    if constexpr (TOGETHER) {
        head = (int)(blockIdx.x % a.c.heads);
        const Item item = item_of(a, blockIdx.x / a.c.heads, 8);
        if (item.sequence < 0) return;  // the whole cluster
        b = item.sequence;
        ct = item.column / 8;
        seq = Sequence{item.first_token, item.tokens, item.length};
        groups = tile_groups(a, seq, ct);
        g0 = (int)((int64_t)groups.count * rank / a.splits);
        run_end = (int64_t)groups.count * (rank + 1) / a.splits - g0;
    } else {
        // the whole cost, and the sequence in which this CTA's run begins
        {
            const int per = (a.b.batch + kWarps * 32 - 1) / (kWarps * 32), b0 = min((int)threadIdx.x * per, a.b.batch), b1 = min(b0 + per, a.b.batch);
            int64_t mine = 0;
            Sequence own{0, 0, 0};
            for (int i = b0; i < b1; ++i) {
                own = sequence_at(a, i);
                mine += cost_of(a, own);
            }
            int64_t upto = mine;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int64_t v = __shfl_up_sync(~0u, upto, d);
                if (lane >= d) upto += v;
            }
            if (lane == 31) scan[warp] = upto;
            __syncthreads();
            int64_t before = upto - mine;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += scan[w];
                total += scan[w];
            }
            total *= a.c.heads;
            const Cut cut = cut_of(total, a.splits);
            ctas = cut.ctas;
            if (total == 0 || blockIdx.x >= ctas) {
                if (threadIdx.x == 0) a.cuts[blockIdx.x] = CutItem{0, 0, 0, 0, 0, 0};
                return;
            }
            run = cut.first(blockIdx.x);
            run_end = cut.first(blockIdx.x + 1);
            int64_t at = before * a.c.heads;
            for (int i = b0; i < b1; ++i) {
                if (per > 1) own = sequence_at(a, i);
                const int64_t cost = (per > 1 ? cost_of(a, own) : mine) * a.c.heads;
                if (run >= at && run < at + cost) {
                    found = i;
                    found_before = at;
                    found_sequence = own;
                }
                at += cost;
            }
            __syncthreads();
            b = found;
            start = found_before;
        }
        seq = found_sequence;
        groups = tile_groups(a, seq, 0);
        while (run >= start + (int64_t)groups.count * a.c.heads) {
            start += (int64_t)groups.count * a.c.heads;
            groups = tile_groups(a, seq, ++ct);
        }
        head = (int)((run - start) / groups.count);
        g0 = (int)((run - start) % groups.count);
    }
    const typename G::Base base = G::base_of(a.c, lane);
    uint32_t inside[G::KB];  // blocks of the lane's keys that begin beyond the head's end take no part, whatever they hold
#pragma unroll
    for (int d = 0; d < G::KB; ++d) inside[d] = (c * (WIDTH / 4) / G::BLOCK + d) * G::BLOCK < a.c.dim ? ~0u : 0u;
    constexpr float kSumLift = kLift + (FMT == kMxfp4 ? kMxLift : 0);

    while (true) {
        const int g1 = (int)min((int64_t)groups.count, g0 + (run_end - run));
        const int column0 = ct * 8, columns = (int)min((int64_t)8, (int64_t)seq.tokens * a.group - column0);
        const int before = seq.length - seq.tokens;  // the position of the first query token
        const int p0 = before + column0 / a.group, p1 = before + (column0 + columns - 1) / a.group;

        // the warp's groups are pair warp, warp + kWarps, ... of the run; rows of the keys of 16 pairs, a lane each
        const int pairs = (g1 - g0 + 1) / 2, mine = pairs > warp ? (pairs - warp + kWarps - 1) / kWarps : 0;
        int rows = -1;
        const auto rows_from = [&](int i) {
            const int g = g0 + 2 * (warp + (i + lane / 2) * kWarps) + lane % 2;
            rows = -1;
            if (g < g1) {
                const int token = group_token(groups, g), page = page_of(a.c, a.b, b, token);
                if (page >= 0) rows = (int)(cache_row(a.c, page, 0, head, token & (a.c.page_size - 1)) / 16);
            }
        };
        const uint32_t ring = smem_addr(shared) + warp * kStages * 2 * G::BYTES;
        uint32_t bad_groups = 0;  // two bits a round: the groups of the round at hand that have no page; the next rounds above
        const auto copy = [&](int i, uint32_t stage) {  // of round i, if there is one; a group of copies either way
            if (i % 16 == 0 && i < mine) rows_from(i);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = i < mine ? __shfl_sync(~0u, rows, i % 16 * 2 + k) : -1;
                bad_groups |= (uint32_t)(row < 0) << (2 * kAhead + k);
                G::copy(base, row, ring + stage + k * G::BYTES, lane);
            }
            close_copies();
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            copy(i, i * 2 * G::BYTES);
            bad_groups >>= 2;
        }
        // groups that every column sees as a whole: list numbers from whole0 to whole1 - 1
        const int whole0 = a.window > 0 && p1 >= a.window ? max(groups.sink, groups.sink + (p1 - a.window) / 16 + 1 - groups.low) : 0;
        const int whole1 = p0 < 0 ? 0 : groups.sink + (p0 + 1) / 16 - groups.low;

        // the queries: column r, elements c WIDTH / 4 .. of it
        uint32_t q[KS][2];
        float qf = a.scale;  // what a score is to be multiplied by
        {
            const bool have = r < columns;
            const int col = column0 + r;
            const T* src = static_cast<const T*>(a.q) + (int64_t)(seq.first_token + (have ? col / a.group : 0)) * a.qt +
                           (int64_t)(head * a.group + (have ? col % a.group : 0)) * a.qh;
            const int d0 = c * (WIDTH / 4);
            float x[WIDTH / 4];
            if (have && a.vec_q && d0 + WIDTH / 4 <= a.c.dim) {
#pragma unroll
                for (int i = 0; i < WIDTH / 4; i += 8) {
                    const uint4 raw = *reinterpret_cast<const uint4*>(src + d0 + i);
                    const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i + j] = to_float<T>(t[j]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < WIDTH / 4; ++i) x[i] = have && d0 + i < a.c.dim ? to_float<T>(src[d0 + i]) : 0.0f;
            }
            if (!REST) {  // bfloat16: the row's largest to [2^11, 2^12)
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < WIDTH / 4; ++i) {
                    const uint32_t bits = __float_as_uint(x[i]) & 0x7fffffffu;
                    most = max(most, bits < kInfBits ? bits : 0u);
                }
                most = max(most, __shfl_xor_sync(~0u, most, 1));
                most = max(most, __shfl_xor_sync(~0u, most, 2));
                const int e = max((int)(most >> 23) - 127 - 11, -126);
                const float2 up = exp2_factors(-e), down = exp2_factors(e);
#pragma unroll
                for (int i = 0; i < WIDTH / 4; ++i) x[i] = x[i] * up.x * up.y;
                qf = qf * down.x * down.y;
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                q[j][0] = half2_of(x[4 * j], x[4 * j + 1]);
                q[j][1] = half2_of(x[4 * j + 2], x[4 * j + 3]);
            }
            if (FMT == kMxfp4) qf *= exp2_int(-kMxLift);
        }
        // this lane's columns in the fragments are 2 c and 2 c + 1
        const float qf0 = __shfl_sync(~0u, qf, 8 * c), qf1 = __shfl_sync(~0u, qf, 8 * c + 4);
        const int pa = 2 * c < columns ? before + (column0 + 2 * c) / a.group : -1;
        const int pb = 2 * c + 1 < columns ? before + (column0 + 2 * c + 1) / a.group : -1;

        float o[KS][4];
#pragma unroll
        for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float ma = minus_infinity(), mb = ma, Ra = ma, Rb = ma, la = 0.0f, lb = 0.0f;
        float sub_ma = 0.0f, sub_mb = 0.0f, sub_Ra = -kLift, sub_Rb = -kLift;  // what is subtracted from scores and exponents

        uint32_t stage = 0;
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            wait_copies<kAhead - 1>();
            __syncwarp();
            const uint32_t bad = bad_groups & 3;
            const int group = g0 + 2 * (warp + i * kWarps);
            const bool whole = group >= whole0 && group + 1 < whole1 && group + 1 < g1 && bad == 0;
            const uint8_t* const at = shared + warp * kStages * 2 * G::BYTES + stage;
            // the stage of the round before is free: every lane has read it
            copy(i + kAhead, stage == 0 ? kAhead * 2 * G::BYTES : stage - 2 * G::BYTES);
            bad_groups >>= 2;
            stage = stage == kAhead * 2 * G::BYTES ? 0 : stage + 2 * G::BYTES;

            // scores: of each group tokens r and r + 8 in rows r and r + 8
            float s[2][4], e[2][2];
            const auto score_group = [&](auto N) {
                constexpr int n = decltype(N)::value;
                const uint8_t* const from = at + n * G::BYTES;
                uint32_t k[2][G::KW], ks[2][G::KB];
                int ke[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    ke[t] = reinterpret_cast<const int8_t*>(from + G::E0)[r + 8 * t];
                    load_words<G::KW>(from + (r + 8 * t) * G::ROW + c * (G::ROW / 4), k[t]);
                    half_scales<FMT, G::KB>(from + G::S0 + (r + 8 * t) * G::BLOCKS + c * (WIDTH / 4) / G::BLOCK, ke[t], ks[t]);
#pragma unroll
                    for (int d = 0; d < G::KB; ++d) ks[t][d] &= inside[d];
                }
                float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // two chains of MMAs
                constexpr int PER = KS / G::KB;  // MMAs of a block of a lane's codes
                auto score_step = [&](auto J) {
                    constexpr int j = decltype(J)::value;
                    const uint32_t s0 = ks[0][j / PER], s1 = ks[1][j / PER];
                    constexpr int w = j / 2, lo = j % 2 * 2;
                    mma16816(j % 2 ? y : x, mul_half2(codes2<lo>(k[0][w]), s0), mul_half2(codes2<lo>(k[1][w]), s1),
                             mul_half2(codes2<lo + 1>(k[0][w]), s0), mul_half2(codes2<lo + 1>(k[1][w]), s1), q[j][0], q[j][1]);
                };
                static_for<KS>(score_step);
                // 2^-127 counts as 0: rows of zeros have it, and those below 2^-125
                const float k0 = __uint_as_float((uint32_t)(ke[0] + 127) << 23), k1 = __uint_as_float((uint32_t)(ke[1] + 127) << 23);
                s[n][0] = (x[0] + y[0]) * qf0 * k0;
                s[n][1] = (x[1] + y[1]) * qf1 * k0;
                s[n][2] = (x[2] + y[2]) * qf0 * k1;
                s[n][3] = (x[3] + y[3]) * qf1 * k1;
                e[n][0] = (float)reinterpret_cast<const int8_t*>(from + G::E0 + 16)[r];
                e[n][1] = (float)reinterpret_cast<const int8_t*>(from + G::E0 + 16)[r + 8];
                if (!whole) {
                    if (bad >> n & 1) {
                        s[n][0] = s[n][1] = s[n][2] = s[n][3] = not_a_number();
                        e[n][0] = e[n][1] = 0.0f;
                    }
                    const int t0 = group_token(groups, group + n) + r;
                    const bool there = group + n < g1;
                    if (!there || !sees(pa, t0, a.window, a.sinks)) s[n][0] = minus_infinity();
                    if (!there || !sees(pb, t0, a.window, a.sinks)) s[n][1] = minus_infinity();
                    if (!there || !sees(pa, t0 + 8, a.window, a.sinks)) s[n][2] = minus_infinity();
                    if (!there || !sees(pb, t0 + 8, a.window, a.sinks)) s[n][3] = minus_infinity();
                }
            };
            static_for<2>(score_group);
            // what a weight in the sum and a token's weight are 2 to the power of
            float x[2][4], t[2][4];
            const auto exponents = [&]() {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        t[n][i] = s[n][i] - (i & 1 ? sub_mb : sub_ma);
                        x[n][i] = t[n][i] + (e[n][i / 2] - (i & 1 ? sub_Rb : sub_Ra));
                    }
                }
            };
            exponents();
            const auto most = [](const float (&v)[2][4], int i) { return fmaxf(fmaxf(v[0][i], v[0][i + 2]), fmaxf(v[1][i], v[1][i + 2])); };
            const float sa = most(s, 0), sb = most(s, 1);
            if (__any_sync(~0u, sa > ma + kLag || sb > mb + kLag || fmaxf(most(x, 0), most(x, 1)) > kLag + kLift)) {
                float na = sa, nb = sb;
#pragma unroll
                for (int d = 4; d < 32; d *= 2) {
                    na = fmaxf(na, __shfl_xor_sync(~0u, na, d));
                    nb = fmaxf(nb, __shfl_xor_sync(~0u, nb, d));
                }
                na = fmaxf(ma, na);
                nb = fmaxf(mb, nb);
                la *= power2(ma - reference(na));
                lb *= power2(mb - reference(nb));
                Ra = relative(Ra, ma, na);
                Rb = relative(Rb, mb, nb);
                ma = na, mb = nb;
                sub_ma = reference(ma), sub_mb = reference(mb), sub_Ra = 0.0f, sub_Rb = 0.0f;
                exponents();
                float Na = most(x, 0), Nb = most(x, 1);
#pragma unroll
                for (int d = 4; d < 32; d *= 2) {
                    Na = fmaxf(Na, __shfl_xor_sync(~0u, Na, d));
                    Nb = fmaxf(Nb, __shfl_xor_sync(~0u, Nb, d));
                }
                Na = fmaxf(Ra, Na);
                Nb = fmaxf(Rb, Nb);
                const float fa = power2(Ra - reference(Na)), fb = power2(Rb - reference(Nb));
#pragma unroll
                for (int d = 0; d < KS; ++d) {
                    o[d][0] *= fa;
                    o[d][1] *= fb;
                    o[d][2] *= fa;
                    o[d][3] *= fb;
                }
                Ra = Na, Rb = Nb;
                sub_Ra = reference(Ra) - kLift, sub_Rb = reference(Rb) - kLift;
                exponents();
            }
            la += (power2(t[0][0]) + power2(t[0][2])) + (power2(t[1][0]) + power2(t[1][2]));
            lb += (power2(t[0][1]) + power2(t[0][3])) + (power2(t[1][1]) + power2(t[1][3]));

            const auto weigh_group = [&](auto N) {
                constexpr int n = decltype(N)::value;
                const uint8_t* const from = at + n * G::BYTES;
                const float w[4] = {power2(x[n][0]), power2(x[n][1]), power2(x[n][2]), power2(x[n][3])};
                const uint32_t h0 = half2_of(w[0], w[1]), h1 = half2_of(w[2], w[3]);
                const uint32_t w0 = transpose8x8(h0), w1 = transpose8x8(h1);
                uint32_t x0 = 0, x1 = 0;
                if (REST) {
                    x0 = transpose8x8(half2_of(w[0] - low_half(h0), w[1] - high_half(h0)));
                    x1 = transpose8x8(half2_of(w[2] - low_half(h1), w[3] - high_half(h1)));
                }
                // values: tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9 in rows of the same numbers
                uint32_t v[4][G::VW], hv[4][G::VB], vs[2][G::VB];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int row = 2 * c + (t & 1) + (t >> 1) * 8;
                    load_words<G::VW>(from + G::V0 + row * G::ROW + row / 2 * 32 + r * (G::ROW / 8), v[t]);
                    half_scales<FMT, G::VB>(from + G::S0 + 16 * G::BLOCKS + row * G::BLOCKS + r * (WIDTH / 8) / G::BLOCK,
                                            FMT == kMxfp4 ? reinterpret_cast<const int8_t*>(from + G::E0 + 16)[row] : 0, hv[t]);
                }
                if (!whole) {
                    // a NaN reaches only the columns that see its token
#pragma unroll
                    for (int d = 0; d < G::VB; ++d) {
                        uint32_t nan = 0;
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            if ((bad >> n & 1) || half_is_nan(hv[t][d])) {
                                nan |= 1u << t;
                                hv[t][d] = 0;
                            }
                        }
                        if (group + n < g1 && __any_sync(~0u, nan != 0)) {
#pragma unroll 1
                            for (int cc = 0; cc < 4; ++cc) {
                                const uint32_t theirs = __shfl_sync(~0u, nan, (lane & ~3) | cc);
#pragma unroll 1
                                for (int t = 0; t < 4; ++t) {
                                    if (!(theirs >> t & 1)) continue;
                                    const int j = group_token(groups, group + n) + 2 * cc + (t & 1) + (t >> 1) * 8;
                                    const bool hit_a = sees(pa, j, a.window, a.sinks), hit_b = sees(pb, j, a.window, a.sinks);
                                    constexpr int SPAN = KS / G::VB;
#pragma unroll
                                    for (int e = d * SPAN; e < (d + 1) * SPAN; ++e) {
                                        if (hit_a) o[e][0] = o[e][2] = not_a_number();
                                        if (hit_b) o[e][1] = o[e][3] = not_a_number();
                                    }
                                }
                            }
                            __syncwarp();
                        }
                    }
                }
#pragma unroll
                for (int d = 0; d < G::VB; ++d) {
                    vs[0][d] = both_low(hv[0][d], hv[1][d]);
                    vs[1][d] = both_low(hv[2][d], hv[3][d]);
                }
                auto value_word = [&](auto W) {
                    constexpr int w = decltype(W)::value;
                    // bytes of two tokens: even elements in xe, odd ones in xo
                    const uint32_t m = 0x0f0f0f0fu;
                    const uint32_t xe = (v[0][w] & m) | (v[1][w] << 4 & ~m), xo = (v[0][w] >> 4 & m) | (v[1][w] & ~m);
                    const uint32_t ye = (v[2][w] & m) | (v[3][w] << 4 & ~m), yo = (v[2][w] >> 4 & m) | (v[3][w] & ~m);
                    auto tile = [&](auto I) {
                        constexpr int i = decltype(I)::value, d = w * 4 + i;
                        constexpr int blk = d / (KS / G::VB);
                        const uint32_t a0 = mul_half2(codes2<i>(xe), vs[0][blk]), a1 = mul_half2(codes2<i>(xo), vs[0][blk]);
                        const uint32_t a2 = mul_half2(codes2<i>(ye), vs[1][blk]), a3 = mul_half2(codes2<i>(yo), vs[1][blk]);
                        mma16816(o[d], a0, a1, a2, a3, w0, w1);
                        if (REST) mma16816(o[d], a0, a1, a2, a3, x0, x1);
                    };
                    static_for<4>(tile);
                };
                static_for<G::VW>(value_word);
            };
            static_for<2>(weigh_group);
        }
        wait_copies<0>();
        __syncthreads();  // the warps' stages become their sums

        // the warps' parts
#pragma unroll
        for (int d = 4; d < 32; d *= 2) {
            la += __shfl_xor_sync(~0u, la, d);
            lb += __shfl_xor_sync(~0u, lb, d);
        }
        if (r == 0) {
            s_m[warp][2 * c] = ma;
            s_m[warp][2 * c + 1] = mb;
            s_R[warp][2 * c] = Ra;
            s_R[warp][2 * c + 1] = Rb;
            s_l[warp][2 * c] = la;
            s_l[warp][2 * c + 1] = lb;
        }
        {
            float* mine_a = sums + (warp * 8 + 2 * c) * ROW + r * (WIDTH / 8);
            float* mine_b = mine_a + ROW;
#pragma unroll
            for (int d = 0; d < KS; ++d) {
                *reinterpret_cast<float2*>(mine_a + 2 * d) = make_float2(o[d][0], o[d][2]);
                *reinterpret_cast<float2*>(mine_b + 2 * d) = make_float2(o[d][1], o[d][3]);
            }
        }
        __syncthreads();
        constexpr int LANES = kWarps * 32 / 8;  // threads of a column
        const int col = threadIdx.x / LANES, at = threadIdx.x % LANES;
        if (col < columns) {
            float m = s_m[0][col], R = s_R[0][col];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) join_references(m, R, s_m[w][col], s_R[w][col]);
            float l = 0.0f, f[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                l += s_l[w][col] * power2(s_m[w][col] - reference(m));
                f[w] = power2(relative(s_R[w][col], s_m[w][col], m) - reference(R));
            }
            const bool any = before + (column0 + col) / a.group >= 0;
            const bool complete = !TOGETHER && g0 == 0 && g1 == groups.count;
            const int64_t token = seq.first_token + (column0 + col) / a.group, h = head * a.group + (column0 + col) % a.group;
            const int64_t part = (2LL * blockIdx.x + (g0 == 0 ? 1 : 0)) * 8 + col;
            const Finish z = finish_of(R, l, kSumLift, any);
            T* out = static_cast<T*>(a.out) + token * a.ot + h * a.oh;
            float* const merged = sums + kWarps * 8 * ROW + col * ROW;
            if (TOGETHER && at == 0) {
                merged[WIDTH] = m;
                merged[WIDTH + 1] = R;
                merged[WIDTH + 2] = l;
            }
            if (!TOGETHER && !complete && at == 0) a.part[part] = make_float4(m, R, l, any ? 1.0f : 0.0f);
#pragma unroll
            for (int d = at * 4; d < WIDTH; d += LANES * 4) {
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 x = *reinterpret_cast<const float4*>(sums + (w * 8 + col) * ROW + d);
                    y[0] = fmaf(x.x, f[w], y[0]);
                    y[1] = fmaf(x.y, f[w], y[1]);
                    y[2] = fmaf(x.z, f[w], y[2]);
                    y[3] = fmaf(x.w, f[w], y[3]);
                }
                if (TOGETHER) *reinterpret_cast<float4*>(merged + d) = make_float4(y[0], y[1], y[2], y[3]);
                else if (complete) store4(out, d, a.c.dim, a.vec_out, z, y);
                else *reinterpret_cast<float4*>(a.sums + part * WIDTH + d) = make_float4(y[0], y[1], y[2], y[3]);
            }
        }
        if constexpr (TOGETHER) {
            // CTA `rank` sums columns rank, rank + splits, ...
            cluster_sync();
            const uint32_t merged = smem_addr(sums + kWarps * 8 * ROW);
            for (int col = rank; col < columns; col += a.splits) {
                const uint32_t from = merged + col * ROW * 4;
                float m = minus_infinity(), R = m, l = 0.0f, f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (k >= a.splits) break;
                    join_references(m, R, read_cluster(from + WIDTH * 4, k), f[k] = read_cluster(from + WIDTH * 4 + 4, k));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (k >= a.splits) break;
                    const float own = read_cluster(from + WIDTH * 4, k);
                    l += read_cluster(from + WIDTH * 4 + 8, k) * power2(own - reference(m));
                    f[k] = power2(relative(f[k], own, m) - reference(R));
                }
                const bool any = before + (column0 + col) / a.group >= 0;
                const Finish z = finish_of(R, l, kSumLift, any);
                T* out = static_cast<T*>(a.out) + (int64_t)(seq.first_token + (column0 + col) / a.group) * a.ot +
                         (int64_t)(head * a.group + (column0 + col) % a.group) * a.oh;
                for (int d = threadIdx.x; d < a.c.dim; d += kWarps * 32) {
                    float y = 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (k >= a.splits) break;
                        y = fmaf(read_cluster(from + d * 4, k), f[k], y);
                    }
                    out[d] = from_float<T>(any ? y * z.x * z.x * z.inverse : 0.0f);
                }
            }
            cluster_sync();  // nobody's memory goes while another reads it
            break;
        }
        // the next item
        run += g1 - g0;
        if (run >= run_end) {
            if (threadIdx.x == 0) {
                CutItem cut{0, 0, 0, 0, 0, 0};
                if (g0 == 0 && g1 < groups.count)
                    cut = CutItem{columns, (int)(Cut{total, ctas}.owner(run + groups.count - g1 - 1) - blockIdx.x), seq.first_token, column0, head, before};
                a.cuts[blockIdx.x] = cut;
            }
            break;
        }
        __syncthreads();
        g0 = 0;
        if (++head == a.c.heads) {
            head = 0;
            if (++ct == tiles_of(a, seq)) {
                ct = 0;
                do seq = sequence_at(a, ++b);
                while (seq.tokens == 0);
            }
            groups = tile_groups(a, seq, ct);
        }
    }
}

// A row's parts, a thread for four elements: the references first, a lane for a part.
template <typename T, int WIDTH>
__global__ void __launch_bounds__(128) join_kernel(const AttendArgs a, float lift) {
    constexpr int WARPS = WIDTH == 256 ? 2 : 1;  // of a row
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rows = a.b.tokens * a.heads;
    const int64_t row = (int64_t)blockIdx.x * (4 / WARPS) + warp / WARPS;
    if (row >= rows) return;
    const int64_t token = row / a.heads, h = row % a.heads;
    const int s = search(a.b, token, [&](int i) { return a.b.starts[i]; });
    if (s < 0 || a.b.starts[s] < 0 || a.b.starts[s + 1] <= token || a.b.starts[s + 1] > a.b.tokens || !a.takes(a.b.starts[s + 1] - a.b.starts[s])) return;
    // the item that the row is of, and its parts
    constexpr int ROWS = WIDTH == 256 ? 128 : 256;
    const int s0 = a.b.starts[s], tokens = a.b.starts[s + 1] - s0, before = length_of(a.b, s) - tokens;
    const int column = ((int)token - s0) * a.group + (int)(h % a.group), first = column / ROWS * ROWS, last = min(first + ROWS, tokens * a.group) - 1;
    const int splits = parts_of((groups_of(a.c, a.b, before + first / a.group, before + last / a.group, a.window, a.sinks).count + 7) / 8, a.splits);
    if (splits == 1) return;  // written as a whole
    float m = minus_infinity(), R = m;
    float4 mine = make_float4(m, m, 0.0f, 0.0f);
    for (int i = lane; i < splits; i += 32) {
        const float4 p = a.part[i * rows + row];
        if (i < 32) mine = p;
        join_references(m, R, p.x, p.y);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) join_references(m, R, __shfl_xor_sync(~0u, m, d), __shfl_xor_sync(~0u, R, d));
    const bool any = __shfl_sync(~0u, mine.w, 0) != 0.0f;
    const int at = ((warp % WARPS) * 32 + lane) * 4;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
    for (int i0 = 0; i0 < splits; i0 += 32) {
        if (i0 > 0) mine = i0 + lane < splits ? a.part[(i0 + lane) * rows + row] : make_float4(minus_infinity(), minus_infinity(), 0.0f, 0.0f);
        l += mine.z * power2(mine.x - reference(m));
        const float f = power2(relative(mine.y, mine.x, m) - reference(R));
        const int n = min(32, splits - i0);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float w = __shfl_sync(~0u, f, i);
            if (at < WIDTH) {
                const float4 x = *reinterpret_cast<const float4*>(a.sums + ((i0 + i) * rows + row) * WIDTH + at);
                y[0] = fmaf(x.x, w, y[0]);
                y[1] = fmaf(x.y, w, y[1]);
                y[2] = fmaf(x.z, w, y[2]);
                y[3] = fmaf(x.w, w, y[3]);
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(~0u, l, d);
    if (at < WIDTH) store4(static_cast<T*>(a.out) + token * a.ot + h * a.oh, at, a.c.dim, a.vec_out, finish_of(R, l, lift, any), y);
}

// The outputs of the items that were cut: block i that which CTA i began, PER warps for
// a column, each with every PER-th part.
template <typename T, int WIDTH, int PER>
__global__ void __launch_bounds__(8 * PER * 32) join_cut_kernel(const AttendArgs a, float lift) {
    constexpr int VALUES = WIDTH / 32;  // of a lane
    constexpr int BATCH = 8;            // parts loaded at once
    __shared__ float y_of[PER > 1 ? 8 * PER : 1][PER > 1 ? WIDTH : 1];
    __shared__ float l_of[8 * PER];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, column = warp / PER, share = warp % PER;
    const CutItem item = a.cuts[blockIdx.x];
    if (item.columns == 0) return;
    const int parts = item.others + 1;
    const auto slot = [&](int i) { return (2LL * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * 8 + column; };
    float m = minus_infinity(), R = m, l = 0.0f, y[VALUES];
#pragma unroll
    for (int k = 0; k < VALUES; ++k) y[k] = 0.0f;
    if (column < item.columns) {
        for (int i = lane; i < parts; i += 32) {
            const float4 p = a.part[slot(i)];
            join_references(m, R, p.x, p.y);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) join_references(m, R, __shfl_xor_sync(~0u, m, d), __shfl_xor_sync(~0u, R, d));
        for (int i0 = share; i0 < parts; i0 += BATCH * PER) {
            float x[BATCH][VALUES];
            float4 p[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int64_t at = slot(min(i0 + i * PER, parts - 1));
                p[i] = a.part[at];
#pragma unroll
                for (int k = 0; k < VALUES; ++k) x[i][k] = a.sums[at * WIDTH + lane + 32 * k];
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (i0 + i * PER >= parts) continue;
                l += p[i].z * power2(p[i].x - reference(m));
                const float f = power2(relative(p[i].y, p[i].x, m) - reference(R));
#pragma unroll
                for (int k = 0; k < VALUES; ++k) y[k] = fmaf(x[i][k], f, y[k]);
            }
        }
        if (PER > 1) {
#pragma unroll
            for (int k = 0; k < VALUES; ++k) y_of[warp][lane + 32 * k] = y[k];
            if (lane == 0) l_of[warp] = l;
        }
    }
    if (PER > 1) __syncthreads();
    if (share != 0 || column >= item.columns) return;
#pragma unroll
    for (int w = 1; w < PER; ++w) {
        l += l_of[warp + w];
#pragma unroll
        for (int k = 0; k < VALUES; ++k) y[k] += y_of[warp + w][lane + 32 * k];
    }
    const int col = item.column + column;
    const bool any = item.before + col / a.group >= 0;
    const Finish z = finish_of(R, l, lift, any);
    T* out = static_cast<T*>(a.out) + (int64_t)(item.first_token + col / a.group) * a.ot + (int64_t)(item.head * a.group + col % a.group) * a.oh;
#pragma unroll
    for (int k = 0; k < VALUES; ++k)
        if (lane + 32 * k < a.c.dim) out[lane + 32 * k] = from_float<T>(any ? y[k] * z.x * z.x * z.inverse : 0.0f);
}

template <int WIDTH, int FMT>
constexpr size_t columns_smem() {
    return std::max<size_t>((kWarps + 1) * 8 * (WIDTH + 4) * sizeof(float), (size_t)kWarps * Stage<WIDTH, FMT>::STAGES * 2 * Stage<WIDTH, FMT>::BYTES);
}
template <typename T, int WIDTH, int FMT>
cudaError_t columns(const AttendArgs& a, cudaStream_t st) {
    const size_t smem = columns_smem<WIDTH, FMT>();
    if (a.together) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(a.tiles(8) * a.c.heads), (unsigned)a.splits);
        cfg.blockDim = dim3(kWarps * 32);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1;
        attr[0].val.clusterDim.y = (unsigned)a.splits;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, attend_columns_kernel<T, WIDTH, FMT, true>, a);
    }
    cudaError_t err = launch_pdl(attend_columns_kernel<T, WIDTH, FMT, false>, dim3((unsigned)a.splits), dim3(kWarps * 32), smem, st, a);
    if (err != cudaSuccess) return err;
    // few items for many CTAs: many parts of each
    const float lift = kLift + (FMT == kMxfp4 ? kMxLift : 0);
    const bool long_items = a.tiles(8) * a.c.heads * 8 < a.splits;
    return long_items ? launch_pdl(join_cut_kernel<T, WIDTH, WIDTH == 256 ? 2 : 4>, dim3((unsigned)a.splits), dim3(WIDTH == 256 ? 512 : 1024), 0, st, a, lift)
                      : launch_pdl(join_cut_kernel<T, WIDTH, 1>, dim3((unsigned)a.splits), dim3(256), 0, st, a, lift);
}
template <typename T, int WIDTH>
cudaError_t join(const AttendArgs& a, float lift, cudaStream_t st) {
    const int64_t rows = a.b.tokens * a.heads, per = WIDTH == 256 ? 2 : 4;
    return launch_pdl(join_kernel<T, WIDTH>, dim3((unsigned)((rows + per - 1) / per)), dim3(128), 0, st, a, lift);
}

// CTAs that the SMs hold at once.
template <typename T, int WIDTH, int FMT>
int resident() {
    static std::atomic<int> cached[64];
    int dev = 0, per = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    const size_t smem = columns_smem<WIDTH, FMT>();
    if (smem > 48 * 1024 &&
        (cudaFuncSetAttribute(attend_columns_kernel<T, WIDTH, FMT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
         cudaFuncSetAttribute(attend_columns_kernel<T, WIDTH, FMT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)) {
        (void)cudaGetLastError();
        return device_sms();
    }
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, attend_columns_kernel<T, WIDTH, FMT, false>, kWarps * 32, smem) != cudaSuccess || per < 1) {
        (void)cudaGetLastError();
        return device_sms();
    }
    n = per * device_sms();
    cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

// f(type, width, format) for those of the call.
template <class F>
auto with_kernel(const AttendArgs& a, int type, F f) {
    const auto width = [&](auto t, auto fmt) {
        using W = std::integral_constant<int, 64>;
        using X = std::integral_constant<int, 128>;
        using Y = std::integral_constant<int, 256>;
        return a.c.width == 64 ? f(t, W{}, fmt) : a.c.width == 128 ? f(t, X{}, fmt) : f(t, Y{}, fmt);
    };
    const auto format = [&](auto t) {
        return a.c.fmt == kMxfp4 ? width(t, std::integral_constant<int, kMxfp4>{}) : width(t, std::integral_constant<int, kNvfp4>{});
    };
    return type == DDGEMM_BF16 ? format(__nv_bfloat16{}) : format(__half{});
}

}  // namespace

// Short sequences (as far as the page table and the window say) in few enough items: a
// cluster for each, of up to 8 CTAs with 256 tokens or more, 512 at most, all on the SMs at
// once.  (523 tokens, 8 heads: 10.1 us, 14.7 as runs and a second launch; 288 items of 1036
// tokens 24 us in two rounds, 18.5 as runs.)
void plan_attend_columns(AttendArgs& a, int type) {
    const int ctas = with_kernel(a, type, [](auto t, auto w, auto f) { return resident<decltype(t), decltype(w)::value, decltype(f)::value>(); });
    const int64_t table = (int64_t)a.b.table_pages * a.c.page_size, longest = a.window > 0 ? std::min<int64_t>(table, (int64_t)a.window + a.sinks + 32) : table;
    const int64_t items = a.tiles(8) * a.c.heads;
    const int64_t share = std::min<int64_t>({8, (longest + 255) / 256, ctas / std::max<int64_t>(1, items)});
    a.together = share >= 1 && longest <= share * 512;
    a.splits = a.together ? (int)share : ctas;
}

cudaError_t launch_attend_columns(const AttendArgs& a, int type, cudaStream_t st) {
    return with_kernel(a, type, [&](auto t, auto w, auto f) { return columns<decltype(t), decltype(w)::value, decltype(f)::value>(a, st); });
}

cudaError_t launch_attend_join(const AttendArgs& a, int type, float lift, cudaStream_t st) {
    if (type == DDGEMM_BF16)
        return a.c.width == 64 ? join<__nv_bfloat16, 64>(a, lift, st) : a.c.width == 128 ? join<__nv_bfloat16, 128>(a, lift, st) : join<__nv_bfloat16, 256>(a, lift, st);
    return a.c.width == 64 ? join<__half, 64>(a, lift, st) : a.c.width == 128 ? join<__half, 128>(a, lift, st) : join<__half, 256>(a, lift, st);
}

}  // namespace ddg
