// attend_tile.cu -- attention over the 4-bit cache for many queries, on the tensor
// cores (tcgen05).
//
// A CTA takes tiles of 128 (query token, head of the group) rows of one sequence and
// key/value head, two at a time (one of width 256), over the cache in tiles of 128
// tokens, eight groups of 16 wherever their pages lie.  Warps: four for the softmax of
// each tile of rows, then 8 (16 of width 256) that turn codes into 16-bit keys and
// values, then one that issues the MMAs:
//   S = Q K^T       operands in shared memory, 128-byte swizzle, f32 in tensor memory;
//   P = 2^(S f - m) a thread for a row, from tensor memory and back into it in 16
//                   bits, over S;
//   O += P V        P from tensor memory, V as it lies (tokens by head elements).
// One tile's softmax overlaps the other's MMAs; O stays in tensor memory and is
// multiplied only when a row's reference m has to follow: a row's weights are taken by
// the m so far, in one pass, and only where 32 of them come to more than kMost does m
// become the largest score, up to a whole number.
//
// The conversion is shared by the 256 rows.  Exponents of rows become relative to the
// tile's largest, for keys a factor of all its scores and for values one of all its
// weights: codes times scales are exact in 16 bits while a tile's rows are within 2^9 of
// one another (mxfp4: down to 2^-27 of the row's largest block).  One of the warps without
// another task looks at the exponents; an item with rows further apart, or with scores of
// 2^21 and more, is done again behind the loops, a step after the other.
//
// Measured: a prompt of 8192 tokens, 32 heads over 8 of 128, mxfp4, bfloat16: 538 us, 1.0
// PF/s (the simple kernel with mma.sync that was here first: 5008).  A pair of tiles takes
// 4700 clocks for 128 tokens: each row's pass over its scores about half of them (in four steps
// of 32: wait for tensor memory, fma, 2^x, sum, round, store), then its products with V
// and the next K, 1024, and the waits between; the tensor pipe is busy for 2048 of them, the
// converters for 3000.  So the chain of one row's softmax and its MMAs bounds it.  Scores
// of 64 tokens, in two buffers, would overlap them, but read Q from shared memory twice as
// often: 593 us where this form took 548.  Three chunks of 100 to 700 tokens behind 2111 to
// 16000, 5 queries a head of 256, nvfp4, float16: 340 us, 0.53 PF/s; the rest of the weights is a
// second product there (22 bits for bfloat16 too: 8192 tokens in 711 us for 538, the error
// against 64 bits the same, the output's rounding), K and V have one stage each, and the
// converters' stores (twice 64 KB a tile), the MMAs' reads and the waits for each other's stage
// make 5900 clocks a tile.  Values in two halves that come and go by themselves, or codes
// loaded a line at a time, changed nothing.
#include <algorithm>

#include "attend.cuh"
#include "umma.cuh"

namespace ddg {
namespace {

constexpr unsigned long long kWaitNs = 2000000000ULL;  // bounded waits: 2 s
constexpr float kMost = 32768.0f;  // a row's reference follows where 32 weights are more than this in all
constexpr int kShift = 3;      // the values' exponent follows by more than 2^3 either way
constexpr float kLift = 7.0f;  // the weight of a score equal to the reference is 2^(7 + up to 3 either way)
// What the loops are for; an item beyond is done again by careful_item.
constexpr int kSpread = 9;     // exponents of a tile's keys, and of its values, are so far apart at most: mxfp4 blocks down to
                               // 2^-27 of their row's largest are exact then, as nvfp4 ones
constexpr int kReach = 12;     // of all values of an item: one of 2^12 times another's size has a weight of 2^-24 or more where it counts
constexpr float kMostScore = 2097152.0f;  // references are below 2^21, so that lifts and exponents are not lost beside them
constexpr int kRing = 4;  // tiles whose rows, exponents and marks are kept
constexpr int kNoToken = -4096;  // in the place of an exponent
constexpr int kNone = 4096;      // of the least of no exponents

__device__ unsigned int g_attend_timeouts = 0;

// By how much codes times scales are lifted: the largest becomes 2^15.4 (E4M3) or 2^15.6.
template <int FMT> __host__ __device__ constexpr int lift_of() { return FMT == kMxfp4 ? 13 : 4; }

template <int WIDTH>
struct Shape {
    static constexpr int NQ = WIDTH == 256 ? 1 : 2;       // tiles of rows
    // threads that convert: where one tile of rows shares them, twice as many (three chunks, see above: 336 us for 363)
    static constexpr int CONVERTERS = WIDTH == 256 ? 512 : 256;
    static constexpr int MMA_WARP = 4 * NQ + CONVERTERS / 32, THREADS = (MMA_WARP + 4) * 32;  // the last three warps have no task
    static constexpr int STAGES = WIDTH == 256 ? 1 : 2;   // of keys, and of values
    static constexpr int BLOCK_BYTES = 128 * 128;         // 128 rows of 64 elements
    static constexpr int TILE_BYTES = WIDTH / 64 * BLOCK_BYTES;
    static constexpr int K0 = NQ * TILE_BYTES, V0 = K0 + STAGES * TILE_BYTES;
    static constexpr int SMEM = V0 + STAGES * TILE_BYTES + 1024;
    static constexpr int BUFFERS = 2 / NQ;                // of scores, of a tile of rows
    static constexpr int PIECES = WIDTH / 32;                     // of 32 codes, of a token
    static constexpr int PER_PASS = CONVERTERS / PIECES;          // tokens that the threads convert at once
    static constexpr int PASSES = 128 / PER_PASS;
    static constexpr uint32_t S_COL = 0, O_COL = 256;
    // registers of a thread by role: of those that each is launched with, a part of the SM has 480 for its warps (one
    // of each tile's softmax, two or four that convert, one of the last four)
    static constexpr int SOFTMAX_REGS = NQ == 2 ? 136 : 176, CONVERT_REGS = NQ == 2 ? 80 : 64, MMA_REGS = 48;
    static_assert(THREADS / 128 * (NQ == 2 ? 96 : 80) == 480 && NQ * SOFTMAX_REGS + CONVERTERS / 128 * CONVERT_REGS + MMA_REGS <= 480, "registers of the launch");
};

// What the softmax has to know of a tile.
struct TileInfo {
    float key_factor;
    int value_exponent;
    uint32_t bad;  // groups whose page is not there
};

// A thread's pieces of a tile's keys or values.
template <int PASSES>
struct Raw {
    uint4 codes[PASSES];
    uint16_t scales[PASSES];
};

// Eight codes as four pairs of halves.
__device__ __forceinline__ uint4 halves_of(uint32_t w) {
    uint4 h;
    asm("{\n"
        " .reg .b8 t0, t1, t2, t3;\n"
        " mov.b32 {t0, t1, t2, t3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, t0;\n"
        " cvt.rn.f16x2.e2m1x2 %1, t1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, t2;\n"
        " cvt.rn.f16x2.e2m1x2 %3, t3;\n"
        "}\n"
        : "=r"(h.x), "=r"(h.y), "=r"(h.z), "=r"(h.w)
        : "r"(w));
    return h;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void store_shared(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Loads that stay where they are written, ahead of the conversions of the tile before.
__device__ __forceinline__ uint4 fetch16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint16_t fetch2(const void* p) {
    uint16_t v;
    asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint16_t fetch1(const void* p) {
    uint16_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int fetch_signed1(const void* p) {
    int v;
    asm volatile("ld.global.s8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int fetch4(const void* p) {
    int v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// D = A B^T (+ D) with A in tensor memory.
__device__ __forceinline__ void mma_from_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void store_tmem16(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// The same columns as tc5::ld32, without the wait: the values are there after
// wait_tmem_loads, which names them so that no use moves ahead of it.
__device__ __forceinline__ void start_load32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]),
          "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),
          "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void wait_tmem_loads(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                   "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void wait_tmem_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// 16 columns of 32 bits, with the wait for them.
__device__ __forceinline__ void load_tmem16(uint32_t at, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at)
        : "memory");
}
// 32 weights (and what their rounding left) times a power of two.
template <bool REST>
__device__ __forceinline__ void follow_weights(uint32_t at, uint32_t by) {
    wait_tmem_stores();
#pragma unroll
    for (int k = 0; k < (REST ? 2 : 1); ++k) {
        uint32_t v[16];
        load_tmem16(at + 16 * k, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = mul_half2(v[i], by);
        store_tmem16(at + 16 * k, v);
    }
}

template <bool REST>
__device__ __noinline__ void call_follow_weights(uint32_t at, uint32_t by) { follow_weights<REST>(at, by); }

// The scales of 32 codes (two blocks of nvfp4, in the halves of raw) as halves, each in both halves of a word, 2^add
// (mxfp4: the byte joins it) or 2^(o + add) (nvfp4) times; o: the row's exponent, kNoToken for 0.  Those of values that
// are NaN become 0, and the answer is whether there are any.
template <int FMT>
__device__ __forceinline__ bool piece_scales(uint32_t raw, int o, int add, uint32_t inside, bool value, uint32_t (&s)[2]) {
    bool found = false;
    if (FMT == kMxfp4) {
        const float power = exp2_int(min(max((int)raw + add, -126), 15));
        s[0] = raw == 255u ? 0x7fff7fffu : half2_of(power, power);
        if (o == kNoToken) s[0] = 0;
    } else {
        const float power = exp2_int(min(max(o + add, -126), 15));  // 0 as a half where there is no token
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s[0]) : "h"((uint16_t)raw));
        if (o == kNoToken) s[0] = 0;
        s[0] = mul_half2(s[0], half2_of(power, power));
    }
    s[0] &= inside;
    if (value) {  // NaN: 0 here, and looked for at the end
        const __half2 is = __hisnan2(*reinterpret_cast<const __half2*>(&s[0]));
        const uint32_t nan = *reinterpret_cast<const uint32_t*>(&is);
        if (nan != 0) {
            found = true;
            s[0] &= (nan & 0xffffu ? 0u : 0xffffu) | (nan >> 16 ? 0u : 0xffff0000u);
        }
    }
    s[1] = FMT == kMxfp4 ? s[0] : __byte_perm(s[0], s[0], 0x3232);
    if (FMT == kNvfp4) s[0] = __byte_perm(s[0], s[0], 0x1010);
    return found;
}
// 32 codes times their scales to a row of 128 bytes, 16 swizzled bytes at a time.
__device__ __forceinline__ void store_piece(uint32_t to, const uint4& codes, const uint32_t (&s)[2]) {
    const uint32_t words[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int k0 = 0; k0 < 4; ++k0) {
        uint4 v = halves_of(words[k0]);
        const uint32_t sc = s[k0 / 2];
        v.x = mul_half2(v.x, sc);
        v.y = mul_half2(v.y, sc);
        v.z = mul_half2(v.z, sc);
        v.w = mul_half2(v.w, sc);
        store_shared(to ^ (uint32_t)(k0 << 4), v);
    }
}
// Blocks of the part-th 32 elements that begin beyond the head's end take no part, whatever they hold.
template <int BLOCK>
__device__ __forceinline__ uint32_t inside_of(int part, int dim) {
    return (part * 32 < dim ? 0xffffu : 0u) | (part * 32 + BLOCK % 32 < dim ? 0xffff0000u : 0u);
}
// Where they go: the token's row, swizzled.
__device__ __forceinline__ uint32_t piece_place(int part, int t, uint32_t block_bytes) {
    return part / 2 * block_bytes + t * 128 + (uint32_t)(((part % 2 * 4) ^ (t % 8)) << 4);
}
// What a tile's scores are times beside the row's own factor.
template <int FMT>
__device__ __forceinline__ float key_factor_of(int key_exponent) { return mxfp4_scale((uint32_t)(key_exponent + 127)) * exp2_int(-lift_of<FMT>()); }

// Bits of the 32 tokens of groups g and g + 1: those that a query at p sees.
__device__ __forceinline__ uint32_t seen_bits(const Groups& groups, int p, int window, int sinks, int g0) {
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int g = g0 + k, j0 = group_token(groups, g);
        const uint32_t upto = (1u << min(max(p - j0 + 1, 0), 16)) - 1u;
        uint32_t from = 0xffffu;
        if (window > 0) from = ~((1u << min(max(p - window - j0 + 1, 0), 16)) - 1u) | ((1u << min(max(sinks - j0, 0), 16)) - 1u);
        if (g < groups.count) bits |= (upto & from & 0xffffu) << (16 * k);
    }
    return bits;
}

// S = Q K^T of a tile of rows, and O = (O +) P V, issued by one thread; shared-memory addresses of the operands.
template <int WIDTH>
__device__ __forceinline__ void issue_scores(uint32_t s_at, uint32_t q, uint32_t k_tile) {
    using S = Shape<WIDTH>;
    constexpr uint32_t DESC = tc5::idesc_f16(false, false, false, 128, 128);
    const uint64_t qd = tc5::desc_kmajor_sw128(q), kd = tc5::desc_kmajor_sw128(k_tile);
#pragma unroll
    for (int k = 0; k < WIDTH / 16; ++k) {
        const uint64_t at = (uint64_t)(k / 4 * (S::BLOCK_BYTES / 16) + k % 4 * 2);
        tc5::mma_f16_single(s_at, qd + at, kd + at, DESC, k > 0 ? 1u : 0u);
    }
}
template <int WIDTH, bool REST>
__device__ __forceinline__ void issue_sums(uint32_t o_at, uint32_t p_at, uint32_t v_tile, bool add) {
    using S = Shape<WIDTH>;
    constexpr uint32_t DESC = tc5::idesc_f16(false, false, true, 128, WIDTH);
    const uint64_t vd = tc5::desc_mnmajor_sw128(v_tile, S::BLOCK_BYTES);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t from = p_at + k / 2 * 32 + k % 2 * 8;
        mma_from_tmem(o_at, from, vd + k * (2048 / 16), DESC, add || k != 0 ? 1u : 0u);
        if (REST) mma_from_tmem(o_at, from + 16, vd + k * (2048 / 16), DESC, 1u);
    }
}

struct Barriers {
    uint64_t q, k_full[2], k_empty[2], v_full[2], v_empty[2], done, careful;
    uint64_t s[2], p[2], o[2];
    uint64_t info[kRing];  // of tiles in turn
};

// NaN in an output row (or its part) for the blocks of values that are NaN in a token
// of groups g0 .. g1 - 1 that the row sees.
template <typename T, int WIDTH, int FMT>
__device__ __noinline__ void mark_nan(const AttendArgs& a, const Item& item, const Groups& groups, int head, int p, int g0, int g1,
                                      int64_t token, int64_t h, bool cut) {
    constexpr int BLOCK = mx4_block(FMT), BLOCKS = WIDTH / BLOCK;
    uint32_t blocks = 0;
    for (int g = g0; g < g1; ++g) {
        const int first = group_token(groups, g), page = page_of(a.c, a.b, item.sequence, first);
        if (page < 0) continue;
        const uint8_t* row = a.c.scales + cache_row(a.c, page, 1, head, first & (a.c.page_size - 1)) * BLOCKS;
        for (int t = 0; t < 16; ++t) {
            if (!sees(p, first + t, a.window, a.sinks)) continue;
            for (int b = 0; b < BLOCKS; ++b) {
                const uint32_t byte = row[t * BLOCKS + b];
                if (FMT == kMxfp4 ? byte == 255u : (byte & 0x7fu) == 0x7fu) blocks |= 1u << b;
            }
        }
    }
    const int64_t part = ((int64_t)blockIdx.z * (a.b.tokens * a.heads) + token * a.heads + h) * WIDTH;
    T* out = static_cast<T*>(a.out) + token * a.ot + h * a.oh;
    for (int d = 0; d < a.c.dim; ++d) {
        if (!(blocks >> (d / BLOCK) & 1)) continue;
        if (cut) a.sums[part + d] = not_a_number();
        else out[d] = from_float<T>(not_a_number());
    }
}

// The power of two that a query row of bfloat16 is divided by: its largest element (0 where that is) comes to [2^11, 2^12).
template <typename T>
__device__ __forceinline__ int query_exponent(const T* src, int dim, bool vec, bool have) {
    uint32_t most = 0;
    if (have) {
        if (vec) {
            for (int d = 0; d + 8 <= dim; d += 8) {
                const uint4 raw = *reinterpret_cast<const uint4*>(src + d);
                const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t bits = __float_as_uint(to_float<T>(t[j])) & 0x7fffffffu;
                    most = max(most, bits < kInfBits ? bits : 0u);
                }
            }
        }
        for (int d = vec ? dim / 8 * 8 : 0; d < dim; ++d) {
            const uint32_t bits = __float_as_uint(to_float<T>(src[d])) & 0x7fffffffu;
            most = max(most, bits < kInfBits ? bits : 0u);
        }
    }
    return max((int)(most >> 23) - 127 - 11, -126);
}

// A row's softmax: l = sum 2^(s - m), and its sums in tensor memory are times 2^(m + exponent).
struct RowState {
    float m, l;
    int exponent;
};
// The row's output, or its part.
template <typename T, int WIDTH, int FMT>
__device__ __forceinline__ void store_row(const AttendArgs& a, const RowState& row, int p, int64_t token, int64_t h, bool have, bool cut, bool summed, uint32_t o_at) {
    const float R = (float)row.exponent;
    const int64_t part = (int64_t)blockIdx.z * (a.b.tokens * a.heads) + token * a.heads + h;
    const Finish z = finish_of(R, row.l, kLift + lift_of<FMT>(), p >= 0);
    if (cut && have) a.part[part] = make_float4(row.m, R, row.l, p >= 0 ? 1.0f : 0.0f);
#pragma unroll 1
    for (int c = 0; c < WIDTH; c += 32) {
        uint32_t v[32];
        if (summed) {
            tc5::ld32(o_at + c, v);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        if (have) {
            if (cut) {
                float4* to = reinterpret_cast<float4*>(a.sums + part * WIDTH + c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    to[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
            } else {
                T* out = static_cast<T*>(a.out) + token * a.ot + h * a.oh;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    float y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = p < 0 ? 0.0f : __uint_as_float(v[i + k]) * z.x * z.x * z.inverse;
                    if (a.vec_out && c + i + 8 <= a.c.dim) {
                        store8(out + c + i, y);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (c + i + k < a.c.dim) out[c + i + k] = from_float<T>(y[k]);
                    }
                }
            }
        }
        __syncwarp();
    }
}

__device__ __forceinline__ uint32_t word_of(const uint32_t (&w)[4], int i) { return i < 2 ? i < 1 ? w[0] : w[1] : i < 3 ? w[2] : w[3]; }

// A tile's step for a row of any scores and values.  Scores are rounded before the reference is subtracted, so that
// nothing is lost beside large ones, and the references are of what the row sees: m follows its largest score, the
// exponent its largest score with the tile's values, unless what O holds is far above it.  exponent: of the tile's
// values; seen: bits of its tokens; lost: its groups without a page.
template <int WIDTH, bool REST>
__device__ __forceinline__ void careful_step(RowState& row, float f, int exponent, const uint32_t (&seen)[4], uint32_t lost, uint32_t s_at, uint32_t o_at, bool first) {
    // 16 scores from the c-th on
    const auto load_scores = [&](int c, float (&s)[16]) {
        uint32_t v[16];
        load_tmem16(s_at + c, v);
        const uint32_t bits = word_of(seen, c / 32) >> (c % 32);
        const bool gone = lost >> (c / 16) & 1u;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = bits >> i & 1u ? (gone ? not_a_number() : __uint_as_float(v[i]) * f) : minus_infinity();
    };
    float top = minus_infinity();
#pragma unroll 1
    for (int c = 0; c < 128; c += 16) {
        float s[16];
        load_scores(c, s);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[i]);
    }
    top = ceilf(top);
    const float m = fmaxf(row.m, top), sub = reference(m);
    const float own = (top - sub) + (float)exponent, before = first ? minus_infinity() : relative((float)row.exponent, row.m, m);
    float most = 0.0f;
    if (!first) {
#pragma unroll 1
        for (int c = 0; c < WIDTH; c += 16) {
            uint32_t v[16];
            load_tmem16(o_at + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(__uint_as_float(v[i])));
        }
    }
    // O stays below 2^100, beside which new terms (below 2^40) may vanish
    const float least = most > 0.0f ? before + (float)((int)(__float_as_uint(most) >> 23) - 227) : minus_infinity();
    float R = top == minus_infinity() ? before : fmaxf(own, least);
    R = R > -0x1p20f ? R : top == minus_infinity() ? (float)exponent : -0x1p20f;  // (the former: nothing seen so far)
    if (!first) {
        const float2 turn = exp2_factors((int)fminf(fmaxf(before - R, -200.0f), 200.0f));
#pragma unroll 1
        for (int c = 0; c < WIDTH; c += 16) {
            uint32_t v[16];
            load_tmem16(o_at + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * turn.x * turn.y);
            store_tmem16(o_at + c, v);
        }
    }
    const float up = (float)exponent - R + kLift;
    float sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        uint32_t w[16], rest[16];
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
            float s[16];
            load_scores(c + k, s);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float t0 = s[i] - sub, t1 = s[i + 1] - sub;
                sum += power2(t0) + power2(t1);
                const float u0 = power2(t0 + up), u1 = power2(t1 + up);
                const uint32_t h = half2_of(u0, u1);
                w[(k + i) / 2] = h;
                if (REST) {
                    const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h));
                    rest[(k + i) / 2] = half2_of(u0 - back.x, u1 - back.y);
                }
            }
        }
        store_tmem16(s_at + c, w);
        if (REST) store_tmem16(s_at + c + 16, rest);
    }
    row = RowState{m, fmaf(row.l, power2(row.m - sub), sum), (int)R};
}

// An item (or its part of n tiles) again from the start, of any scores and exponents of rows, by the softmax's warps
// alone and one step after the other: a tile's tokens in as many passes as leave each pass keys, and values, within
// 2^kSpread of one another, so that no row's bits depend on another's size, seen or not.  About three times the time
// of the loops; a pass more a tile for each 2^kSpread.
template <typename T, int WIDTH, int FMT>
__device__ __forceinline__ void careful_item(const AttendArgs& a, const Item& item, const Groups& groups, int head, int t0, int n, uint32_t base, uint32_t tmem,
                                          uint32_t done, int16_t (*exponents)[128], bool cut) {
    using S = Shape<WIDTH>;
    constexpr bool REST = std::is_same_v<T, __half>;
    constexpr int THREADS = 128 * S::NQ, PIECES = S::PIECES, BLOCK = mx4_block(FMT), BLOCKS = WIDTH / BLOCK;
    const int thread = threadIdx.x, warp = uniform_warp(), lane = thread & 31, x = warp / 4;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t s_at = tmem + S::S_COL + x * S::BUFFERS * 128 + lanes, o_at = tmem + S::O_COL + x * WIDTH + lanes;
    const bool have = thread < item.columns;
    const int query = item.column + thread, p = have ? item.length - item.tokens + query / a.group : -1;
    float factor = fabsf(a.scale);
    if (!REST) {
        const T* const q = static_cast<const T*>(a.q) + (have ? (item.first_token + query / a.group) * a.qt + (int64_t)(head * a.group + query % a.group) * a.qh : 0);
        factor = scale_by_exp2(factor, query_exponent(q, a.c.dim, a.vec_q, have));
    }
    RowState row{p >= 0 ? minus_infinity() : 0.0f, 0.0f, 0};
    uint32_t phase = 0;
    bool ok = true, first = true;
    const auto meet = [] { asm volatile("bar.sync 2, %0;" ::"n"(THREADS) : "memory"); };
    // MMAs of one thread behind everyone's writes, and everyone behind the MMAs.  Who gave up a wait once waits no more,
    // and meets the others all the same.
    const auto with_mmas = [&](auto issue) {
        tc5::fence_before_sync();
        meet();
        if (warp == 0) {
            tc5::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < S::NQ; ++i) issue(i);
                tc5::commit(done);
            }
            __syncwarp();
        }
        ok = ok && warp_wait(done, phase, kWaitNs);
        phase ^= 1;
        tc5::fence_after_sync();
    };
    const auto row_of = [&](int tile, int t, int kv) -> int64_t {  // of a token in the cache, -1 where there is none
        const int g = (t0 + tile) * 8 + t / 16, token = group_token(groups, g) + t % 16;
        const int page = g < groups.count && token < item.length ? page_of(a.c, a.b, item.sequence, token) : -1;
        return page < 0 ? -1 : cache_row(a.c, page, kv, head, token & (a.c.page_size - 1));
    };
    for (int tile = 0; tile < n; ++tile) {
        for (int i = thread; i < 256; i += THREADS) {
            const int64_t r = row_of(tile, i % 128, i / 128);
            exponents[i / 128][i % 128] = r < 0 ? kNoToken : a.c.exponents[r];
        }
        const int g = (t0 + tile) * 8 + lane % 8;
        const uint32_t bad = __ballot_sync(~0u, lane < 8 && g < groups.count && page_of(a.c, a.b, item.sequence, group_token(groups, g)) < 0);
        meet();
        int ke[4], ve[4];
        uint32_t left[4], rest;  // tokens still to come; every warp finds the same
#pragma unroll
        for (int i = 0; i < 4; ++i) ke[i] = exponents[0][32 * i + lane], ve[i] = exponents[1][32 * i + lane], left[i] = ~0u;
        do {
            const auto within = [](int e, int most) { return e <= -127 || most - e <= kSpread; };  // zeros and no tokens: with any
            int key = kNoToken, value = kNoToken;
#pragma unroll
            for (int i = 0; i < 4; ++i) key = max(key, left[i] >> lane & 1u ? ke[i] : kNoToken);
            key = __reduce_max_sync(~0u, key);
#pragma unroll
            for (int i = 0; i < 4; ++i) value = max(value, (left[i] >> lane & 1u) && within(ke[i], key) ? ve[i] : kNoToken);
            value = __reduce_max_sync(~0u, value);
            uint32_t now[4];
            rest = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                now[i] = __ballot_sync(~0u, (left[i] >> lane & 1u) && within(ke[i], key) && within(ve[i], value));
                left[i] &= ~now[i];
                rest |= left[i];
            }
            key = max(key, -127);
            value = max(value, -127);
#pragma unroll 1
            for (int i = thread; i < 256 * PIECES; i += THREADS) {
                const int kv = i / (128 * PIECES), t = i / PIECES % 128, part = i % PIECES;
                const int o = exponents[kv][t];
                uint4 codes = make_uint4(0, 0, 0, 0);
                uint32_t s[2] = {0, 0};
                if (o != kNoToken && word_of(now, t / 32) >> (t % 32) & 1u) {
                    const int64_t r = row_of(tile, t, kv);
                    codes = fetch16(a.c.codes + r * (WIDTH / 2) + part * 16);
                    const uint8_t* const scales = a.c.scales + r * BLOCKS + part * (32 / BLOCK);
                    piece_scales<FMT>(FMT == kMxfp4 ? fetch1(scales) : fetch2(scales), o, lift_of<FMT>() - (kv ? value : key) - (FMT == kMxfp4 ? 127 : 0),
                                      inside_of<BLOCK>(part, a.c.dim), kv, s);
                }
                store_piece(base + (kv ? S::V0 : S::K0) + piece_place(part, t, S::BLOCK_BYTES), codes, s);
            }
            fence_async();
            with_mmas([&](int i) { issue_scores<WIDTH>(tmem + S::S_COL + i * S::BUFFERS * 128, base + i * S::TILE_BYTES, base + S::K0); });
            uint32_t seen[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) seen[i] = now[i] & seen_bits(groups, p, a.window, a.sinks, (t0 + tile) * 8 + 2 * i);
            careful_step<WIDTH, REST>(row, fmaxf(factor * key_factor_of<FMT>(key), 0x1p-120f), value, seen, bad, s_at, o_at, first);
            wait_tmem_stores();
            with_mmas([&](int i) { issue_sums<WIDTH, REST>(tmem + S::O_COL + i * WIDTH, tmem + S::S_COL + i * S::BUFFERS * 128, base + S::V0, !first); });
            first = false;
        } while (rest != 0);
    }
    if (!ok && lane == 0) atomicAdd(&g_attend_timeouts, 1u);
    store_row<T, WIDTH, FMT>(a, row, p, item.first_token + query / a.group, head * a.group + query % a.group, have, cut, ok, o_at);
}

// The two ways in which the kernel calls it.  A call costs its loops registers, more or fewer by what is held over them
// (us, against a copy without: 8192 tokens of width 128: 532; all found anew 539, handed over 550; chunks of width 256:
// 339; 351 and 344; a kernel of its own behind this one: 5 us more for every call, 22 for 17 of 60 tokens).
template <typename T, int WIDTH, int FMT>
__device__ __noinline__ void careful_item_anew(const AttendArgs& a, uint32_t smem, const uint32_t* tmem_slot, uint32_t done, int16_t (*exponents)[128]) {
    const int head = (int)(blockIdx.x % a.c.heads);
    const Item item = item_of(a, (int64_t)((gridDim.x - 1 - blockIdx.x) / a.c.heads), 128 * Shape<WIDTH>::NQ);
    const int before = item.length - item.tokens;
    const Groups groups = groups_of(a.c, a.b, before + item.column / a.group, before + (item.column + item.columns - 1) / a.group, a.window, a.sinks);
    const int tiles = (groups.count + 7) / 8, parts = parts_of(tiles, a.splits);
    const int t0 = (int)((unsigned)tiles * blockIdx.z / (unsigned)parts), t1 = (int)((unsigned)tiles * (blockIdx.z + 1) / (unsigned)parts);
    careful_item<T, WIDTH, FMT>(a, item, groups, head, t0, t1 - t0, (smem + 1023u) & ~1023u, *tmem_slot, done, exponents, parts > 1);
}
template <typename T, int WIDTH, int FMT>
__device__ __noinline__ void careful_item_handed(const AttendArgs& a, const Item& item, const Groups& groups, int head, int t0, int n, uint32_t base, uint32_t tmem,
                                                 uint32_t done, int16_t (*exponents)[128], bool cut) {
    careful_item<T, WIDTH, FMT>(a, item, groups, head, t0, n, base, tmem, done, exponents, cut);
}

template <typename T, int WIDTH, int FMT>
__global__ void __launch_bounds__(Shape<WIDTH>::THREADS, 1) attend_tile_kernel(const AttendArgs a) {
    using S = Shape<WIDTH>;
    constexpr bool REST = std::is_same_v<T, __half>;  // what the rounding of weights leaves enters the sum too
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ __align__(8) Barriers bars;
    __shared__ uint32_t tmem_slot;
    __shared__ TileInfo info[kRing];
    __shared__ int rows[kRing][8];  // of groups of keys, in 16s, -1 where there is no page
    __shared__ int16_t exponents[kRing][2][128];  // of keys and values
    __shared__ int any_nan;                       // in values
    __shared__ bool cut;                          // the item has other parts (here, not in a register all the way: 13 us less of 560, 8192 tokens)
    __shared__ __align__(16) int largest[2][2][4];  // of the tiles in turn
    __shared__ bool far_rows, large_scores;         // what the loops are not for

    pdl_wait();
    pdl_launch_dependents();
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int head = (int)(blockIdx.x % a.c.heads);
    // the last rows of a sequence see the most tokens: they go first
    const Item item = item_of(a, (int64_t)((gridDim.x - 1 - blockIdx.x) / a.c.heads), 128 * S::NQ);
    if (item.sequence < 0) return;
    const int before = item.length - item.tokens;
    const auto position = [&](int column) { return before + (item.column + column) / a.group; };
    const int p0 = position(0), p1 = position(item.columns - 1);
    const Groups groups = groups_of(a.c, a.b, p0, p1, a.window, a.sinks);
    const int tiles = (groups.count + 7) / 8;
    const int parts = parts_of(tiles, a.splits);
    if ((int)blockIdx.z >= parts) return;
    if (threadIdx.x == 0) cut = parts > 1;
    // up to 2^24 tiles, 64 parts
    const int t0 = (int)((unsigned)tiles * blockIdx.z / (unsigned)parts), t1 = (int)((unsigned)tiles * (blockIdx.z + 1) / (unsigned)parts);
    // tiles that the rows of tile x see, counted from t0
    int need[2] = {0, 0};
#pragma unroll
    for (int x = 0; x < S::NQ; ++x) {
        if (item.columns > x * 128) {
            const int last = position(min(item.columns, (x + 1) * 128) - 1);
            const int count = last < 0 ? 0 : min(groups.count, groups.sink + max(0, last / 16 + 1 - groups.low));
            need[x] = max(0, min((count + 7) / 8, t1) - t0);
        }
    }
    const int n = max(need[0], need[1]);

    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_full = smem_addr(&bars.q), done = smem_addr(&bars.done);
    const auto bar = [&](uint64_t* b, int i) { return smem_addr(b) + 8u * (uint32_t)i; };
    if (threadIdx.x == 0) {
        mbar_init(q_full, 4 * S::NQ);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(bars.k_full, i), S::CONVERTERS / 32);
            mbar_init(bar(bars.v_full, i), S::CONVERTERS / 32);
            mbar_init(bar(bars.k_empty, i), 1);
            mbar_init(bar(bars.v_empty, i), 1);
            mbar_init(bar(bars.s, i), 1);
            mbar_init(bar(bars.p, i), 4);
            mbar_init(bar(bars.o, i), 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar(bars.info, i), 1);
        }
        mbar_init(done, 1);
        mbar_init(smem_addr(&bars.careful), 1);
        any_nan = 0;
        far_rows = large_scores = false;
        fence_barrier_init();
    }
    if (warp == S::MMA_WARP) {
        tc5::tmem_alloc(smem_addr(&tmem_slot), 512);
        tc5::tmem_relinquish();
    }
    tc5::fence_before_sync();
    __syncthreads();
    tc5::fence_after_sync();
    const uint32_t tmem = tmem_slot;

    if (warp < 4 * S::NQ) {
        // ---- softmax: a thread for a row ----
        more_registers<S::SOFTMAX_REGS>();
        const int x = warp / 4, quarter = warp % 4, row = quarter * 32 + lane;
        const int column = x * 128 + row;
        const bool have = column < item.columns;
        const int p = have ? position(column) : -1;
        const int first = position(x * 128), last = position(min(item.columns, (x + 1) * 128) - 1);
        const int query = item.column + column;
        const int64_t token = item.first_token + query / a.group, h = head * a.group + query % a.group;
        float factor = fabsf(a.scale);
        {   // the row into shared memory, 64 elements (128 bytes, swizzled) at a time
            const T* src = static_cast<const T*>(a.q) + (have ? token * a.qt + h * a.qh : 0);
            const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
            float2 up = make_float2(sign, 1.0f);
            if (!REST) {
                const int e = query_exponent(src, a.c.dim, a.vec_q, have);
                const float2 down = exp2_factors(e);
                up = exp2_factors(-e);
                up.x *= sign;
                factor = factor * down.x * down.y;
            }
            const uint32_t q = base + x * S::TILE_BYTES + row * 128;
#pragma unroll 4
            for (int d = 0; d < WIDTH; d += 8) {
                float v[8];
                if (have && a.vec_q && d + 8 <= a.c.dim) {
                    const uint4 raw = *reinterpret_cast<const uint4*>(src + d);
                    const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = to_float<T>(t[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = have && d + j < a.c.dim ? to_float<T>(src[d + j]) : 0.0f;
                }
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = half2_of(v[2 * j] * up.x * up.y, v[2 * j + 1] * up.x * up.y);
                store_shared(q + d / 64 * S::BLOCK_BYTES + (uint32_t)((d / 8 % 8 ^ row % 8) << 4), make_uint4(w[0], w[1], w[2], w[3]));
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t o_at = tmem + S::O_COL + x * WIDTH + lanes;
        float m = p >= 0 ? minus_infinity() : 0.0f, l = 0.0f;
        int reference_exponent = 0;
        bool ok = true;
        const int mine = need[x];
        for (int j = 0; j < mine; ++j) {
            const int buffer = x * S::BUFFERS + j % S::BUFFERS;
            const uint32_t s_at = tmem + S::S_COL + buffer * 128 + lanes;
            ok = warp_wait(bar(bars.info, j % kRing), (j / kRing) & 1, kWaitNs);
            ok = ok && warp_wait(bar(bars.s, buffer), (j / S::BUFFERS) & 1, kWaitNs);
            if (!ok) break;
            tc5::fence_after_sync();
            const TileInfo& tile = info[j % kRing];
            const float f = fmaxf(factor * tile.key_factor, 0x1p-120f);  // no 0: minus infinity stays what it is
            const int g0 = (t0 + j) * 8;
            const int begin = group_token(groups, g0), end = group_token(groups, g0 + 7) + 15;
            const bool whole = tile.bad == 0 && g0 + 8 <= groups.count && end <= first && (a.window == 0 || begin > last - a.window);
            // scores of what is not seen become minus infinity, of tokens without a page NaN
            const auto mask = [&](int c, uint32_t (&s)[32]) {
                const uint32_t bits = seen_bits(groups, p, a.window, a.sinks, g0 + c / 16), lost = tile.bad >> (c / 16);
                const uint32_t nan = (lost & 1u ? 0xffffu : 0u) | (lost & 2u ? 0xffff0000u : 0u);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = bits >> i & 1u ? (nan >> i & 1u ? 0x7fc00000u : s[i]) : 0xff800000u;
            };
            // The values' exponent first: it is the same for all rows.
            int shift = tile.value_exponent - reference_exponent;
            float turn = 1.0f;  // what O has to be multiplied by
            if (j == 0) {
                reference_exponent = tile.value_exponent;
                shift = 0;
            } else if (shift > kShift || shift < -kShift) {
                const float2 t = exp2_factors(-shift);
                turn = t.x * t.y;
                reference_exponent = tile.value_exponent;
                shift = 0;
            }
            // 32 scores at a time, in one pass: weights by the reference m so far.  Where they come out above kMost
            // (or there is no reference yet), m becomes the largest score, up to a whole number: the weights that are
            // there already change by a power of two.
            float offset = (float)shift + kLift - reference(m), sum = 0.0f;
            const uint64_t ff = pack_pair(f, f);
            uint32_t ring[2][32];  // one half is loaded while the other is worked on
            start_load32(s_at, ring[0]);
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                uint32_t w[16], rest[16];
                uint32_t(&s)[32] = ring[c / 32 & 1];
                wait_tmem_loads(s);
                if (c < 96) start_load32(s_at + c + 32, ring[c / 32 & 1 ^ 1]);
                if (!whole) mask(c, s);
                float part;
                const auto weights = [&]() {
                    const uint64_t oo = pack_pair(offset, offset);
                    uint64_t sums2[2] = {pack_pair(0.0f, 0.0f), pack_pair(0.0f, 0.0f)};
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float u, v;
                        unpack_pair(fma_pair(pack_pair(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), ff, oo), u, v);
                        u = power2(u);
                        v = power2(v);
                        sums2[i / 2 & 1] = add_pair(sums2[i / 2 & 1], pack_pair(u, v));
                        w[i / 2] = half2_of(u, v);
                        if (REST) {
                            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
                            rest[i / 2] = half2_of(u - back.x, v - back.y);
                        }
                    }
                    float other;
                    unpack_pair(add_pair(sums2[0], sums2[1]), part, other);
                    part += other;
                };
                weights();
                if (__any_sync(~0u, part > kMost || m == minus_infinity())) {
                    float tops[4] = {minus_infinity(), minus_infinity(), minus_infinity(), minus_infinity()};
#pragma unroll
                    for (int i = 0; i < 32; ++i) tops[i & 3] = fmaxf(tops[i & 3], __uint_as_float(s[i]));
                    const float top = ceilf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * f);
                    const float by = top > m ? power2(m - top) : 1.0f;
                    m = top > m ? top : m;
                    if (fabsf(m) >= kMostScore && fabsf(m) < -minus_infinity()) large_scores = true;
                    l *= by;
                    sum *= by;
                    turn *= by;
                    offset = (float)shift + kLift - reference(m);
                    if (c < 96) wait_tmem_loads(ring[c / 32 & 1 ^ 1]);  // no load is in flight over a call
                    const uint32_t half = half2_of(by, by);
#pragma unroll 1
                    for (int d = 0; d < c; d += 32) {
                        // a call costs the other loops registers (8192 tokens of width 128: 572 us, 535 so); of width 256
                        // it is the other way round (chunks: 339, 346)
                        if constexpr (S::NQ == 2) follow_weights<REST>(s_at + d, half);
                        else call_follow_weights<REST>(s_at + d, half);
                    }
                    weights();
                }
                sum += part;
                store_tmem16(s_at + c, w);
                if (REST) store_tmem16(s_at + c + 16, rest);
            }
            // The scores were there after the sum of BUFFERS tiles before.  That of the tile before has to be there too
            // where O is to change, and of the last tile, so that one phase at most is open behind the loop.
            const bool change = j > 0 && __any_sync(~0u, turn != 1.0f);
            if (change || (j > 0 && j == mine - 1)) {
                ok = warp_wait(bar(bars.o, x), (j - 1) & 1, kWaitNs);
                if (!ok) break;
                tc5::fence_after_sync();
            }
            if (change) {
#pragma unroll 1
                for (int c = 0; c < WIDTH; c += 16) {
                    uint32_t v[16];
                    load_tmem16(o_at + c, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * turn);
                    store_tmem16(o_at + c, v);
                }
            }
            l = fmaf(sum, exp2_int(-shift - (int)kLift), l);
            wait_tmem_stores();
            tc5::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bars.p, buffer));
        }
        if (ok && mine > 0) {
            ok = warp_wait(bar(bars.o, x), (mine - 1) & 1, kWaitNs);
            tc5::fence_after_sync();
        }
        if (!ok && lane == 0) atomicAdd(&g_attend_timeouts, 1u);
        store_row<T, WIDTH, FMT>(a, RowState{m, l, reference_exponent}, p, token, h, have, cut, mine > 0 && ok, o_at);
        tc5::fence_before_sync();
    } else if (warp < S::MMA_WARP) {
        // ---- codes to 16 bits ----
        fewer_registers<S::CONVERT_REGS>();
        constexpr int PIECES = S::PIECES, PASSES = S::PASSES, BLOCK = mx4_block(FMT), BLOCKS = WIDTH / BLOCK;
        const int thread = threadIdx.x - 4 * S::NQ * 32;
        // In a pass the thread has 32 codes of token t, the part-th of it.  8 lanes in a row have 4 tokens and
        // 2 parts: their 16-byte pieces lie on different banks, and a warp's codes are contiguous all the same.
        constexpr int LOG = PIECES == 2 ? 1 : PIECES == 4 ? 2 : 3;
        const int part = (lane & 1) | (lane >> 3 & (PIECES / 2 - 1)) << 1;
        const int t = (thread >> 5) * (32 >> LOG) + ((lane >> 1 & 3) | lane >> (2 + LOG) << 2);
        // the page table's entry for group thread % 8 of tile j, -1 where it has none, and the row of the keys
        // of the group's first token; an entry is read a tile before it is looked at
        const auto page_for = [&](int j) {
            const int g = (t0 + j) * 8 + thread;
            if (j >= n || g >= groups.count) return -1;
            const int at = group_token(groups, g) >> a.c.page_shift;
            return at < a.b.table_pages ? fetch4(a.b.table + item.sequence * a.b.ld_table + at) : -1;
        };
        const auto row_for = [&](int j, int page) {
            return page < 0 || page >= a.c.pages
                       ? -1
                       : (int)(cache_row(a.c, page, 0, head, group_token(groups, (t0 + j) * 8 + thread) & (a.c.page_size - 1)) / 16);
        };
        const int to_values = a.c.heads * (a.c.page_size / 16);  // rows from a key to its value, in 16s
        int held = -1;
        if (thread < 8) {
            const int first_page = page_for(0), second_page = page_for(1);
            held = page_for(2);
            rows[0][thread] = row_for(0, first_page);
            rows[1][thread] = row_for(1, second_page);
        }
        asm volatile("bar.sync 1, %0;" ::"n"(S::CONVERTERS) : "memory");
        const uint8_t* const code_base = a.c.codes + (t % 16) * (WIDTH / 2) + part * 16;
        const uint8_t* const scale_base = a.c.scales + (t % 16) * BLOCKS + part * (32 / BLOCK);
        // of exponents a thread has one: a key's (threads 0 to 127) or a value's (128 to 255)
        const int kv = thread / 128, et = thread % 128;
        const bool has_exponent = S::CONVERTERS == 256 || kv < 2;
        const int8_t* const exponent_base = a.c.exponents + (kv ? (int64_t)to_values * 16 : 0) + et % 16;
        // tokens of the tiles from t0 on, up to the end of the sequence (only the last group reaches beyond it)
        const int tokens = groups.count > 0 ? (groups.count - 1) * 16 + min(16, item.length - group_token(groups, groups.count - 1)) - t0 * 128 : 0;
        Raw<PASSES> keys, values;  // the ones are loaded while the others are converted
        int exponent = kNoToken;   // of the next tile
        const auto load = [&](int j, int add, Raw<PASSES>& raw) {
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {  // what is not there is read from the first page: its scale becomes 0
                const uint32_t r = (uint32_t)(max(rows[j & (kRing - 1)][i * (S::PER_PASS / 16) + t / 16], 0) + add);
                raw.codes[i] = fetch16(code_base + (uint64_t)r * (16 * WIDTH / 2));
                raw.scales[i] = FMT == kMxfp4 ? fetch1(scale_base + (uint64_t)r * (16 * BLOCKS)) : fetch2(scale_base + (uint64_t)r * (16 * BLOCKS));
            }
        };
        const auto load_exponent = [&](int j) {
            const int r = rows[j & (kRing - 1)][et / 16];
            exponent = kNoToken;
            if (has_exponent && r >= 0 && j * 128 + et < tokens) exponent = fetch_signed1(exponent_base + (uint64_t)(uint32_t)r * 16);
        };
        const uint32_t inside = inside_of<BLOCK>(part, a.c.dim);
        const uint32_t place = base + piece_place(part, t, S::BLOCK_BYTES);
        bool ok = true;
        int key_exponent = 0, value_exponent = 0, next_value_exponent = -127;
        const auto convert = [&](int j, bool value, int e, const Raw<PASSES>& raw) {
            const int stage = j % S::STAGES;
            const int16_t* const own = exponents[j & (kRing - 1)][value ? 1 : 0];
            const uint32_t to = place + (value ? S::V0 : S::K0) + stage * S::TILE_BYTES;
            const int add = lift_of<FMT>() - e - (FMT == kMxfp4 ? 127 : 0);
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                uint32_t s[2];
                if (piece_scales<FMT>(raw.scales[i], own[i * S::PER_PASS + t], add, inside, value, s)) any_nan = 1;
                store_piece(to + i * S::PER_PASS * 128, raw.codes[i], s);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(value ? bars.v_full : bars.k_full, stage));
        };
        // A warp that gave up a wait once goes on without waiting: the others meet it at the barrier.
        const auto convert_keys = [&](int j, bool with_values) {
            const int slot = j & (kRing - 1);
            ok = ok && warp_wait(bar(bars.k_empty, j % S::STAGES), ((j / S::STAGES) & 1) ^ 1, kWaitNs);
            // the scores of tile j - 2 are there: the softmax has done with tile j - 4, whose slot this is
            if (has_exponent) {
                exponents[slot][kv][et] = (int16_t)exponent;
                const int top = __reduce_max_sync(~0u, exponent);
                if (lane == 0) largest[j & 1][kv][et / 32] = top;
            }
            asm volatile("bar.sync 1, %0;" ::"n"(S::CONVERTERS) : "memory");
            if (with_values) load(j - 1, to_values, values);
            const int4 a0 = *reinterpret_cast<const int4*>(largest[j & 1][0]), a1 = *reinterpret_cast<const int4*>(largest[j & 1][1]);
            key_exponent = max(max(max(a0.x, a0.y), max(a0.z, a0.w)), -127);
            const int v = max(max(a1.x, a1.y), max(a1.z, a1.w));
            value_exponent = next_value_exponent;
            next_value_exponent = v > -127 ? v : value_exponent;  // zeros alone: as before
            if (thread / 32 == 1) {
                const uint32_t bad = __ballot_sync(~0u, lane < 8 && (t0 + j) * 8 + lane < groups.count && rows[slot][lane % 8] < 0);
                if (lane == 0) {
                    info[slot].key_factor = key_factor_of<FMT>(key_exponent);
                    info[slot].value_exponent = next_value_exponent;
                    info[slot].bad = bad;
                    mbar_arrive(bar(bars.info, slot));
                }
            }
            if (thread < 8) {  // rows of two tiles on, for loads behind the next barrier
                rows[(j + 2) & (kRing - 1)][thread] = row_for(j + 2, held);
                held = page_for(j + 3);
            }
            convert(j, false, key_exponent, keys);
        };
        if (n > 0) {
            load(0, 0, keys);
            load_exponent(0);
            convert_keys(0, false);
            if (n > 1) {
                load(1, 0, keys);
                load_exponent(1);
            }
            for (int j = 0; j < n; ++j) {  // K(j + 1), then V(j)
                if (j + 1 < n) {
                    convert_keys(j + 1, true);
                } else {
                    load(j, to_values, values);
                    value_exponent = next_value_exponent;
                }
                if (j + 2 < n) {
                    load(j + 2, 0, keys);
                    load_exponent(j + 2);
                }
                ok = ok && warp_wait(bar(bars.v_empty, j % S::STAGES), ((j / S::STAGES) & 1) ^ 1, kWaitNs);
                convert(j, true, value_exponent, values);
            }
        }
        if (!ok && lane == 0) atomicAdd(&g_attend_timeouts, 1u);
    } else if (fewer_registers<S::MMA_REGS>(); warp == S::MMA_WARP && n > 0) {
        // ---- MMAs ----
        const auto score = [&](int x, int j) {
            if (elect_one()) {
                const int buffer = x * S::BUFFERS + j % S::BUFFERS;
                issue_scores<WIDTH>(tmem + S::S_COL + buffer * 128, base + x * S::TILE_BYTES, base + S::K0 + j % S::STAGES * S::TILE_BYTES);
                tc5::commit(bar(bars.s, buffer));
            }
            __syncwarp();
        };
        const auto weigh = [&](int x, int j) {
            if (elect_one()) {
                const int buffer = x * S::BUFFERS + j % S::BUFFERS;
                issue_sums<WIDTH, REST>(tmem + S::O_COL + x * WIDTH, tmem + S::S_COL + buffer * 128, base + S::V0 + j % S::STAGES * S::TILE_BYTES, j != 0);
                tc5::commit(bar(bars.o, x));
            }
            __syncwarp();
        };
        const auto free_stage = [&](uint64_t* b, int j) {
            if (elect_one()) tc5::commit(bar(b, j % S::STAGES));
            __syncwarp();
        };
        const auto keys = [&](int j) { return warp_wait(bar(bars.k_full, j % S::STAGES), (j / S::STAGES) & 1, kWaitNs); };
        // scores go BUFFERS tiles ahead of the sums
        bool ok = warp_wait(q_full, 0, kWaitNs);
        for (int j = 0; j < S::BUFFERS && j < n && ok; ++j) {
            ok = keys(j);
            if (!ok) break;
            tc5::fence_after_sync();
            for (int x = 0; x < S::NQ; ++x)
                if (j < need[x]) score(x, j);
            free_stage(bars.k_empty, j);
        }
        for (int j = 0; j < n && ok; ++j) {
            const int ahead = j + S::BUFFERS;
            ok = warp_wait(bar(bars.v_full, j % S::STAGES), (j / S::STAGES) & 1, kWaitNs);
            for (int x = 0; x < S::NQ && ok; ++x) {
                if (j < need[x]) {
                    ok = warp_wait(bar(bars.p, x * S::BUFFERS + j % S::BUFFERS), (j / S::BUFFERS) & 1, kWaitNs);
                    if (!ok) break;
                    tc5::fence_after_sync();
                    weigh(x, j);
                }
                if (x == S::NQ - 1) free_stage(bars.v_empty, j);
                if (ahead < n) {
                    ok = keys(ahead);
                    if (!ok) break;
                    tc5::fence_after_sync();
                    if (ahead < need[x]) score(x, ahead);
                    if (x == S::NQ - 1) free_stage(bars.k_empty, ahead);
                }
            }
        }
        // every MMA has finished before shared or tensor memory is given up
        if (elect_one()) tc5::commit(done);
        __syncwarp();
        ok = warp_wait(done, 0, kWaitNs) && ok;
        if (!ok && lane == 0) atomicAdd(&g_attend_timeouts, 1u);
    } else if (warp == S::MMA_WARP + 1) {
        // ---- exponents far apart, which the loops are not for ----
        // 16 lanes for a tile: groups of 16 tokens, keys and values
        int most = -127, least = kNone, widest = 0;
        for (int j = lane / 16; j < n + lane / 16; j += 2) {
            const int kv = lane >> 3 & 1, g = (t0 + j) * 8 + lane % 8;
            int top = -127, low = kNone;
            if (j < n && g < groups.count) {
                const int token = group_token(groups, g), page = page_of(a.c, a.b, item.sequence, token);
                if (page >= 0) {
                    const uint4 v = fetch16(a.c.exponents + cache_row(a.c, page, kv, head, token & (a.c.page_size - 1)));
                    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
                    const int here = item.length - token;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int e = (int8_t)(words[i / 4] >> (8 * (i % 4)));
                        if (i < here && e > -127) {  // zeros are of any size
                            top = max(top, e);
                            low = min(low, e);
                        }
                    }
                }
            }
#pragma unroll
            for (int d = 1; d < 8; d *= 2) {
                top = max(top, __shfl_xor_sync(~0u, top, d));
                low = min(low, __shfl_xor_sync(~0u, low, d));
            }
            widest = max(widest, top - low);
            if (kv) most = max(most, top), least = min(least, low);
        }
        const bool far = __reduce_max_sync(~0u, widest) > kSpread || __reduce_max_sync(~0u, most) - __reduce_min_sync(~0u, least) > kReach;
        if (far && lane == 0) far_rows = true;
    }
    tc5::fence_before_sync();
    __syncthreads();
    tc5::fence_after_sync();
    if (far_rows || large_scores) {
        if (threadIdx.x < 128 * S::NQ) {
            if constexpr (S::NQ == 2) careful_item_anew<T, WIDTH, FMT>(a, smem_addr(smem_raw), &tmem_slot, smem_addr(&bars.careful), exponents[0]);
            else careful_item_handed<T, WIDTH, FMT>(a, item, groups, head, t0, n, base, tmem, smem_addr(&bars.careful), exponents[0], cut);
        }
        tc5::fence_before_sync();
        __syncthreads();
        tc5::fence_after_sync();
    }
    if (warp == S::MMA_WARP) {
        __syncwarp();
        tc5::tmem_dealloc(tmem, 512);
    }
    // Values that are NaN entered the sums as 0: where there were any, each row looks for those that it sees
    if (any_nan != 0 && threadIdx.x < 128 * S::NQ && (int)threadIdx.x < item.columns) {
        const int p = position(threadIdx.x), query = item.column + threadIdx.x;
        const int64_t token = item.first_token + query / a.group, h = head * a.group + query % a.group;
        const int x = threadIdx.x / 128;
        mark_nan<T, WIDTH, FMT>(a, item, groups, head, p, t0 * 8, min(groups.count, (t0 + need[x]) * 8), token, h, cut);
    }
}

template <typename T, int WIDTH, int FMT>
cudaError_t launch(const AttendArgs& a, cudaStream_t st) {
    using S = Shape<WIDTH>;
    auto* kernel = attend_tile_kernel<T, WIDTH, FMT>;
    static std::atomic<bool> asked[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!asked[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (err != cudaSuccess) return err;
        asked[dev].store(true, std::memory_order_relaxed);
    }
    const dim3 grid((unsigned)(a.c.heads * a.tiles(128 * S::NQ)), 1, (unsigned)a.splits);
    err = launch_pdl(kernel, grid, dim3(S::THREADS), S::SMEM, st, a);
    if (err != cudaSuccess || a.splits == 1) return err;
    return launch_attend_join(a, std::is_same_v<T, __half> ? DDGEMM_F16 : DDGEMM_BF16, kLift + lift_of<FMT>(), st);
}
template <typename T>
cudaError_t by_width(const AttendArgs& a, cudaStream_t st) {
    if (a.c.fmt == kMxfp4) return a.c.width == 64 ? launch<T, 64, kMxfp4>(a, st) : a.c.width == 128 ? launch<T, 128, kMxfp4>(a, st) : launch<T, 256, kMxfp4>(a, st);
    return a.c.width == 64 ? launch<T, 64, kNvfp4>(a, st) : a.c.width == 128 ? launch<T, 128, kNvfp4>(a, st) : launch<T, 256, kNvfp4>(a, st);
}

}  // namespace

// Enough items for two rounds of the SMs are left whole; fewer are cut so that there are
// up to four rounds of parts, of 512 tokens at least: lengths differ, and a part's start
// costs 3 us.  The host knows the longest sequence that the page table has room for; how
// many parts an item has goes by its own length, on the device (512 tokens of a prompt
// with a table for 8192: 85 us in equal parts of every row).
int attend_tile_parts(const AttendArgs& a) {
    const int rows = a.c.width == 256 ? 128 : 256;
    // sequences that may be taken, if each has a token at least
    int64_t batch = a.b.batch, tokens = a.b.tokens;
    if (a.above > a.group) {
        batch = std::max<int64_t>(1, std::min(batch, (tokens - batch) * a.group / (a.above + 1 - a.group)));
        tokens -= a.b.batch - batch;
    }
    const int64_t items = std::max(tokens * a.group / rows, batch) * a.c.heads;
    const int64_t longest = a.window > 0 ? (int64_t)a.window + a.sinks : (int64_t)a.b.table_pages * a.c.page_size;
    if (items >= 2 * device_sms()) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({4 * device_sms() / std::max<int64_t>(1, items), (longest + 511) / 512, 64}));
}

cudaError_t launch_attend_tile(const AttendArgs& a, int type, cudaStream_t st) {
    return type == DDGEMM_BF16 ? by_width<__nv_bfloat16>(a, st) : by_width<__half>(a, st);
}

cudaError_t read_and_reset_wait_timeouts_attend(unsigned int* count) {
    cudaError_t err = cudaDeviceSynchronize();
    if (err != cudaSuccess) return err;
    err = cudaMemcpyFromSymbol(count, g_attend_timeouts, sizeof(unsigned int));
    if (err != cudaSuccess) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_attend_timeouts, &zero, sizeof(unsigned int));
}

}  // namespace ddg
