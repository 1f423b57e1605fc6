// attend.cu -- attention over the 4-bit cache for few queries, and the sum of parts.
//
// Few queries of a key/value head (a token's group of heads, a few proposed tokens)
// read the whole cache: the floor is its bytes.  A warp takes 16 tokens at a time,
// straight from global memory into the registers of mma.sync fragments: scores as
// S^T = K Q^T (16 tokens by 8 queries), the sum as O^T = V^T P^T, so that 8 queries
// fill an instruction that 16 rows of queries would leave half empty, and the codes
// of a row are contiguous in a thread.  (tcgen05 wants its operands in shared memory
// and 128 rows: each 4-bit row would be written there in 16 bits and read again,
// four times its bytes, for a product that uses 8 of the columns.)
//
// The codes become 16-bit floating point by one conversion for two, the block's
// scale one packed multiplication for two, exactly: E4M3 times E2M1 has 6 bits;
// mxfp4 scales are relative to the row's largest, times 2^13 (a block 2^27 below it
// counts as 0, below the rounding of the 32-bit sum).  Queries are scaled by a power
// of two into the range of 16 bits; what they lose is 2^-36 of their row's largest.
// Weights are rounded to 16 bits (11 significant) for bfloat16 outputs, and what that
// leaves enters the sum too for float16 ones, whose own rounding is as small.
#include <algorithm>

#include "attend.cuh"

namespace ddg {
namespace {

constexpr int kWarps = 4;
constexpr float kLag = 8.0f;    // references follow when they are exceeded by more than 2^8
constexpr float kLift = 7.0f;   // weights are up to 2^(8 + 7), below the largest float16
constexpr int kMxLift = 13;     // mxfp4 scales relative to the row's largest, times 2^13

__device__ __forceinline__ uint32_t half2_of(float a, float b) {  // a in the low half
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
__device__ __forceinline__ float low_half(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float high_half(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
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

// A block's scale as the bits of a half: E4M3 is exact; E8M0 relative to 2^e.
template <int FMT>
__device__ __forceinline__ uint32_t half_scale(uint32_t byte, int e) {
    if (FMT == kNvfp4) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((unsigned short)byte));
        return h2 & 0xffffu;
    }
    const int t = (int)byte - e - 127 + kMxLift + 15;
    return byte == 255u ? 0x7fffu : (uint32_t)min(max(t, 0), 30) << 10;
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

template <int N>  // N words, aligned to their size up to 16 bytes
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        asm volatile("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    } else if constexpr (N == 2) {
        asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "l"(p + 4 * i));
    }
}

// What a lane (r, c) = (lane / 4, lane % 4) reads of a group of 16 tokens: of keys,
// a quarter c of tokens 2 r and 2 r + 1; of values, the eighth r of tokens 4 c .. 4 c + 3.
// Row i of the score fragment is token 2 (i % 8) + i / 8, so that both halves agree
// on the four tokens of a lane.
template <int WIDTH, int FMT>
struct Group16 {
    static constexpr int KW = WIDTH / 32, VW = WIDTH / 64;                 // words of codes of a token
    static constexpr int BLOCK = mx4_block(FMT), BLOCKS = WIDTH / BLOCK;
    static constexpr int KB = WIDTH / 4 / BLOCK > 0 ? WIDTH / 4 / BLOCK : 1;  // blocks a lane's codes touch
    static constexpr int VB = WIDTH / 8 / BLOCK > 0 ? WIDTH / 8 / BLOCK : 1;
    uint32_t k[2][KW], v[4][VW];
    uint8_t ks[2][KB], vs[4][VB];
    uint16_t ke;   // the two keys' exponents
    uint16_t vr;   // the two values' exponents of tokens 2 r, 2 r + 1
    uint32_t ve;   // the four values' (mxfp4)
    bool bad;      // no such page

    __device__ __forceinline__ void load(const CacheView& c, int page, int head, int offset, int lane) {
        bad = page < 0;
        if (bad) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < KW; ++i) k[t][i] = 0;
#pragma unroll
                for (int i = 0; i < KB; ++i) ks[t][i] = 0;
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
#pragma unroll
                for (int i = 0; i < VW; ++i) v[t][i] = 0;
#pragma unroll
                for (int i = 0; i < VB; ++i) vs[t][i] = 0;
            }
            ke = vr = 0;
            ve = 0;
            return;
        }
        const int r = lane / 4, q = lane % 4;
        const int64_t krow = cache_row(c, page, 0, head, offset), vrow = cache_row(c, page, 1, head, offset);
        const uint8_t* kc = c.codes + (krow + 2 * r) * (WIDTH / 2) + q * (WIDTH / 8);
        const uint8_t* vc = c.codes + (vrow + 4 * q) * (WIDTH / 2) + r * (WIDTH / 16);
#pragma unroll
        for (int t = 0; t < 2; ++t) load_words<KW>(kc + t * (WIDTH / 2), k[t]);
#pragma unroll
        for (int t = 0; t < 4; ++t) load_words<VW>(vc + t * (WIDTH / 2), v[t]);
        const uint8_t* ksp = c.scales + (krow + 2 * r) * BLOCKS + q * (WIDTH / 4) / BLOCK;
        const uint8_t* vsp = c.scales + (vrow + 4 * q) * BLOCKS + r * (WIDTH / 8) / BLOCK;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < KB; ++i) ks[t][i] = __ldg(ksp + t * BLOCKS + i);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < VB; ++i) vs[t][i] = __ldg(vsp + t * BLOCKS + i);
        ke = __ldg(reinterpret_cast<const uint16_t*>(c.exponents + krow) + r);
        vr = __ldg(reinterpret_cast<const uint16_t*>(c.exponents + vrow) + r);
        if (FMT == kMxfp4) ve = __ldg(reinterpret_cast<const uint32_t*>(c.exponents + vrow) + q);
    }
};

__device__ __forceinline__ int signed_byte(uint32_t w, int i) { return (int)(int8_t)(uint8_t)(w >> (8 * i)); }

// One block: a tile of 8 columns and a share of its groups, dealt out to the warps
// in turn.
template <typename T, int WIDTH, int FMT>
__global__ void __launch_bounds__(kWarps * 32) attend_columns_kernel(const AttendArgs a) {
    using G = Group16<WIDTH, FMT>;
    constexpr int KS = WIDTH / 16;  // MMAs along the head
    constexpr bool REST = sizeof(T) == 2 && std::is_same_v<T, __half>;
    constexpr int ROW = WIDTH + 4;  // a column's sums in shared memory
    extern __shared__ __align__(16) float sums[];  // [warp][8][ROW]
    __shared__ float s_m[kWarps][8], s_M[kWarps][8], s_l[kWarps][8];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane / 4, c = lane % 4;
    const int head = blockIdx.y;
    const Item item = item_of(a.b, blockIdx.x, a.group, 8);
    if (item.sequence < 0) return;
    const int before = item.length - item.tokens;  // the position of the first query token
    const int p0 = before + item.column / a.group, p1 = before + (item.column + item.columns - 1) / a.group;
    const Groups groups = groups_of(a.c, a.b, p0, p1, a.window, a.sinks);
    const int g0 = (int)((int64_t)groups.count * blockIdx.z / a.splits);
    const int g1 = (int)((int64_t)groups.count * (blockIdx.z + 1) / a.splits);

    // the queries: column r, elements c WIDTH / 4 .. of it
    uint32_t q[KS][2];
    float qf = a.scale;  // what a score is to be multiplied by
    {
        const bool have = r < item.columns;
        const int col = item.column + r;
        const T* src = static_cast<const T*>(a.q) + (int64_t)(item.first_token + (have ? col / a.group : 0)) * a.qt +
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
    const int pa = 2 * c < item.columns ? before + (item.column + 2 * c) / a.group : -1;
    const int pb = 2 * c + 1 < item.columns ? before + (item.column + 2 * c + 1) / a.group : -1;

    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float ma = minus_infinity(), mb = ma, Ma = ma, Mb = ma, la = 0.0f, lb = 0.0f;

    const int mine = g1 - g0 > warp ? (g1 - g0 - warp + kWarps - 1) / kWarps : 0;
    int pages = -1, base = 0;  // pages of 32 rounds, a lane each
    auto page_at = [&](int i) {
        if (i % 32 == 0) {
            base = i;
            pages = i + lane < mine ? page_of(a.c, a.b, item.sequence, group_token(groups, g0 + warp + (i + lane) * kWarps)) : -1;
        }
        return __shfl_sync(~0u, pages, i - base);
    };
    G now, next;
    if (mine > 0) now.load(a.c, page_at(0), head, group_token(groups, g0 + warp) & (a.c.page_size - 1), lane);
    for (int i = 0; i < mine; ++i) {
        const int token = group_token(groups, g0 + warp + i * kWarps);
        if (i + 1 < mine)
            next.load(a.c, page_at(i + 1), head, group_token(groups, g0 + warp + (i + 1) * kWarps) & (a.c.page_size - 1), lane);

        // scores
        uint32_t ks[2][G::KB];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int b = 0; b < G::KB; ++b) ks[t][b] = half_scale<FMT>(now.ks[t][b], signed_byte(now.ke, t)) * 0x10001u;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        constexpr int PER = KS / G::KB;  // MMAs of a block of a lane's codes
        auto score_step = [&](auto J) {
            constexpr int j = decltype(J)::value;
            const uint32_t x = ks[0][j / PER], y = ks[1][j / PER];
            constexpr int w = j / 2, lo = j % 2 * 2;
            mma16816(s, mul_half2(codes2<lo>(now.k[0][w]), x), mul_half2(codes2<lo>(now.k[1][w]), y),
                     mul_half2(codes2<lo + 1>(now.k[0][w]), x), mul_half2(codes2<lo + 1>(now.k[1][w]), y), q[j][0], q[j][1]);
        };
        static_for<KS>(score_step);
        const float k0 = now.bad ? not_a_number() : mxfp4_scale(signed_byte(now.ke, 0) + 127),
                    k1 = now.bad ? not_a_number() : mxfp4_scale(signed_byte(now.ke, 1) + 127);
        s[0] = s[0] * qf0 * k0;
        s[1] = s[1] * qf1 * k0;
        s[2] = s[2] * qf0 * k1;
        s[3] = s[3] * qf1 * k1;
        const bool whole = token + 15 <= p0 && (a.window == 0 || token > p1 - a.window);
        const int t0 = token + 2 * r;
        if (!whole) {
            if (!sees(pa, t0, a.window, a.sinks)) s[0] = minus_infinity();
            if (!sees(pb, t0, a.window, a.sinks)) s[1] = minus_infinity();
            if (!sees(pa, t0 + 1, a.window, a.sinks)) s[2] = minus_infinity();
            if (!sees(pb, t0 + 1, a.window, a.sinks)) s[3] = minus_infinity();
        }
        const float e0 = (float)signed_byte(now.vr, 0), e1 = (float)signed_byte(now.vr, 1);
        float u[4] = {s[0] + e0, s[1] + e0, s[2] + e1, s[3] + e1};
        const float sa = fmaxf(s[0], s[2]), sb = fmaxf(s[1], s[3]), ua = fmaxf(u[0], u[2]), ub = fmaxf(u[1], u[3]);
        if (__any_sync(~0u, sa > ma + kLag || sb > mb + kLag || ua > Ma + kLag || ub > Mb + kLag)) {
            float na = sa, nb = sb, Na = ua, Nb = ub;
#pragma unroll
            for (int d = 4; d < 32; d *= 2) {
                na = fmaxf(na, __shfl_xor_sync(~0u, na, d));
                nb = fmaxf(nb, __shfl_xor_sync(~0u, nb, d));
                Na = fmaxf(Na, __shfl_xor_sync(~0u, Na, d));
                Nb = fmaxf(Nb, __shfl_xor_sync(~0u, Nb, d));
            }
            na = fmaxf(ma, na);
            nb = fmaxf(mb, nb);
            Na = fmaxf(Ma, Na);
            Nb = fmaxf(Mb, Nb);
            la *= power2(ma - reference(na));
            lb *= power2(mb - reference(nb));
            const float fa = power2(Ma - reference(Na)), fb = power2(Mb - reference(Nb));
#pragma unroll
            for (int d = 0; d < KS; ++d) {
                o[d][0] *= fa;
                o[d][1] *= fb;
                o[d][2] *= fa;
                o[d][3] *= fb;
            }
            ma = na, mb = nb, Ma = Na, Mb = Nb;
        }
        const float ra = reference(ma), rb = reference(mb), Ra = reference(Ma) - kLift, Rb = reference(Mb) - kLift;
        la += power2(s[0] - ra) + power2(s[2] - ra);
        lb += power2(s[1] - rb) + power2(s[3] - rb);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            u[i] = power2(u[i] - Ra);
            u[i + 1] = power2(u[i + 1] - Rb);
        }
        const uint32_t h0 = half2_of(u[0], u[1]), h1 = half2_of(u[2], u[3]);
        const uint32_t w0 = transpose8x8(h0), w1 = transpose8x8(h1);
        uint32_t x0 = 0, x1 = 0;
        if (REST) {
            x0 = transpose8x8(half2_of(u[0] - low_half(h0), u[1] - high_half(h0)));
            x1 = transpose8x8(half2_of(u[2] - low_half(h1), u[3] - high_half(h1)));
        }

        // values: tokens 4 c, 4 c + 2 (rows 2 c, 2 c + 1) and 4 c + 1, 4 c + 3 (rows 2 c + 8, 2 c + 9)
        uint32_t vs[2][G::VB];
#pragma unroll
        for (int b = 0; b < G::VB; ++b) {
            uint32_t h[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) h[t] = half_scale<FMT>(now.vs[t][b], signed_byte(now.ve, t));
            if (!whole) {
                // a NaN reaches only the columns that see its token
                uint32_t nan = 0;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (half_is_nan(h[t])) {
                        nan |= 1u << t;
                        h[t] = 0;
                    }
                }
                if (__any_sync(~0u, nan != 0)) {
#pragma unroll 1
                    for (int cc = 0; cc < 4; ++cc) {
                        const uint32_t theirs = __shfl_sync(~0u, nan, (lane & ~3) | cc);
#pragma unroll 1
                        for (int t = 0; t < 4; ++t) {
                            if (!(theirs >> t & 1)) continue;
                            const bool hit_a = sees(pa, token + 4 * cc + t, a.window, a.sinks);
                            const bool hit_b = sees(pb, token + 4 * cc + t, a.window, a.sinks);
                            constexpr int SPAN = KS / G::VB;
#pragma unroll
                            for (int d = b * SPAN; d < (b + 1) * SPAN; ++d) {
                                if (hit_a) o[d][0] = o[d][2] = not_a_number();
                                if (hit_b) o[d][1] = o[d][3] = not_a_number();
                            }
                        }
                    }
                }
            }
            vs[0][b] = h[0] | h[2] << 16;
            vs[1][b] = h[1] | h[3] << 16;
        }
        auto value_word = [&](auto W) {
            constexpr int w = decltype(W)::value;
            // bytes of (token, token + 2): even elements in xe, odd ones in xo
            const uint32_t m = 0x0f0f0f0fu;
            const uint32_t xe = (now.v[0][w] & m) | (now.v[2][w] << 4 & ~m), xo = (now.v[0][w] >> 4 & m) | (now.v[2][w] & ~m);
            const uint32_t ye = (now.v[1][w] & m) | (now.v[3][w] << 4 & ~m), yo = (now.v[1][w] >> 4 & m) | (now.v[3][w] & ~m);
            auto tile = [&](auto I) {
                constexpr int i = decltype(I)::value, d = w * 4 + i;
                constexpr int b = d / (KS / G::VB);
                const uint32_t a0 = mul_half2(codes2<i>(xe), vs[0][b]), a1 = mul_half2(codes2<i>(xo), vs[0][b]);
                const uint32_t a2 = mul_half2(codes2<i>(ye), vs[1][b]), a3 = mul_half2(codes2<i>(yo), vs[1][b]);
                mma16816(o[d], a0, a1, a2, a3, w0, w1);
                if (REST) mma16816(o[d], a0, a1, a2, a3, x0, x1);
            };
            static_for<4>(tile);
        };
        static_for<G::VW>(value_word);
        now = next;
    }

    // the warps' parts
#pragma unroll
    for (int d = 4; d < 32; d *= 2) {
        la += __shfl_xor_sync(~0u, la, d);
        lb += __shfl_xor_sync(~0u, lb, d);
    }
    if (r == 0) {
        s_m[warp][2 * c] = ma;
        s_m[warp][2 * c + 1] = mb;
        s_M[warp][2 * c] = Ma;
        s_M[warp][2 * c + 1] = Mb;
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
    if (col >= item.columns) return;
    float m = s_m[0][col], M = s_M[0][col];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        m = fmaxf(m, s_m[w][col]);
        M = fmaxf(M, s_M[w][col]);
    }
    float l = 0.0f, f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        l += s_l[w][col] * power2(s_m[w][col] - reference(m));
        f[w] = power2(s_M[w][col] - reference(M));
    }
    const int64_t token = item.first_token + (item.column + col) / a.group, h = head * a.group + (item.column + col) % a.group;
    const int64_t row = token * a.heads + h;
    const bool any = before + (item.column + col) / a.group >= 0;
    if (a.splits > 1) {
        const int64_t part = blockIdx.z * (a.b.tokens * a.heads) + row;
        if (at == 0) a.part[part] = make_float4(m, M, l, any ? 1.0f : 0.0f);
#pragma unroll
        for (int d = at * 4; d < WIDTH; d += LANES * 4) {
            float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(sums + (w * 8 + col) * ROW + d);
                y.x = fmaf(x.x, f[w], y.x);
                y.y = fmaf(x.y, f[w], y.y);
                y.z = fmaf(x.z, f[w], y.z);
                y.w = fmaf(x.w, f[w], y.w);
            }
            *reinterpret_cast<float4*>(a.sums + part * WIDTH + d) = y;
        }
        return;
    }
    const Finish z = finish_of(m, M, l, kLift + (FMT == kMxfp4 ? kMxLift : 0), any);
    T* out = static_cast<T*>(a.out) + token * a.ot + h * a.oh;
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
        store4(out, d, a.c.dim, a.vec_out, z, y);
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
    const int s = search(a.b, token, 1, 1, 0);
    if (s < 0 || a.b.starts[s] < 0 || a.b.starts[s + 1] <= token || a.b.starts[s + 1] > a.b.tokens) return;
    float m = minus_infinity(), M = m;
    float4 mine = make_float4(m, m, 0.0f, 0.0f);
    for (int i = lane; i < a.splits; i += 32) {
        const float4 p = a.part[i * rows + row];
        if (i < 32) mine = p;
        m = fmaxf(m, p.x);
        M = fmaxf(M, p.y);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        M = fmaxf(M, __shfl_xor_sync(~0u, M, d));
    }
    const bool any = __shfl_sync(~0u, mine.w, 0) != 0.0f;
    const int at = ((warp % WARPS) * 32 + lane) * 4;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
    for (int i0 = 0; i0 < a.splits; i0 += 32) {
        if (i0 > 0) mine = i0 + lane < a.splits ? a.part[(i0 + lane) * rows + row] : make_float4(minus_infinity(), minus_infinity(), 0.0f, 0.0f);
        l += mine.z * power2(mine.x - reference(m));
        const float f = power2(mine.y - reference(M));
        const int n = min(32, a.splits - i0);
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
    if (at < WIDTH) store4(static_cast<T*>(a.out) + token * a.ot + h * a.oh, at, a.c.dim, a.vec_out, finish_of(m, M, l, lift, any), y);
}

template <typename T, int WIDTH>
cudaError_t columns(const AttendArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)attend_tiles(a.b, a.group, 8), (unsigned)a.c.heads, (unsigned)a.splits);
    const size_t smem = (size_t)kWarps * 8 * (WIDTH + 4) * sizeof(float);
    return a.c.fmt == kMxfp4 ? launch_pdl(attend_columns_kernel<T, WIDTH, kMxfp4>, grid, dim3(kWarps * 32), smem, st, a)
                             : launch_pdl(attend_columns_kernel<T, WIDTH, kNvfp4>, grid, dim3(kWarps * 32), smem, st, a);
}
template <typename T, int WIDTH>
cudaError_t join(const AttendArgs& a, float lift, cudaStream_t st) {
    const int64_t rows = a.b.tokens * a.heads, per = WIDTH == 256 ? 2 : 4;
    return launch_pdl(join_kernel<T, WIDTH>, dim3((unsigned)((rows + per - 1) / per)), dim3(128), 0, st, a, lift);
}

// How many parts a row's tokens are cut into: as many blocks as the SMs hold (4
// each), at least 4 groups of 16 tokens for each of a block's warps.
int parts_of(const AttendArgs& a) {
    const int64_t tiles = std::max(a.b.tokens * a.group / 8, (int64_t)a.b.batch) * a.c.heads;
    const int64_t longest = a.window > 0 ? a.window + a.sinks : (int64_t)a.b.table_pages * a.c.page_size;
    const int64_t most = (longest + kWarps * 64 - 1) / (kWarps * 64);
    const int64_t want = 4LL * device_sms() / std::max<int64_t>(1, tiles);
    return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, 128}));
}

}  // namespace

int attend_columns_parts(const AttendArgs& a) { return parts_of(a); }

cudaError_t launch_attend_columns(const AttendArgs& a, int type, cudaStream_t st) {
    cudaError_t err;
    if (type == DDGEMM_BF16)
        err = a.c.width == 64 ? columns<__nv_bfloat16, 64>(a, st) : a.c.width == 128 ? columns<__nv_bfloat16, 128>(a, st) : columns<__nv_bfloat16, 256>(a, st);
    else
        err = a.c.width == 64 ? columns<__half, 64>(a, st) : a.c.width == 128 ? columns<__half, 128>(a, st) : columns<__half, 256>(a, st);
    if (err != cudaSuccess || a.splits == 1) return err;
    return launch_attend_join(a, type, kLift + (a.c.fmt == kMxfp4 ? kMxLift : 0), st);
}

cudaError_t launch_attend_join(const AttendArgs& a, int type, float lift, cudaStream_t st) {
    if (type == DDGEMM_BF16)
        return a.c.width == 64 ? join<__nv_bfloat16, 64>(a, lift, st) : a.c.width == 128 ? join<__nv_bfloat16, 128>(a, lift, st) : join<__nv_bfloat16, 256>(a, lift, st);
    return a.c.width == 64 ? join<__half, 64>(a, lift, st) : a.c.width == 128 ? join<__half, 128>(a, lift, st) : join<__half, 256>(a, lift, st);
}

}  // namespace ddg
