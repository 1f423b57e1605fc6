// mx4.cuh -- the 4-bit microscaled matrix formats (declarations in ddgemm.h):
// layout arithmetic shared by host and device, and the device routines that
// turn 32-bit values into codes and scales.
//
// A matrix of `rows` rows of length K holds E2M1 codes, two to a byte along k
// (the even k in the low nibble), and one scale byte per block of k:
//   mxfp4: blocks of 32, scale 2^(byte - 127) (E8M0; 255 is NaN);
//   nvfp4: blocks of 16, E4M3 scale, and an exponent e per row; a value is
//          code * scale * 2^e.
// The scales lie in tiles of 128 rows by 4 blocks (512 bytes), row r and block
// b at (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4: the order in which a tile
// is copied into tensor memory, lane r % 32 and one 32-bit column for each 32
// rows.  K is padded to MX4_TILE_K in the scales (byte 0) and to 32 in the
// codes (code 0).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace ddg {

constexpr int MX4_TILE_K = 256;  // k of one 128-byte row of codes: a stage of the products

constexpr int kMxfp4 = DDGEMM_MXFP4, kNvfp4 = DDGEMM_NVFP4;

__host__ __device__ constexpr int mx4_block(int fmt) { return fmt == kMxfp4 ? 32 : 16; }
// scale tiles (4 blocks of k) per MX4_TILE_K
__host__ __device__ constexpr int mx4_tiles_per_k(int fmt) { return MX4_TILE_K / mx4_block(fmt) / 4; }
__host__ __device__ inline int64_t mx4_scale_tiles(int fmt, int64_t K) {
    return (K + MX4_TILE_K - 1) / MX4_TILE_K * mx4_tiles_per_k(fmt);
}
__host__ __device__ inline int64_t mx4_code_bytes(int64_t K) { return round_up(K, 32) / 2; }
__host__ __device__ inline int64_t mx4_scale_bytes(int fmt, int64_t rows, int64_t K) {
    return (rows + 127) / 128 * mx4_scale_tiles(fmt, K) * 512;
}
// Offset of the four scale bytes of row r in scale tile t of its 128 rows.
__host__ __device__ inline int64_t mx4_scale_word(int64_t r, int64_t t, int64_t tiles) {
    return ((r / 128) * tiles + t) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4;
}

#ifdef __CUDACC__

constexpr uint32_t kInfBits = 0x7f800000u;

// 2^e as a float, -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 2^s as two factors of the same direction, so that no partial result leaves the
// range before the whole does.  s is bounded to +-200: beyond, what is scaled
// here (codes times scales, 2^-10 to 2^12, and sums of their products, 2^-20 to
// 2^45) is 0 or infinite in 32 bits anyway.
__device__ __forceinline__ float2 exp2_factors(int s) {
    s = min(max(s, -200), 200);
    const int h = s >> 1;
    return make_float2(exp2_int(h), exp2_int(s - h));
}
// The sum of two exponents that may be any 32-bit numbers, bounded to 32 bits.
__device__ __forceinline__ int add_exponents(int a, int b) {
    int s;
    asm("add.sat.s32 %0, %1, %2;" : "=r"(s) : "r"(a), "r"(b));
    return s;
}
__device__ __forceinline__ float scale_by_exp2(float x, int s) {
    const float2 f = exp2_factors(s);
    return x * f.x * f.y;
}

// The E8M0 byte of a block whose largest magnitude has these bits:
// floor(log2 max) - 2 (so that the largest value lies in [4, 8) before it
// saturates at 6), 255 (NaN) where a value is infinite or NaN.
__device__ __forceinline__ uint32_t mxfp4_scale_byte(uint32_t max_bits) {
    if (max_bits >= kInfBits) return 255u;
    const int b = (int)(max_bits >> 23) - 2;
    return (uint32_t)(b > 0 ? b : 0);
}
// 1 / scale, a power of two; 0 for NaN.
__device__ __forceinline__ float mxfp4_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float mxfp4_scale(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : byte == 0u ? __uint_as_float(0x00400000u)
                                                                    : __uint_as_float(byte << 23);
}

// The exponent of an nvfp4 row whose largest finite magnitude has these bits:
// the least e >= -100 with max <= 6 * 448 * 2^e (2688 = 1.3125 * 2^11); 0 for
// a zero row.
__device__ __forceinline__ int nvfp4_row_exponent(uint32_t max_bits) {
    if (max_bits == 0u) return 0;
    const int e = (int)(max_bits >> 23) - 127 - ((max_bits & 0x7fffffu) <= 0x280000u ? 11 : 10);
    return e > -100 ? e : -100;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((unsigned short)byte));
    return __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu)));
}

// y / s with r = 1 / s correctly rounded: one residual correction of y * r
// gives the correctly rounded quotient (Markstein's theorem), and rounding
// that to E2M1 is the same as rounding the exact quotient: |y - t s| is at
// least one last place of y for every tie point t (3 bits) but a true tie.
__device__ __forceinline__ float quotient(float y, float s, float r) {
    const float q = y * r;
    return fmaf(fmaf(-q, s, y), r, q);
}

__device__ __forceinline__ float sixth(float x) { return quotient(x, 6.0f, 1.0f / 6.0f); }

// The E4M3 byte of an nvfp4 block: max / (6 * 2^e) rounded to nearest, at
// least the smallest scale for a block that is not zero; 127 (NaN) where a
// value is infinite or NaN.  `unit` is 2^-e.  The sixth is correctly rounded
// (but for values so small that the scale is the least one anyway), and none
// but a true tie of the E4M3 grid lands on one (6 t has at most 8 significant
// bits, so max differs from it by at least one of its own last places, more
// than half a last place of the quotient).
__device__ __forceinline__ uint32_t nvfp4_scale_byte(uint32_t max_bits, float unit) {
    if (max_bits >= kInfBits) return 127u;
    if (max_bits == 0u) return 0u;
    const float want = sixth(__uint_as_float(max_bits)) * unit;
    unsigned short two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(want));
    const uint32_t byte = two & 0xffu;
    return byte > 0u ? byte : 1u;
}

// The scale of an nvfp4 block and its row's power of two in one: exact and
// normal (2^-109 .. 2^126), as is the reciprocal.  Both 0 for a zero block and
// for NaN: quotients of finite values are then 0.
__device__ __forceinline__ float nvfp4_step(uint32_t byte, int e) {
    return byte == 127u ? 0.0f : e4m3_value(byte) * exp2_int(e);
}
__device__ __forceinline__ float nvfp4_inverse(uint32_t byte, float step) {
    return byte == 0u || byte == 127u ? 0.0f : __frcp_rn(step);
}

// The same step before the row's exponent is known.  A power of two commutes
// with rounding to E4M3's four significant bits, so max / 6 rounded to four
// bits is the step of every block whose scale is not subnormal, whatever e
// (max a finite magnitude's bits; at least the least step there is, 2^-109).
__device__ __forceinline__ float nvfp4_wide_step(uint32_t max_bits) {
    if (max_bits == 0u) return 0.0f;
    uint32_t b = __float_as_uint(sixth(__uint_as_float(max_bits)));
    b = (b + 0x7ffffu + (b >> 20 & 1u)) & ~0xfffffu;
    return fmaxf(__uint_as_float(b), exp2_int(-109));
}

// The same for two values with scales of their own, on packed 32-bit pairs.
__device__ __forceinline__ uint64_t pack_pair(float a, float b) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ void unpack_pair(uint64_t p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// `minus_s`: the scales negated.
__device__ __forceinline__ uint64_t quotient_pair(uint64_t y, uint64_t minus_s, uint64_t r) {
    const uint64_t q = mul_pair(y, r);
    return fma_pair(fma_pair(q, minus_s, y), r, q);
}

// The bytes of four blocks, the first lowest, where the sign bit marks a block
// that is to be NaN: the same operations, two blocks at a time.
__device__ __forceinline__ uint32_t nvfp4_scale_bytes(const uint4& marked, float unit) {
    const uint32_t bits[4] = {marked.x & 0x7fffffffu, marked.y & 0x7fffffffu, marked.z & 0x7fffffffu,
                              marked.w & 0x7fffffffu};
    const uint64_t minus_six = pack_pair(-6.0f, -6.0f), part = pack_pair(1.0f / 6.0f, 1.0f / 6.0f), units = pack_pair(unit, unit);
    float want[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint64_t most = pack_pair(__uint_as_float(bits[i]), __uint_as_float(bits[i + 1]));
        unpack_pair(mul_pair(quotient_pair(most, minus_six, part), units), want[i], want[i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) want[i] = bits[i] != 0u ? fmaxf(want[i], 0x1p-9f) : 0.0f;
    uint32_t word;
    asm("{\n"
        " .reg .b16 t0, t1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 t0, %2, %1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 t1, %4, %3;\n"
        " mov.b32 %0, {t0, t1};\n"
        "}\n"
        : "=r"(word)
        : "f"(want[0]), "f"(want[1]), "f"(want[2]), "f"(want[3]));
    if ((marked.x | marked.y | marked.z | marked.w) >> 31) {
        word |= (marked.x >> 31) * 0x7fu | (marked.y >> 31) * 0x7f00u | (marked.z >> 31) * 0x7f0000u |
                (marked.w >> 31) * 0x7f000000u;
    }
    return word;
}

// Whether one of four bytes (none above 127) is 1 to 8: a subnormal scale, or
// the least normal one, perhaps rounded up to.
__device__ __forceinline__ bool nvfp4_low_scales(uint32_t word) {
    return ((word + 0x7f7f7f7fu) & ~(word + 0x77777777u) & 0x80808080u) != 0u;
}

// Eight values (already divided by their scales) as eight E2M1 codes, the
// first in the lowest nibble; to nearest, ties to even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&y)[8]) {
    uint32_t w;
    asm("{\n"
        " .reg .b8 t0, t1, t2, t3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n"
        " mov.b32 %0, {t0, t1, t2, t3};\n"
        "}\n"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return w;
}

__device__ __forceinline__ void e2m1_unpack8(uint32_t w, float (&y)[8]) {
    uint32_t h[4];
    asm("{\n"
        " .reg .b8 t0, t1, t2, t3;\n"
        " mov.b32 {t0, t1, t2, t3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, t0;\n"
        " cvt.rn.f16x2.e2m1x2 %1, t1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, t2;\n"
        " cvt.rn.f16x2.e2m1x2 %3, t3;\n"
        "}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = __half2float(__ushort_as_half((unsigned short)(h[i] & 0xffffu)));
        y[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(h[i] >> 16)));
    }
}

// ---- element types of inputs and outputs (DDGEMM_F32, _BF16, _F16) ----

template <typename T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// Eight floats as consecutive elements from a 16-byte aligned address on.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&y)[8]) {
    constexpr int W = sizeof(T) * 8 / 16;
    uint4 raw[W];
    T* t = reinterpret_cast<T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = from_float<T>(y[i]);
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(p)[i] = raw[i];
}

#endif  // __CUDACC__

}  // namespace ddg
