// mx4.cu -- conversion to and from the 4-bit microscaled formats (mx4.cuh).
//
// Quantisation reads each value once and writes 4 bits and its share of a
// scale byte: bound by HBM (2.56 bytes per 16-bit value for nvfp4, 2.53 for
// mxfp4) with about 10 instructions to hide for every 32 values of a warp.
// Columns of 8192 x 16384 16-bit values to nvfp4: 56 us and 15 us to finish the
// scales (0.90 of the copy rate in the first, 63% of the issue slots), to mxfp4 51
// us; back to 16 bits 51 us (343 MB, 0.98 of the copy rate).  Rows, which a warp
// converts a value at a time, take the issue slots: 74 us to mxfp4 (75% of them, 54%
// of HBM), 121 us to nvfp4 (quotients instead of products: 76%, 33%); 4096 x 4096
// rows 10.2 and 37.5 us; one row of 8192 1.7 us behind another launch.
#include "launch.cuh"
#include "mx4.cuh"

namespace ddg {
namespace {

constexpr int QWARPS = 8;  // warps per block of the row kernels

// A lane's 8 values of each of N tiles of 256 k of a row, from tile kt on and
// `step` tiles apart (zero beyond K).  Where the row is 16-byte aligned and a
// multiple of 8 long, the loads are issued without a branch between them (an
// address beyond the row is pulled back into it): all are in flight together.
template <typename T, int N>
__device__ __forceinline__ void load_tiles(const T* row, int64_t kt, int64_t step, int lane, int64_t K, bool vec,
                                           float (&x)[N][8]) {
    if (vec) {
        constexpr int W = sizeof(T) / 2;
        uint4 raw[N][W];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t k0 = min((kt + j * step) * MX4_TILE_K + lane * 8, K - 8);
#pragma unroll
            for (int i = 0; i < W; ++i) raw[j][i] = reinterpret_cast<const uint4*>(row + k0)[i];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const bool in = (kt + j * step) * MX4_TILE_K + lane * 8 < K;
            const T* t = reinterpret_cast<const T*>(raw[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[j][i] = in ? to_float<T>(t[i]) : 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t k0 = (kt + j * step) * MX4_TILE_K + lane * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[j][i] = k0 + i < K ? to_float<T>(row[k0 + i]) : 0.0f;
        }
    }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A warp's 256 k of one row: codes and scale words.  `e` is the exponent of
// an nvfp4 row.
template <int FMT>
__device__ __forceinline__ void quantize_tile(const float (&x)[8], int e, int lane, int64_t row, int64_t kt,
                                              int64_t K, uint8_t* codes, int64_t ldq, uint8_t* scales) {
    constexpr int LANES = mx4_block(FMT) / 8;  // lanes that share a block
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(x[i]));
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) m = max(m, __shfl_xor_sync(~0u, m, d));
    float y[8];
    uint32_t byte;
    if (FMT == kMxfp4) {
        byte = mxfp4_scale_byte(m);
        const float inv = mxfp4_inverse(byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
    } else {
        byte = nvfp4_scale_byte(m, exp2_int(-e));
        const float s = nvfp4_step(byte, e), r = nvfp4_inverse(byte, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = quotient(x[i], s, r);
    }
    if (kt * MX4_TILE_K + lane * 8 < round_up(K, 32))
        *reinterpret_cast<uint32_t*>(codes + row * ldq + kt * (MX4_TILE_K / 2) + lane * 4) = e2m1_pack8(y);
    // four blocks' bytes to one word, on the first lane of their 4 * LANES lanes
    uint32_t w = byte << (8 * (lane / LANES % 4));
    w |= __shfl_xor_sync(~0u, w, LANES);
    w |= __shfl_xor_sync(~0u, w, 2 * LANES);
    if (lane % (4 * LANES) == 0) {
        const int64_t t = kt * mx4_tiles_per_k(FMT) + lane / (4 * LANES);
        *reinterpret_cast<uint32_t*>(scales + mx4_scale_word(row, t, mx4_scale_tiles(FMT, K))) = w;
    }
}

// mxfp4 rows: one warp for TILES times 256 k of a row, all loaded before the
// first is converted (one tile where there are few: latency counts then).
template <typename T, int TILES>
__global__ void __launch_bounds__(QWARPS * 32) mxfp4_rows_kernel(const T* X, int64_t ldx, int64_t rows, int64_t K,
                                                                 bool vec, uint8_t* codes, int64_t ldq,
                                                                 uint8_t* scales) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t kts = (K + MX4_TILE_K - 1) / MX4_TILE_K, steps = (kts + TILES - 1) / TILES;
    const int64_t item = (int64_t)blockIdx.x * QWARPS + (threadIdx.x >> 5);
    if (item >= rows * steps) return;
    const int64_t row = item / steps, kt = item % steps * TILES;
    float x[TILES][8];
    load_tiles<T, TILES>(X + row * ldx, kt, 1, lane, K, vec, x);
#pragma unroll
    for (int j = 0; j < TILES; ++j)
        if (kt + j < kts) quantize_tile<kMxfp4>(x[j], 0, lane, row, kt + j, K, codes, ldq, scales);
}

// nvfp4 rows: one block for a row.  The row's values stay in registers
// between the maximum and the conversion as far as KEEP tiles per warp reach
// (16 warps: 16384 values); longer rows are read again.
constexpr int ROW_WARPS = 16;
template <typename T>
__global__ void __launch_bounds__(ROW_WARPS * 32) nvfp4_rows_kernel(const T* X, int64_t ldx, int64_t K, bool vec,
                                                                 uint8_t* codes, int64_t ldq, uint8_t* scales,
                                                                 int32_t* exponents) {
    constexpr int KEEP = 4;
    __shared__ uint32_t part[ROW_WARPS];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    const int64_t kts = (K + MX4_TILE_K - 1) / MX4_TILE_K;
    const T* src = X + row * ldx;
    float keep[KEEP][8];
    uint32_t m = 0;
    auto take = [&](const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = abs_bits(x[i]);
            m = max(m, b < kInfBits ? b : 0u);
        }
    };
    load_tiles<T, KEEP>(src, warp, warps, lane, K, vec, keep);
#pragma unroll
    for (int j = 0; j < KEEP; ++j) take(keep[j]);
    for (int64_t kt = warp + (int64_t)KEEP * warps; kt < kts; kt += warps) {
        float x[1][8];
        load_tiles<T, 1>(src, kt, 1, lane, K, vec, x);
        take(x[0]);
    }
    m = __reduce_max_sync(~0u, m);
    if (lane == 0) part[warp] = m;
    __syncthreads();
    m = part[0];
    for (int w = 1; w < warps; ++w) m = max(m, part[w]);
    const int e = nvfp4_row_exponent(m);
    if (threadIdx.x == 0) exponents[row] = e;
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        const int64_t kt = warp + (int64_t)j * warps;
        if (kt < kts) quantize_tile<kNvfp4>(keep[j], e, lane, row, kt, K, codes, ldq, scales);
    }
    for (int64_t kt = warp + (int64_t)KEEP * warps; kt < kts; kt += warps) {
        float x[1][8];
        load_tiles<T, 1>(src, kt, 1, lane, K, vec, x);
        quantize_tile<kNvfp4>(x[0], e, lane, row, kt, K, codes, ldq, scales);
    }
}

// Two consecutive elements, as they lie in memory.
template <typename T> struct Two;
template <> struct Two<float> {
    using raw = uint2;
    static __device__ __forceinline__ void split(uint2 r, float& a, float& b) { a = __uint_as_float(r.x), b = __uint_as_float(r.y); }
    static __device__ __forceinline__ uint2 join(float a, float b) { return make_uint2(__float_as_uint(a), __float_as_uint(b)); }
};
template <> struct Two<__nv_bfloat16> {
    static constexpr bool kBrain = true;
    using raw = uint32_t;
    static __device__ __forceinline__ void split(uint32_t r, float& a, float& b) {
        a = __uint_as_float(r << 16), b = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t join(__nv_bfloat16 a, __nv_bfloat16 b) {
        return (uint32_t)__bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16;
    }
};
template <> struct Two<__half> {
    static constexpr bool kBrain = false;
    using raw = uint32_t;
    static __device__ __forceinline__ void split(uint32_t r, float& a, float& b) {
        a = __half2float(__ushort_as_half((unsigned short)(r & 0xffffu)));
        b = __half2float(__ushort_as_half((unsigned short)(r >> 16)));
    }
    static __device__ __forceinline__ uint32_t join(__half a, __half b) {
        return (uint32_t)__half_as_ushort(a) | (uint32_t)__half_as_ushort(b) << 16;
    }
};

// Largest magnitudes of two columns over N rows, as the bits of floats (with
// infinities and NaN, which are larger than any finite value; FINITE: without).
// 16-bit values are compared two at a time as integers.
template <typename T, int N, bool FINITE>
__device__ __forceinline__ void max_pair(const typename Two<T>::raw* raw, uint32_t& m0, uint32_t& m1) {
    if constexpr (sizeof(T) == 4) {
        m0 = m1 = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t x = raw[i].x & 0x7fffffffu, y = raw[i].y & 0x7fffffffu;
            m0 = max(m0, !FINITE || x < kInfBits ? x : 0u);
            m1 = max(m1, !FINITE || y < kInfBits ? y : 0u);
        }
    } else {
        constexpr uint32_t inf = sizeof(T) == 2 && Two<T>::kBrain ? 0x7f807f80u : 0x7c007c00u;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t x = raw[i] & 0x7fff7fffu;
            if (FINITE) x &= __vcmpltu2(x, inf);
            m = __vmaxu2(m, x);
        }
        float a, b;
        Two<T>::split(m, a, b);
        m0 = __float_as_uint(a);
        m1 = __float_as_uint(b);
    }
}

// Columns c and c + 1 of N consecutive rows from k on (zero beyond R and K).
// The whole rows of a full tile are loaded without a branch between them, so
// that all N loads are in flight together.
template <typename T, int N>
__device__ __forceinline__ void load_columns(const T* X, int64_t ldx, int64_t k, int64_t c, int64_t K, int64_t R, bool vec,
                                             typename Two<T>::raw (&raw)[N]) {
    const T* p = X + k * ldx + c;
    if (vec && k + N <= K && c + 2 <= R) {
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = *reinterpret_cast<const typename Two<T>::raw*>(p + i * ldx);
    } else {
        const T zero = from_float<T>(0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i)
            raw[i] = Two<T>::join(k + i < K && c < R ? p[i * ldx] : zero, k + i < K && c + 1 < R ? p[i * ldx + 1] : zero);
    }
}

// The largest of four blocks' finite magnitudes (the sign bit is a mark).
__device__ __forceinline__ uint32_t largest(const uint4& b) {
    return max(max(b.x & 0x7fffffffu, b.y & 0x7fffffffu), max(b.z & 0x7fffffffu, b.w & 0x7fffffffu));
}

// Columns of X (K x R) as rows of the result: a block takes 64 columns and 256
// k.  Warp w reads rows 32 w .. + 31, a lane two columns of them, so a lane
// holds whole blocks of k and needs no exchange for their maxima; codes and
// scales go through shared memory (rows of 33 and 5 words: no bank conflicts)
// and leave as whole 128-byte rows.  X is read once in either format: nvfp4 codes
// are made with nvfp4_wide_step, and the blocks' largest magnitudes go to `most`
// for nvfp4_finish_kernel, which a pass over X for the columns' maxima ahead of
// this one would replace at 0.25 bytes a value less written but 2 more read
// (8192 x 16384 values: 102 us with that pass, 71 without).
template <typename T, int FMT>
__global__ void __launch_bounds__(256) mx4_columns_kernel(const T* X, int64_t ldx, int64_t R, int64_t K, bool vec,
                                                          uint8_t* codes, int64_t ldq, uint8_t* scales, float* most) {
    constexpr int BLOCK = mx4_block(FMT), WORDS = mx4_tiles_per_k(FMT);
    __shared__ uint32_t code[64][33];   // row p: column (p % 32) * 2 + p / 32 of the tile
    __shared__ uint32_t scale[64][FMT == kMxfp4 ? 5 : 17];  // scale bytes, or largest magnitudes
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * 64, kt = blockIdx.y;
    const int64_t c = r0 + lane * 2, k0 = kt * MX4_TILE_K + warp * 32;
    typename Two<T>::raw raw[32];
    load_columns<T, 32>(X, ldx, k0, c, K, R, vec, raw);
#pragma unroll
    for (int b = 0; b < 32 / BLOCK; ++b) {
        uint32_t m[2], mark[2] = {0, 0};
        max_pair<T, BLOCK, false>(raw + b * BLOCK, m[0], m[1]);
        if (FMT == kNvfp4 && (m[0] >= kInfBits || m[1] >= kInfBits)) {  // rare: the finite ones alone
            mark[0] = m[0] >= kInfBits ? 0x80000000u : 0u;
            mark[1] = m[1] >= kInfBits ? 0x80000000u : 0u;
            max_pair<T, BLOCK, true>(raw + b * BLOCK, m[0], m[1]);
        }
        float s[2] = {0.0f, 0.0f}, r[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (FMT == kMxfp4) {
                const uint32_t byte = mxfp4_scale_byte(m[j]);
                r[j] = mxfp4_inverse(byte);
                reinterpret_cast<uint8_t*>(&scale[j * 32 + lane][0])[warp] = (uint8_t)byte;
            } else {
                s[j] = nvfp4_wide_step(m[j]);
                r[j] = s[j] > 0.0f ? __frcp_rn(s[j]) : 0.0f;
                scale[j * 32 + lane][warp * 2 + b] = m[j] | mark[j];
            }
        }
        const uint64_t rr = pack_pair(r[0], r[1]), ss = pack_pair(-s[0], -s[1]);
#pragma unroll
        for (int q = 0; q < BLOCK / 8; ++q) {
            float y[2][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[2];
                Two<T>::split(raw[b * BLOCK + q * 8 + i], v[0], v[1]);
                const uint64_t vv = pack_pair(v[0], v[1]);
                unpack_pair(FMT == kMxfp4 ? mul_pair(vv, rr) : quotient_pair(vv, ss, rr), y[0][i], y[1][i]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) code[j * 32 + lane][warp * 4 + b * (BLOCK / 8) + q] = e2m1_pack8(y[j]);
        }
    }
    __syncthreads();
    // 64 rows of 128 bytes, 16 bytes a thread: 8 threads a row
    const int64_t bytes = mx4_code_bytes(K);
#pragma unroll
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int p = i / 8, at = i % 8;
        const int64_t row = r0 + p % 32 * 2 + p / 32;
        if (row < R && kt * 128 + at * 16 < bytes)
            *reinterpret_cast<uint4*>(codes + row * ldq + kt * 128 + at * 16) =
                make_uint4(code[p][at * 4], code[p][at * 4 + 1], code[p][at * 4 + 2], code[p][at * 4 + 3]);
    }
    const int64_t tiles = mx4_scale_tiles(FMT, K);
    if (FMT == kMxfp4) {
        if (threadIdx.x < 64 * WORDS) {
            const int p = threadIdx.x % 64, w = threadIdx.x / 64;
            const int64_t row = r0 + p % 32 * 2 + p / 32;
            if (row < R) *reinterpret_cast<uint32_t*>(scales + mx4_scale_word(row, kt * WORDS + w, tiles)) = scale[p][w];
        }
    } else {  // 16 magnitudes a row: 64 bytes, 4 threads a row; after all of them, the largest finite one of the 16
        const int i = threadIdx.x / 4, p = i % 2 * 32 + i / 2, at = threadIdx.x % 4 * 4;
        const int64_t row = r0 + i;
        const uint4 b = make_uint4(scale[p][at], scale[p][at + 1], scale[p][at + 2], scale[p][at + 3]);
        uint32_t m = largest(b);
        m = max(m, __shfl_xor_sync(~0u, m, 1));
        m = max(m, __shfl_xor_sync(~0u, m, 2));
        if (row < R) {
            reinterpret_cast<uint4*>(most)[(kt * R + row) * 4 + at / 4] = b;
            if (at == 0) reinterpret_cast<uint32_t*>(most)[gridDim.y * R * 16 + kt * R + row] = m;
        }
    }
}

// nvfp4 rows whose codes were made block by block with nvfp4_wide_step: from
// the blocks' largest finite magnitudes (the sign bit marks a block that also
// holds an infinity or a NaN; tiles * 4 values a row, 0 beyond K) the row's
// exponent and the scales.  Where a scale is subnormal (the block's largest is below 2^-14.8 of the row's) the step has
// fewer bits than the codes were made with: they are made again, from the
// values themselves (row i being column i of X) or, without X, from the codes.
template <typename T>
__device__ __forceinline__ void remake_codes(uint32_t word, uint4 b, int e, int64_t t, int64_t row, int64_t K, uint8_t* codes,
                                          const T* X, int64_t ldx) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const uint32_t byte = word >> (8 * i) & 0xffu;
        const uint32_t top = (i == 0 ? b.x : i == 1 ? b.y : i == 2 ? b.z : b.w) & 0x7fffffffu;
        const float was = nvfp4_wide_step(top), is = nvfp4_step(byte, e);
        if (byte == 0u || byte > 8u || was == is) continue;
        const float r = nvfp4_inverse(byte, is);
        uint32_t* c = reinterpret_cast<uint32_t*>(codes + (t * 4 + i) * 8);
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
            float y[8];
            const int64_t k = (t * 4 + i) * 16 + q * 8;
            e2m1_unpack8(c[q], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v = y[j] * was;
                if (X != nullptr) v = k + j < K ? to_float<T>(X[(k + j) * ldx + row]) : 0.0f;
                y[j] = quotient(v, is, r);
            }
            c[q] = e2m1_pack8(y);
        }
    }
}

// A block of threads takes a row, or (WARP) a warp, which needs no barrier: many
// rows of at most 128 tiles, which a warp holds in registers (the block of 8192 x
// 1024 x 2048 78 us, 84 otherwise; no gain from 256 tiles on, 363 us for 361).
template <bool WARP>
__global__ void __launch_bounds__(256, 4) nvfp4_finish_kernel(const float* most, int64_t rows, int64_t K, uint8_t* codes,
                                                              int64_t ldq, uint8_t* scales, int32_t* exponents) {
    constexpr int KEPT = WARP ? 4 : 1;  // a thread's first tiles stay in registers, others are read again
    __shared__ uint32_t part[8];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = WARP ? (int64_t)blockIdx.x * 8 + warp : blockIdx.x, tiles = mx4_scale_tiles(kNvfp4, K);
    const int first = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
    if (WARP && row >= rows) return;
    const uint4* src = reinterpret_cast<const uint4*>(most) + row * tiles;
    uint4 kept[KEPT];
#pragma unroll
    for (int j = 0; j < KEPT; ++j) kept[j] = first + j * step < tiles ? src[first + j * step] : make_uint4(0, 0, 0, 0);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < KEPT; ++j) m = max(m, largest(kept[j]));
    for (int64_t t = first + KEPT * step; t < tiles; t += step) m = max(m, largest(src[t]));
    m = __reduce_max_sync(~0u, m);
    if constexpr (!WARP) {
        if (lane == 0) part[warp] = m;
        __syncthreads();
        m = part[0];
        for (int w = 1; w < blockDim.x >> 5; ++w) m = max(m, part[w]);
    }
    const int e = nvfp4_row_exponent(m);
    const float unit = exp2_int(-e);
    if (first == 0) exponents[row] = e;
    bool low = false;
    auto tile = [&](const uint4& b, int64_t t) {
        const uint32_t word = nvfp4_scale_bytes(b, unit);
        low |= nvfp4_low_scales(word);
        *reinterpret_cast<uint32_t*>(scales + mx4_scale_word(row, t, tiles)) = word;
    };
#pragma unroll
    for (int j = 0; j < KEPT; ++j)
        if (first + j * step < tiles) tile(kept[j], first + j * step);
    for (int64_t t = first + KEPT * step; t < tiles; t += step) tile(src[t], t);
    if (!low) return;
#pragma unroll 1
    for (int64_t t = first; t < tiles; t += step) {
        const uint32_t word = nvfp4_scale_bytes(src[t], unit);
        if (nvfp4_low_scales(word)) remake_codes<float>(word, src[t], e, t, row, K, codes + row * ldq, nullptr, 0);
    }
}

// The same for what mx4_columns_kernel leaves: for every 256 k the blocks'
// magnitudes, 16 a row, and after all of them the rows' largest.  A block of
// threads takes the 128 rows of a scale tile and 1024 k: all it reads and the
// scales it writes are contiguous.  (8192 x 16384: 15 us; 22 with a row for a
// block of threads, whose scales left 4 bytes at a time.)
template <typename T>
__global__ void __launch_bounds__(256) nvfp4_finish_columns_kernel(const uint32_t* most, int64_t R, int64_t K, uint8_t* codes,
                                                                   int64_t ldq, uint8_t* scales, int32_t* exponents,
                                                                   const T* X, int64_t ldx) {
    constexpr int KTS = 4, N = 128 * 4 * KTS / 256;
    __shared__ uint32_t part[2][128];
    __shared__ __align__(16) uint32_t words[KTS * 4][128];  // a scale tile each, stored 16 bytes at a time
    pdl_wait();
    pdl_launch_dependents();
    const int64_t r0 = (int64_t)blockIdx.x * 128, kt0 = (int64_t)blockIdx.y * KTS, kts = (K + MX4_TILE_K - 1) / MX4_TILE_K;
    const int64_t tiles = kts * 4;
    const int at = threadIdx.x % 4, i0 = threadIdx.x / 4;  // tile of its 256 k, row (and the 64th after it)
    uint4 b[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int64_t kt = kt0 + j / 2, row = r0 + i0 + j % 2 * 64;
        b[j] = kt < kts && row < R ? reinterpret_cast<const uint4*>(most)[(kt * R + row) * 4 + at] : make_uint4(0, 0, 0, 0);
    }
    {
        const int i = threadIdx.x % 128, half = threadIdx.x / 128;
        const uint32_t* rows = most + kts * R * 16 + r0 + i;
        uint32_t m = 0;
        if (r0 + i < R) {
#pragma unroll 8
            for (int64_t kt = half; kt < kts; kt += 2) m = max(m, rows[kt * R]);
        }
        part[half][i] = m;
    }
    __syncthreads();
    int e[2];
    float unit[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        e[j] = nvfp4_row_exponent(max(part[0][i0 + j * 64], part[1][i0 + j * 64]));
        unit[j] = exp2_int(-e[j]);
        if (blockIdx.y == 0 && at == 0 && r0 + i0 + j * 64 < R) exponents[r0 + i0 + j * 64] = e[j];
    }
    uint32_t low = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint32_t word = nvfp4_scale_bytes(b[j], unit[j % 2]);
        const int i = i0 + j % 2 * 64;
        words[j / 2 * 4 + at][i % 32 * 4 + i / 32] = word;
        low |= (uint32_t)nvfp4_low_scales(word) << j;
    }
    __syncthreads();
    const int64_t left = min((int64_t)KTS * 4, tiles - kt0 * 4);
    uint8_t* to = scales + mx4_scale_word(r0, kt0 * 4, tiles);
    if (r0 + 128 <= R) {
#pragma unroll
        for (int i = threadIdx.x; i < KTS * 4 * 32; i += 256)
            if (i / 32 < left)
                reinterpret_cast<uint4*>(to)[i] = *reinterpret_cast<const uint4*>(&words[i / 32][i % 32 * 4]);
    } else {
        for (int i = threadIdx.x; i < KTS * 4 * 128; i += 256)
            if (i / 128 < left && r0 + i % 128 / 4 + i % 4 * 32 < R) reinterpret_cast<uint32_t*>(to)[i] = words[i / 128][i % 128];
    }
    while (low != 0u) {
        const int j = __ffs(low) - 1;
        low &= low - 1;
        const int64_t kt = kt0 + j / 2, row = r0 + i0 + j % 2 * 64;
        const uint4 again = reinterpret_cast<const uint4*>(most)[(kt * R + row) * 4 + at];
        remake_codes(nvfp4_scale_bytes(again, unit[j % 2]), again, e[j % 2], kt * 4 + at, row, K, codes + row * ldq, X, ldx);
    }
}

// The values a matrix stands for: one warp for 1024 k of a row, in four steps
// of 8 codes a lane (whole 512-byte runs of 16-bit values leave a warp at
// once), all of their codes and scales loaded before the first conversion.
constexpr int DSTEPS = 4;
template <typename T, int FMT>
__global__ void __launch_bounds__(QWARPS * 32) mx4_dequantize_kernel(const uint8_t* codes, int64_t ldq,
                                                                     const uint8_t* scales, const int32_t* exponents,
                                                                     int64_t rows, int64_t K, T* X, int64_t ldx,
                                                                     bool vec) {
    constexpr int LANES = mx4_block(FMT) / 8;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, block = lane / LANES;
    const int64_t kts = (K + MX4_TILE_K - 1) / MX4_TILE_K, steps = (kts + DSTEPS - 1) / DSTEPS;
    const int64_t item = (int64_t)blockIdx.x * QWARPS + (threadIdx.x >> 5);
    if (item >= rows * steps) return;
    const int64_t row = item / steps, kt0 = item % steps * DSTEPS;
    const uint8_t* src = codes + row * ldq;
    const uint8_t* sc = scales + mx4_scale_word(row, 0, mx4_scale_tiles(FMT, K)) + block % 4;
    const float2 unit = FMT == kMxfp4 ? make_float2(1.0f, 1.0f) : exp2_factors(exponents[row]);
    uint32_t w[DSTEPS], byte[DSTEPS];
#pragma unroll
    for (int j = 0; j < DSTEPS; ++j) {
        const int64_t kt = kt0 + j, k0 = kt * MX4_TILE_K + lane * 8;
        w[j] = byte[j] = 0;
        if (k0 < K) {
            w[j] = *reinterpret_cast<const uint32_t*>(src + k0 / 2);
            byte[j] = sc[(kt * mx4_tiles_per_k(FMT) + block / 4) * 512];
        }
    }
#pragma unroll
    for (int j = 0; j < DSTEPS; ++j) {
        const int64_t k0 = (kt0 + j) * MX4_TILE_K + lane * 8;
        if (k0 >= K) return;
        float y[8];
        e2m1_unpack8(w[j], y);
        const float s = FMT == kMxfp4 ? mxfp4_scale(byte[j]) : e4m3_value(byte[j]) * unit.x;  // exact
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = FMT == kMxfp4 ? y[i] * s : y[i] * s * unit.y;
        T* dst = X + row * ldx + k0;
        if (vec && k0 + 8 <= K) {
            store8(dst, y);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k0 + i < K) dst[i] = from_float<T>(y[i]);
        }
    }
}

template <typename T>
cudaError_t quantize_typed(const Mx4Quantize& q, const T* X, cudaStream_t st) {
    const int64_t kts = (q.K + MX4_TILE_K - 1) / MX4_TILE_K;
    if (!q.cols) {
        const bool vec = (uintptr_t)X % 16 == 0 && q.ldx * sizeof(T) % 16 == 0 && q.K % 8 == 0;
        if (q.fmt == kMxfp4) {
            // four tiles a warp once that leaves every SM its 64 warps
            const bool many = q.rows * kts >= 4 * 64 * device_sms();
            const int64_t items = many ? q.rows * ((kts + 3) / 4) : q.rows * kts;
            return launch_pdl(many ? mxfp4_rows_kernel<T, 4> : mxfp4_rows_kernel<T, 1>,
                              dim3((unsigned)((items + QWARPS - 1) / QWARPS)), dim3(QWARPS * 32), 0, st, X, q.ldx,
                              q.rows, q.K, vec, q.codes, q.ldq, q.scales);
        }
        const unsigned warps = (unsigned)(kts < ROW_WARPS ? kts : ROW_WARPS);
        return launch_pdl(nvfp4_rows_kernel<T>, dim3((unsigned)q.rows), dim3(warps * 32), 0, st, X, q.ldx, q.K, vec,
                          q.codes, q.ldq, q.scales, q.exponents);
    }
    const bool vec = (uintptr_t)X % (2 * sizeof(T)) == 0 && q.ldx % 2 == 0;
    const dim3 grid((unsigned)((q.rows + 63) / 64), (unsigned)kts);
    const cudaError_t err =
        q.fmt == kMxfp4 ? launch_pdl(mx4_columns_kernel<T, kMxfp4>, grid, dim3(256), 0, st, X, q.ldx, q.rows, q.K, vec,
                                     q.codes, q.ldq, q.scales, (float*)nullptr)
                        : launch_pdl(mx4_columns_kernel<T, kNvfp4>, grid, dim3(256), 0, st, X, q.ldx, q.rows, q.K, vec,
                                     q.codes, q.ldq, (uint8_t*)nullptr, q.most);
    if (err != cudaSuccess || q.fmt == kMxfp4) return err;
    return launch_pdl(nvfp4_finish_columns_kernel<T>, dim3((unsigned)((q.rows + 127) / 128), (unsigned)((kts + 3) / 4)),
                      dim3(256), 0, st, reinterpret_cast<const uint32_t*>(q.most), q.rows, q.K, q.codes, q.ldq, q.scales,
                      q.exponents, X, q.ldx);
}

template <typename T>
cudaError_t dequantize_typed(int fmt, int64_t rows, int64_t K, const uint8_t* codes, int64_t ldq,
                             const uint8_t* scales, const int32_t* exponents, T* X, int64_t ldx, cudaStream_t st) {
    const int64_t items = rows * ((K + DSTEPS * MX4_TILE_K - 1) / (DSTEPS * MX4_TILE_K));
    const bool vec = (uintptr_t)X % 16 == 0 && ldx * sizeof(T) % 16 == 0;
    const dim3 grid((unsigned)((items + QWARPS - 1) / QWARPS)), block(QWARPS * 32);
    return fmt == kMxfp4 ? launch_pdl(mx4_dequantize_kernel<T, kMxfp4>, grid, block, 0, st, codes, ldq, scales,
                                      exponents, rows, K, X, ldx, vec)
                         : launch_pdl(mx4_dequantize_kernel<T, kNvfp4>, grid, block, 0, st, codes, ldq, scales,
                                      exponents, rows, K, X, ldx, vec);
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Quantize& q, cudaStream_t st) {
    if (q.rows == 0 || q.K == 0) return cudaSuccess;
    switch (q.type) {
        case DDGEMM_F32: return quantize_typed(q, static_cast<const float*>(q.X), st);
        case DDGEMM_BF16: return quantize_typed(q, static_cast<const __nv_bfloat16*>(q.X), st);
        default: return quantize_typed(q, static_cast<const __half*>(q.X), st);
    }
}

cudaError_t launch_nvfp4_finish(const float* most, int64_t rows, int64_t K, uint8_t* codes, int64_t ldq, uint8_t* scales,
                                int32_t* exponents, cudaStream_t st) {
    if (rows == 0 || K == 0) return cudaSuccess;
    const int64_t tiles = mx4_scale_tiles(kNvfp4, K);
    if (rows >= 16 * device_sms() && tiles <= 128)
        return launch_pdl(nvfp4_finish_kernel<true>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, most, rows, K,
                          codes, ldq, scales, exponents);
    const unsigned threads = (unsigned)(tiles >= 256 ? 256 : (tiles + 31) / 32 * 32);
    return launch_pdl(nvfp4_finish_kernel<false>, dim3((unsigned)rows), dim3(threads), 0, st, most, rows, K, codes, ldq,
                      scales, exponents);
}

cudaError_t launch_mx4_dequantize(int fmt, int type, int64_t rows, int64_t K, const uint8_t* codes, int64_t ldq,
                                  const uint8_t* scales, const int32_t* exponents, void* X, int64_t ldx,
                                  cudaStream_t st) {
    if (rows == 0 || K == 0) return cudaSuccess;
    switch (type) {
        case DDGEMM_F32:
            return dequantize_typed(fmt, rows, K, codes, ldq, scales, exponents, static_cast<float*>(X), ldx, st);
        case DDGEMM_BF16:
            return dequantize_typed(fmt, rows, K, codes, ldq, scales, exponents, static_cast<__nv_bfloat16*>(X), ldx, st);
        default:
            return dequantize_typed(fmt, rows, K, codes, ldq, scales, exponents, static_cast<__half*>(X), ldx, st);
    }
}

}  // namespace ddg
