// mx4.cu -- conversion to and from the 4-bit microscaled formats (mx4.cuh).
//
// Quantisation reads each value once and writes 4 bits and its share of a
// scale byte: bound by HBM (2.56 bytes per 16-bit value for nvfp4, 2.53 for
// mxfp4; the conversions are about 3 instructions per value).
#include "launch.cuh"
#include "mx4.cuh"

namespace ddg {
namespace {

constexpr int QWARPS = 8;  // warps per block of the row kernels

// A lane's 8 values of a row, k = k0 .. k0 + 7 (zero beyond K).
template <typename T>
__device__ __forceinline__ void load_row8(const T* row, int64_t k0, int64_t K, bool vec, float (&x)[8]) {
    if (vec && k0 + 8 <= K) {
        load8(row + k0, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = k0 + i < K ? to_float<T>(row[k0 + i]) : 0.0f;
    }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A warp's 256 k of one row: codes and scale words.  `unit` is 2^-e of an
// nvfp4 row.
template <int FMT>
__device__ __forceinline__ void quantize_tile(const float (&x)[8], float unit, int lane, int64_t row, int64_t kt,
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
        byte = nvfp4_scale_byte(m, unit);
        const float s = e4m3_value(byte), r = byte == 0u || byte == 127u ? 0.0f : __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = r == 0.0f ? 0.0f : quotient(x[i] * unit, s, r);
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

// mxfp4 rows: one warp for 256 k of a row.
template <typename T>
__global__ void __launch_bounds__(QWARPS * 32) mxfp4_rows_kernel(const T* X, int64_t ldx, int64_t rows, int64_t K,
                                                                 bool vec, uint8_t* codes, int64_t ldq,
                                                                 uint8_t* scales) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t kts = (K + MX4_TILE_K - 1) / MX4_TILE_K;
    const int64_t item = (int64_t)blockIdx.x * QWARPS + (threadIdx.x >> 5);
    if (item >= rows * kts) return;
    const int64_t row = item / kts, kt = item % kts;
    float x[8];
    load_row8(X + row * ldx, kt * MX4_TILE_K + lane * 8, K, vec, x);
    quantize_tile<kMxfp4>(x, 1.0f, lane, row, kt, K, codes, ldq, scales);
}

// nvfp4 rows: one block for a row.  The row's values stay in registers
// between the maximum and the conversion as far as KEEP tiles per warp reach
// (8 warps: 16384 values of 16 bits, 8192 of 32); longer rows are read again.
template <typename T>
__global__ void __launch_bounds__(QWARPS * 32) nvfp4_rows_kernel(const T* X, int64_t ldx, int64_t K, bool vec,
                                                                 uint8_t* codes, int64_t ldq, uint8_t* scales,
                                                                 int32_t* exponents) {
    constexpr int KEEP = sizeof(T) == 2 ? 8 : 4;
    __shared__ uint32_t part[QWARPS];
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
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        const int64_t kt = warp + (int64_t)j * warps;
        if (kt < kts) load_row8(src, kt * MX4_TILE_K + lane * 8, K, vec, keep[j]);
    }
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
        if (warp + (int64_t)j * warps < kts) take(keep[j]);
    for (int64_t kt = warp + (int64_t)KEEP * warps; kt < kts; kt += warps) {
        float x[8];
        load_row8(src, kt * MX4_TILE_K + lane * 8, K, vec, x);
        take(x);
    }
    m = __reduce_max_sync(~0u, m);
    if (lane == 0) part[warp] = m;
    __syncthreads();
    m = part[0];
    for (int w = 1; w < warps; ++w) m = max(m, part[w]);
    const int e = nvfp4_row_exponent(m);
    const float unit = exp2_int(-e);
    if (threadIdx.x == 0) exponents[row] = e;
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
        const int64_t kt = warp + (int64_t)j * warps;
        if (kt < kts) quantize_tile<kNvfp4>(keep[j], unit, lane, row, kt, K, codes, ldq, scales);
    }
    for (int64_t kt = warp + (int64_t)KEEP * warps; kt < kts; kt += warps) {
        float x[8];
        load_row8(src, kt * MX4_TILE_K + lane * 8, K, vec, x);
        quantize_tile<kNvfp4>(x, unit, lane, row, kt, K, codes, ldq, scales);
    }
}

// Two consecutive elements of a row of X as floats (zero beyond R).
template <typename T>
__device__ __forceinline__ void load_pair(const T* row, int64_t c, int64_t R, bool vec, float& a, float& b) {
    if (vec && c + 2 <= R) {
        struct alignas(2 * sizeof(T)) Two { T a, b; };
        const Two t = *reinterpret_cast<const Two*>(row + c);
        a = to_float<T>(t.a);
        b = to_float<T>(t.b);
    } else {
        a = c < R ? to_float<T>(row[c]) : 0.0f;
        b = c + 1 < R ? to_float<T>(row[c + 1]) : 0.0f;
    }
}

// Largest finite magnitude of each column of X (K x R), as bits, over 256
// rows per block: 64 columns, 8 warps of 32 rows.
template <typename T>
__global__ void __launch_bounds__(256) column_max_kernel(const T* X, int64_t ldx, int64_t R, int64_t K, bool vec,
                                                         uint32_t* most) {
    __shared__ uint32_t part[8][64];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane * 2, k0 = (int64_t)blockIdx.y * 256 + warp * 32;
    uint32_t m0 = 0, m1 = 0;
#pragma unroll 16
    for (int i = 0; i < 32; ++i) {
        float a = 0.0f, b = 0.0f;
        if (k0 + i < K) load_pair(X + (k0 + i) * ldx, c, R, vec, a, b);
        const uint32_t x = abs_bits(a), y = abs_bits(b);
        m0 = max(m0, x < kInfBits ? x : 0u);
        m1 = max(m1, y < kInfBits ? y : 0u);
    }
    part[warp][lane * 2] = m0;
    part[warp][lane * 2 + 1] = m1;
    __syncthreads();
    if (threadIdx.x < 64 && (int64_t)blockIdx.x * 64 + threadIdx.x < R) {
        uint32_t m = part[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max(m, part[w][threadIdx.x]);
        if (m > 0) atomicMax(most + (int64_t)blockIdx.x * 64 + threadIdx.x, m);
    }
}

// Columns of X (K x R) as rows of the result: a block takes 64 columns and 256
// k.  Warp w reads rows 32 w .. + 31, a lane two columns of them, so a lane
// holds whole blocks of k and needs no exchange for their maxima; codes and
// scales go through shared memory and leave as whole 128-byte rows.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) mx4_columns_kernel(const T* X, int64_t ldx, int64_t R, int64_t K, bool vec,
                                                          const uint32_t* most, uint8_t* codes, int64_t ldq,
                                                          uint8_t* scales, int32_t* exponents) {
    constexpr int BLOCK = mx4_block(FMT), WORDS = mx4_tiles_per_k(FMT);
    __shared__ __align__(16) uint8_t code[64][128 + 16];
    __shared__ __align__(16) uint8_t scale[64][4 * WORDS];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * 64, kt = blockIdx.y;
    const int64_t c = r0 + lane * 2, k0 = kt * MX4_TILE_K + warp * 32;
    float x[2][32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        x[0][i] = x[1][i] = 0.0f;
        if (k0 + i < K) load_pair(X + (k0 + i) * ldx, c, R, vec, x[0][i], x[1][i]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = lane * 2 + j;
        int e = 0;
        if (FMT == kNvfp4 && r0 + row < R) {
            e = nvfp4_row_exponent(most[r0 + row]);
            if (kt == 0 && warp == 0) exponents[r0 + row] = e;
        }
        const float unit = exp2_int(-e);
#pragma unroll
        for (int b = 0; b < 32 / BLOCK; ++b) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) m = max(m, abs_bits(x[j][b * BLOCK + i]));
            uint32_t byte;
            float s = 1.0f, r;
            if (FMT == kMxfp4) {
                byte = mxfp4_scale_byte(m);
                r = mxfp4_inverse(byte);
            } else {
                byte = nvfp4_scale_byte(m, unit);
                s = e4m3_value(byte);
                r = byte == 0u || byte == 127u ? 0.0f : __frcp_rn(s);
            }
            scale[row][warp * (32 / BLOCK) + b] = (uint8_t)byte;
#pragma unroll
            for (int q = 0; q < BLOCK / 8; ++q) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = x[j][b * BLOCK + q * 8 + i];
                    y[i] = FMT == kMxfp4 ? v * r : r == 0.0f ? 0.0f : quotient(v * unit, s, r);
                }
                *reinterpret_cast<uint32_t*>(&code[row][warp * 16 + b * (BLOCK / 2) + q * 4]) = e2m1_pack8(y);
            }
        }
    }
    __syncthreads();
    // 64 rows of 128 bytes, 16 bytes a thread: 8 threads a row
    const int64_t bytes = mx4_code_bytes(K);
#pragma unroll
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int row = i / 8, at = i % 8 * 16;
        if (r0 + row < R && kt * 128 + at < bytes)
            *reinterpret_cast<uint4*>(codes + (r0 + row) * ldq + kt * 128 + at) =
                *reinterpret_cast<const uint4*>(&code[row][at]);
    }
    const int64_t tiles = mx4_scale_tiles(FMT, K);
    for (int i = threadIdx.x; i < 64 * WORDS; i += 256) {
        const int row = i % 64, w = i / 64;
        if (r0 + row < R)
            *reinterpret_cast<uint32_t*>(scales + mx4_scale_word(r0 + row, kt * WORDS + w, tiles)) =
                *reinterpret_cast<const uint32_t*>(&scale[row][w * 4]);
    }
}

// The values a matrix stands for: one warp for 256 k of a row, 8 codes a lane.
template <typename T, int FMT>
__global__ void __launch_bounds__(QWARPS * 32) mx4_dequantize_kernel(const uint8_t* codes, int64_t ldq,
                                                                     const uint8_t* scales, const int32_t* exponents,
                                                                     int64_t rows, int64_t K, T* X, int64_t ldx,
                                                                     bool vec) {
    constexpr int LANES = mx4_block(FMT) / 8;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t kts = (K + MX4_TILE_K - 1) / MX4_TILE_K;
    const int64_t item = (int64_t)blockIdx.x * QWARPS + (threadIdx.x >> 5);
    if (item >= rows * kts) return;
    const int64_t row = item / kts, kt = item % kts, k0 = kt * MX4_TILE_K + lane * 8;
    if (k0 >= K) return;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + row * ldq + k0 / 2);
    const int block = lane / LANES;
    const uint32_t byte = scales[mx4_scale_word(row, kt * mx4_tiles_per_k(FMT) + block / 4, mx4_scale_tiles(FMT, K)) +
                                 block % 4];
    float y[8];
    e2m1_unpack8(w, y);
    const float s = FMT == kMxfp4 ? mxfp4_scale(byte) : e4m3_value(byte);
    const float unit = FMT == kMxfp4 ? 1.0f : exp2_int(exponents[row]);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * s * unit;
    T* dst = X + row * ldx + k0;
    if (vec && k0 + 8 <= K) {
        store8(dst, y);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k0 + i < K) dst[i] = from_float<T>(y[i]);
    }
}

template <typename T>
cudaError_t quantize_typed(const Mx4Quantize& q, const T* X, cudaStream_t st) {
    const int64_t kts = (q.K + MX4_TILE_K - 1) / MX4_TILE_K;
    if (!q.cols) {
        const bool vec = (uintptr_t)X % 16 == 0 && q.ldx * sizeof(T) % 16 == 0;
        if (q.fmt == kMxfp4) {
            const int64_t items = q.rows * kts;
            return launch_pdl(mxfp4_rows_kernel<T>, dim3((unsigned)((items + QWARPS - 1) / QWARPS)),
                              dim3(QWARPS * 32), 0, st, X, q.ldx, q.rows, q.K, vec, q.codes, q.ldq, q.scales);
        }
        const unsigned warps = (unsigned)(kts < QWARPS ? kts : QWARPS);
        return launch_pdl(nvfp4_rows_kernel<T>, dim3((unsigned)q.rows), dim3(warps * 32), 0, st, X, q.ldx, q.K, vec,
                          q.codes, q.ldq, q.scales, q.exponents);
    }
    const bool vec = (uintptr_t)X % (2 * sizeof(T)) == 0 && q.ldx % 2 == 0;
    const dim3 grid((unsigned)((q.rows + 63) / 64), (unsigned)kts);
    if (q.fmt == kMxfp4)
        return launch_pdl(mx4_columns_kernel<T, kMxfp4>, grid, dim3(256), 0, st, X, q.ldx, q.rows, q.K, vec,
                          (const uint32_t*)nullptr, q.codes, q.ldq, q.scales, (int32_t*)nullptr);
    cudaError_t err = cudaMemsetAsync(q.column_max, 0, (size_t)q.rows * 4, st);
    if (err != cudaSuccess) return err;
    // the maxima follow a memset, which is no kernel: an ordinary launch
    column_max_kernel<T><<<grid, 256, 0, st>>>(X, q.ldx, q.rows, q.K, vec, q.column_max);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return launch_pdl(mx4_columns_kernel<T, kNvfp4>, grid, dim3(256), 0, st, X, q.ldx, q.rows, q.K, vec,
                      (const uint32_t*)q.column_max, q.codes, q.ldq, q.scales, q.exponents);
}

template <typename T>
cudaError_t dequantize_typed(int fmt, int64_t rows, int64_t K, const uint8_t* codes, int64_t ldq,
                             const uint8_t* scales, const int32_t* exponents, T* X, int64_t ldx, cudaStream_t st) {
    const int64_t items = rows * ((K + MX4_TILE_K - 1) / MX4_TILE_K);
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
