// mx4_gemm.cu -- products of matrices in 4-bit microscaled form
// (C = alpha A B^T) and the two products of the 4-bit gated block: operands,
// epilogues and launches for the two kernels that multiply.  Up to 64 rows of A
// the weights are what has to be moved and split_gemm.cuh streams them over all
// SMs (1 x 8192 x 8192 nvfp4 9.1 us from HBM, 6.8 from L2); more rows are the tensor
// pipe's work and go by CTA pairs in tile_gemm.cuh (8192^3 nvfp4 161 us).
#include <cmath>

#include "activation.cuh"
#include "mx4.cuh"
#include "split_gemm.cuh"
#include "tile_gemm.cuh"

namespace ddg {
namespace {

// The row exponents of an nvfp4 operand for 32 columns: lane i holds that of
// column c + i (0 beyond N).
__device__ __forceinline__ int column_exponent(const int32_t* f, int64_t c, int64_t N, int lane) {
    return f != nullptr && c + lane < N ? f[c + lane] : 0;
}

// 32 values of a row times 2^(er + f_j + ea), lane j holding f_j.  Exponents of
// ordinary size take two multiplications by powers of two; the rest go by their
// sum, lest a partial product leave the range (or its normal part) alone.
__device__ __forceinline__ bool ordinary_exponent(int e) { return (uint32_t)e + 40u <= 80u; }
__device__ __forceinline__ void scale_columns(float (&v)[32], int er, int fc, int ea) {
    if (__all_sync(~0u, ordinary_exponent(er) && ordinary_exponent(fc) && ordinary_exponent(ea))) {
        const float row = exp2_int(er + ea), column = exp2_int(fc);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= row * __shfl_sync(~0u, column, i);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = scale_by_exp2(v[i], add_exponents(add_exponents(er, __shfl_sync(~0u, fc, i)), ea));
    }
}

// alpha as it enters the epilogues: of nvfp4, whose accumulators get a power of two
// besides, a factor in [1/2, 1) and an exponent that joins the rows', so that no
// partial product leaves the range where the result does not.
struct Factor {
    float value;
    int exponent;
};
Factor split_factor(int kind, float alpha) {
    Factor f{alpha, 0};
    if (kind == kKindNv && std::isfinite(alpha)) f.value = std::frexp(alpha, &f.exponent);
    return f;
}

// C = alpha * accumulators * 2^(e_i + f_j), rounded once.
template <int KIND, typename T, int NT_, bool ALIGNED>
struct EpiScale {
    static constexpr int NT = NT_, GROUPS = NT / 64;
    T* C;
    int64_t ldc, M, N;
    const int32_t *e, *f;
    Factor alpha;
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int, int, int64_t row, int nt, int group, int lane, Release release) const {
        const int er = KIND == kKindNv && row < M ? e[row] : 0;
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
            const int c = group * 64 + j * 32;
            const int64_t col = (int64_t)nt * NT + c;
            uint32_t v[32];
            tc5::ld32(acc + c, v);
            if (j == 1) release();
            if (col >= N) continue;
            float o[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(v[i]) * alpha.value;
            if (KIND == kKindNv) {
                scale_columns(o, er, column_exponent(f, col, N, lane), alpha.exponent);
            }
            store_block<ALIGNED>(C, ldc, row - lane, M, col, N, o, lane);
        }
    }
};

// A block of hidden values: 16 of a thread's 32 (nvfp4), codes made before the
// row's exponent is known; the largest finite magnitude, marked by the sign bit
// if the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t nonfinite_mark(uint32_t bits) { return bits >= kInfBits ? 0x80000000u : 0u; }
__device__ __forceinline__ float nvfp4_hidden_block(const float* h, uint32_t (&w)[2]) {
    uint32_t m = 0, mark = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t b = __float_as_uint(h[i]) & 0x7fffffffu;
        mark |= nonfinite_mark(b);
        m = max(m, b < kInfBits ? b : 0u);
    }
    const float s = nvfp4_wide_step(m), r = s > 0.0f ? __frcp_rn(s) : 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = quotient(h[k * 8 + i], s, r);
        w[k] = e2m1_pack8(y);
    }
    return __uint_as_float(m | mark);
}

// h = act(g) * u, both in 32 bits, from 32 columns of g and 32 of u in turn:
// a thread holds 32 hidden values of its row, whole blocks of either format.
// The last tile also clears the padding of k.
template <int KIND, int NT_>
struct EpiGate4 {
    static constexpr int NT = NT_, GROUPS = NT / 64;
    uint8_t *codes, *scales;
    float* most;  // nvfp4: instead of the scales
    int64_t ld;   // bytes of a row of codes
    int64_t M, F;
    int nt;       // n tiles
    const int32_t *e, *f;
    int act;
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int, int, int64_t row, int n, int group, int lane, Release release) const {
        uint32_t raw[32];
        float g[32], u[32];
        tc5::ld32(acc + group * 64, raw);
#pragma unroll
        for (int i = 0; i < 32; ++i) g[i] = __uint_as_float(raw[i]);
        tc5::ld32(acc + group * 64 + 32, raw);
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] = __uint_as_float(raw[i]);
        release();
        const int64_t c = (int64_t)n * (NT / 2) + group * 32;
        if (KIND == kKindNv) {
            const int64_t wc = (int64_t)n * NT + group * 64, W = round_up(F, 32) * 2;
            const int er = row < M ? e[row] : 0;
            scale_columns(g, er, column_exponent(f, wc, W, lane), 0);
            scale_columns(u, er, column_exponent(f, wc + 32, W, lane), 0);
        }
        if (row >= M) return;
        constexpr int FMT = KIND == kKindMx ? kMxfp4 : kNvfp4;
        const int64_t tiles = mx4_scale_tiles(FMT, F);
        if (c < F) {
            float hv[32];
            with_activation(act, [&](auto tag) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float a, da;
                    activation<decltype(tag)::value, false>(g[i], a, da);
                    hv[i] = c + i < F ? a * u[i] : 0.0f;  // rows that fill up W take no part
                }
            });
            uint32_t w[4];
            if (KIND == kKindMx) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(hv[i]) & 0x7fffffffu);
                const uint32_t byte = mxfp4_scale_byte(m);
                const float inv = mxfp4_inverse(byte);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = hv[k * 8 + i] * inv;
                    w[k] = e2m1_pack8(y);
                }
                const int64_t b = c / 32;
                scales[mx4_scale_word(row, b / 4, tiles) + b % 4] = (uint8_t)byte;
            } else {
                float2 m;
                uint32_t lo[2], hi[2];
                m.x = nvfp4_hidden_block(hv, lo);
                m.y = nvfp4_hidden_block(hv + 16, hi);
                w[0] = lo[0], w[1] = lo[1], w[2] = hi[0], w[3] = hi[1];
                *reinterpret_cast<float2*>(most + row * tiles * 4 + c / 16) = m;
            }
            *reinterpret_cast<uint4*>(codes + row * ld + c / 2) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (n == nt - 1 && group == GROUPS - 1) {
            if (KIND == kKindMx)
                for (int64_t b = (F + 31) / 32; b < tiles * 4; ++b) scales[mx4_scale_word(row, b / 4, tiles) + b % 4] = 0;
            else
                for (int64_t b = (F + 31) / 32 * 2; b < tiles * 4; ++b) most[row * tiles * 4 + b] = 0.0f;
        }
    }
};

// The same two epilogues for the split kernel: one value per lane.
template <int KIND, typename T>
struct EpiSplitScale {
    static constexpr int UNITS = 1, HALVES = 1;
    T* C;
    int64_t ldc, N;
    const int32_t *e, *f;
    Factor alpha;
    __device__ __forceinline__ void emit(float v, float, int64_t m, int unit, int lane, int tile) const {
        const int64_t n = (int64_t)tile * 128 + unit * 32 + lane;
        if (n >= N) return;
        v *= alpha.value;
        if (KIND == kKindNv) v = scale_by_exp2(v, add_exponents(add_exponents(e[m], f[n]), alpha.exponent));
        C[m * ldc + n] = from_float<T>(v);
    }
};

template <int KIND>
struct EpiSplitGate4 {
    static constexpr int UNITS = 2, HALVES = 1;
    uint8_t *codes, *scales;
    float* most;
    int64_t ld, F;
    const int32_t *e, *f;
    int act;
    __device__ __forceinline__ void emit(float g, float u, int64_t m, int unit, int lane, int tile) const {
        const int64_t b = (int64_t)tile * 2 + unit, n = b * 32 + lane;  // 32 hidden values
        if (b * 32 >= F) return;
        if (KIND == kKindNv) {
            const int er = e[m];
            g = scale_by_exp2(g, add_exponents(er, f[b * 64 + lane]));
            u = scale_by_exp2(u, add_exponents(er, f[b * 64 + 32 + lane]));
        }
        float a = 0.0f, da;
        with_activation(act, [&](auto tag) { activation<decltype(tag)::value, false>(g, a, da); });
        const float hv = n < F ? a * u : 0.0f;  // rows that fill up W take no part
        const uint32_t bits = __float_as_uint(hv) & 0x7fffffffu;
        constexpr int FMT = KIND == kKindMx ? kMxfp4 : kNvfp4;
        const int64_t tiles = mx4_scale_tiles(FMT, F);
        const bool last = b * 32 + 32 >= F;
        float q;
        if (KIND == kKindMx) {
            const uint32_t byte = mxfp4_scale_byte(__reduce_max_sync(~0u, bits));
            q = hv * mxfp4_inverse(byte);
            if (lane == 0) {
                scales[mx4_scale_word(m, b / 4, tiles) + b % 4] = (uint8_t)byte;
                if (last)  // the padding of k
                    for (int64_t p = b + 1; p < tiles * 4; ++p) scales[mx4_scale_word(m, p / 4, tiles) + p % 4] = 0;
            }
        } else {
            uint32_t top = bits < kInfBits ? bits : 0u, mark = nonfinite_mark(bits);
#pragma unroll
            for (int d = 1; d < 16; d *= 2) {  // of 16 lanes
                top = max(top, __shfl_xor_sync(~0u, top, d));
                mark |= __shfl_xor_sync(~0u, mark, d);
            }
            const float s = nvfp4_wide_step(top), r = s > 0.0f ? __frcp_rn(s) : 0.0f;
            q = quotient(hv, s, r);
            float* row = most + m * tiles * 4;
            if (lane % 16 == 0) row[b * 2 + lane / 16] = __uint_as_float(top | mark);
            if (last)
                for (int64_t p = b * 2 + 2 + lane; p < tiles * 4; p += 32) row[p] = 0.0f;
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(~0u, q, (lane & 3) * 8 + i);
        if (lane < 4) *reinterpret_cast<uint32_t*>(codes + m * ld + b * 16 + lane * 4) = e2m1_pack8(y);
    }
};

cudaError_t map_codes(CUtensorMap* m, const Mx4Matrix& x, int box_rows) {
    const int64_t bytes = mx4_code_bytes(x.K), ld = x.rows > 1 ? x.ldq : round_up(bytes, 16);
    return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, x.codes, bytes, x.rows, ld, 128, box_rows, true);
}
cudaError_t map_scales(CUtensorMap* m, int fmt, const Mx4Matrix& x) {
    return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, x.scales, 128,
                       (x.rows + 127) / 128 * mx4_scale_tiles(fmt, x.K), 512, 128, mx4_tiles_per_k(fmt), false);
}

template <int KIND, class Epi>
cudaError_t product4(const Mx4Matrix& A, const Mx4Matrix& B, const Epi& epi, cudaStream_t st) {
    constexpr int FMT = KIND == kKindMx ? kMxfp4 : kNvfp4;
    TileMaps maps;
    memset(&maps, 0, sizeof(maps));
    cudaError_t err = map_codes(&maps.a[0], A, 128);
    if (err == cudaSuccess) err = map_codes(&maps.b[0], B, Epi::NT / 2);
    if (err == cudaSuccess) err = map_scales(&maps.sa, FMT, A);
    if (err == cudaSuccess) err = map_scales(&maps.sb, FMT, B);
    if (err != cudaSuccess) return err;
    TileArgs g = {};
    g.products = 1;
    TileProduct& q = g.p[0];
    q.mt = (int)((A.rows + 255) / 256);
    q.nt = (int)((B.rows + Epi::NT - 1) / Epi::NT);
    q.nk = (int)((A.K + MX4_TILE_K - 1) / MX4_TILE_K);
    q.segs = 1;
    q.last_steps = (int)((A.K - (int64_t)(q.nk - 1) * MX4_TILE_K + 63) / 64);
    g.tiles_k = (int)mx4_scale_tiles(FMT, A.K);
    return launch_tile_gemm<KIND, kMajorK, false, false>(g, maps, epi, st);
}

// x (tokens x K) times the rows of W.
template <int KIND, class Epi>
cudaError_t split4(const Mx4Matrix& x, const Mx4Matrix& W, bool early, const Epi& epi, cudaStream_t st) {
    constexpr int FMT = KIND == kKindMx ? kMxfp4 : kNvfp4;
    SplitMaps maps;
    memset(&maps, 0, sizeof(maps));
    cudaError_t err = map_codes(&maps.p[0], W, 128);
    if (err == cudaSuccess) err = map_codes(&maps.q, x, split_nq(x.rows));
    if (err != cudaSuccess) return err;
    SplitArgs g = {};
    g.sp = W.scales;
    g.sq = x.scales;
    g.nt = (int)((W.rows + 127) / 128);
    g.nk = (int)((x.K + MX4_TILE_K - 1) / MX4_TILE_K);
    g.last_steps = (int)((x.K - (int64_t)(g.nk - 1) * MX4_TILE_K + 63) / 64);
    g.tiles_k = (int)mx4_scale_tiles(FMT, x.K);
    g.early = early;
    g.M = (int)x.rows;
    return launch_split_gemm<KIND, false>(g, maps, epi, st);
}

int64_t pair_tiles(const Mx4Matrix& A, const Mx4Matrix& B, int nt) { return (A.rows + 255) / 256 * ((B.rows + nt - 1) / nt); }

constexpr double kNarrow4 = 0.78;  // 128 columns for 192: 191 us against 162 for 8192^3 nvfp4
bool narrow4(const Mx4Matrix& A, const Mx4Matrix& B) {
    return narrow_tiles(pair_tiles(A, B, 192), pair_tiles(A, B, 128), kNarrow4);
}

template <int KIND, typename T, int NT, bool ALIGNED>
cudaError_t gemm_sized(const Mx4Gemm& g, cudaStream_t st) {
    return product4<KIND>(g.A, g.B,
                          EpiScale<KIND, T, NT, ALIGNED>{static_cast<T*>(g.C), g.ldc, g.A.rows, g.B.rows, g.A.exponents,
                                                         g.B.exponents, split_factor(KIND, g.alpha)},
                          st);
}

template <int KIND, typename T>
cudaError_t gemm_typed(const Mx4Gemm& g, cudaStream_t st) {
    T* C = static_cast<T*>(g.C);
    if (g.A.rows <= kSplitTokens4)
        return split4<KIND>(g.A, g.B, g.early,
                            EpiSplitScale<KIND, T>{C, g.ldc, g.B.rows, g.A.exponents, g.B.exponents, split_factor(KIND, g.alpha)}, st);
    const bool narrow = narrow4(g.A, g.B), aligned = aligned_rows<T>(C, g.ldc);
    auto f = narrow ? (aligned ? gemm_sized<KIND, T, 128, true> : gemm_sized<KIND, T, 128, false>)
                    : (aligned ? gemm_sized<KIND, T, 192, true> : gemm_sized<KIND, T, 192, false>);
    return f(g, st);
}

template <int KIND>
cudaError_t gemm_kind(const Mx4Gemm& g, cudaStream_t st) {
    switch (g.type) {
        case DDGEMM_F32: return gemm_typed<KIND, float>(g, st);
        case DDGEMM_BF16: return gemm_typed<KIND, __nv_bfloat16>(g, st);
        default: return gemm_typed<KIND, __half>(g, st);
    }
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4Gemm& g, cudaStream_t st) {
    return g.fmt == kMxfp4 ? gemm_kind<kKindMx>(g, st) : gemm_kind<kKindNv>(g, st);
}

namespace {

template <int KIND>
cudaError_t gate_kind(const Mx4Gate& g, cudaStream_t st) {
    uint8_t *codes = const_cast<uint8_t*>(g.hq.codes), *scales = const_cast<uint8_t*>(g.hq.scales);
    const int64_t ld = g.hq.ldq;
    if (g.x.rows <= kSplitTokens4)
        return split4<KIND>(g.x, g.W, true,  // x was quantised by the launch before, which waited for all before it
                            EpiSplitGate4<KIND>{codes, scales, g.most, ld, g.F, g.x.exponents, g.W.exponents, g.act}, st);
    const auto nt = [&](int n) { return (int)((g.W.rows + n - 1) / n); };
    if (narrow4(g.x, g.W))
        return product4<KIND>(g.x, g.W, EpiGate4<KIND, 128>{codes, scales, g.most, ld, g.x.rows, g.F, nt(128), g.x.exponents,
                                                            g.W.exponents, g.act}, st);
    return product4<KIND>(g.x, g.W, EpiGate4<KIND, 192>{codes, scales, g.most, ld, g.x.rows, g.F, nt(192), g.x.exponents,
                                                        g.W.exponents, g.act}, st);
}

}  // namespace

cudaError_t launch_mx4_gate(const Mx4Gate& g, cudaStream_t st) {
    return g.fmt == kMxfp4 ? gate_kind<kKindMx>(g, st) : gate_kind<kKindNv>(g, st);
}

cudaError_t read_and_reset_wait_timeouts_mx4(unsigned int* count) { return reset_tile_timeouts(count); }

}  // namespace ddg
