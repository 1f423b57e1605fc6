// ff.cu -- the gated feed-forward block in 16 bits,
//   y = h Wd^T,  h = act(x Wg^T) * (x Wu^T)      (Wg, Wu: F x D, Wd: D x F)
// and its gradients
//   dh = dy Wd,  dg = dh * u * act'(g),  du = dh * act(g),
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h,
// as products on CTA pairs (tile_gemm.cuh) with the elementwise work in their
// epilogues.  The training form keeps h (16 bits), a = act(g) and
// b = u * act'(g): the backward pass is then dg = dh b, du = dh a and needs
// neither g and u nor the activation again.
//
// a and b enter dg and du as factors, so their rounding adds to that of dg and
// du themselves.  For bfloat16 (8 significant bits) they are kept as float16 (11)
// with a power of two for every 32 of a row, which takes 2 bytes and leaves the
// gradients' error as 32 bits would; for float16 in 32 bits.
//
// h, dg and du are rounded to the type before the next product.  Of many tokens
// these roundings average out: an output's error is 1.41 times that of its own
// rounding.  Of up to kFullTokens the few largest values decide, and it was up
// to 1.55 times: there what the rounding leaves is kept in as many rows more and
// enters the products too (16 significant bits for bfloat16, 22 for float16).
// Where such a sum is not finite it is the one without the remainders: an infinity
// stays one, as of more tokens.  What this costs, us with and without: 4096 x
// 12288, where the weights bind, forward 49.9 and 49.8, backward 155 and 149 (one
// token), 53.4 and 52.5, 151 and 145 (16); small blocks pay for the launch that
// adds dx's two sums up, 512 x 2048, 16 tokens, 8.6 and 8.3, 18.5 and 16.5, 128 x
// 640, one token, 6.9 and 6.7, 15.8 and 11.3.
#include "activation.cuh"
#include "mx4.cuh"
#include "split_gemm.cuh"
#include "tile_gemm.cuh"

namespace ddg {
namespace {

// The planes a and b of the training form: T rows of ld values, and for
// bfloat16 an exponent byte for every 32 of them.
template <typename T> struct Keep;
template <> struct Keep<__half> { using value = float; };
template <> struct Keep<__nv_bfloat16> { using value = __half; };

struct KeepPlanes {
    void *a, *b;
    uint8_t *ea, *eb;
};

// The exponent byte for values whose largest finite magnitude has these bits,
// and the power of two that brings it to [2^14, 2^15).
__device__ __forceinline__ uint32_t keep_byte(uint32_t max_bits) { return max(max_bits >> 23, 15u); }
__device__ __forceinline__ float keep_scale(uint32_t byte) { return exp2_int(14 + 127 - (int)byte); }
__device__ __forceinline__ float keep_inverse(uint32_t byte) { return exp2_int((int)byte - 127 - 14); }
__device__ __forceinline__ uint32_t finite_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b < kInfBits ? b : 0u;
}

// A thread's 32 consecutive values of a row, at `at`.
__device__ __forceinline__ void keep_row(__half* plane, uint8_t* bytes, int64_t at, float (&v)[32]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, finite_bits(v[i]));
    const uint32_t byte = keep_byte(m);
    const float s = keep_scale(byte);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= s;
    store_row(plane + at, v);
    bytes[at / 32] = (uint8_t)byte;
}
__device__ __forceinline__ void keep_row(float* plane, uint8_t*, int64_t at, float (&v)[32]) { store_row(plane + at, v); }

// One value of 32 in a warp.
__device__ __forceinline__ void keep_lane(__half* plane, uint8_t* bytes, int64_t at, float v, int lane) {
    const uint32_t byte = keep_byte(__reduce_max_sync(~0u, finite_bits(v)));
    plane[at] = __float2half_rn(v * keep_scale(byte));
    if (lane == 0) bytes[at / 32] = (uint8_t)byte;
}
__device__ __forceinline__ void keep_lane(float* plane, uint8_t*, int64_t at, float v, int) { plane[at] = v; }

// 16 kept values of a row; `at / 32` is their block.
__device__ __forceinline__ void kept16(const __half* plane, const uint8_t* bytes, int64_t at, float (&v)[16]) {
    uint32_t w[8];
    load_v8(plane + at, w);
    const float s = keep_inverse(bytes[at / 32]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}
__device__ __forceinline__ void kept16(const float* plane, const uint8_t*, int64_t at, float (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t w[8];
        load_v8(plane + at + 8 * k, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * k + i] = __uint_as_float(w[i]);
    }
}

// The part of v that hi, v rounded, leaves (0 where that is infinite or NaN).
template <typename T>
__device__ __forceinline__ float remainder_of(float v, T hi) {
    const float h = to_float<T>(hi);
    return finite_bits(h) == (__float_as_uint(h) & 0x7fffffffu) ? v - h : 0.0f;
}

// v, a sum over rounded values and what the roundings leave, unless that is not
// finite: a remainder times an infinity of the other operand is a NaN of its own
// (0 inf) or has the other sign.  Then the sum over the rounded values alone.
__device__ __forceinline__ bool is_finite(float v) { return (__float_as_uint(v) & 0x7fffffffu) < kInfBits; }
__device__ __forceinline__ float with_rest(float v, float rest) {
    const float sum = v + rest;
    return is_finite(sum) ? sum : v;
}

// A weight gradient of few tokens, C[m, n] = sum over t of a[t, m] b[t, n] and as
// many terms with what the roundings of a (or b) leave, all in one accumulator:
// the terms of the rounded values again, for elements that are not finite.
template <typename T>
struct RoundedTerms {
    const T *a, *b;
    int64_t lda, ldb;
    int tokens;
};
// A bit for each of a thread's values that is not finite; whether a warp has any
// takes one operation a value (0 v is 0 or NaN).
__device__ __forceinline__ uint32_t not_finite(const float (&f)[32]) {
    float nan[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 32; ++i) nan[i % 4] = fmaf(f[i], 0.0f, nan[i % 4]);
    const float any = (nan[0] + nan[1]) + (nan[2] + nan[3]);
    uint32_t bad = 0;
    if (__any_sync(~0u, any != any)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) bad |= is_finite(f[i]) ? 0u : 1u << i;
    }
    return bad;
}
// `bad`: those of a thread's 32 columns from c on of its row, which the warp has
// just stored.
template <typename T>
__device__ __forceinline__ void store_rounded_terms(const RoundedTerms<T>& t, uint32_t bad, T* C, int64_t ldc, int64_t row,
                                                    int64_t M, int64_t c, int64_t N) {
    __syncwarp();
    if (row >= M) return;
#pragma unroll 1
    for (; bad != 0u; bad &= bad - 1) {
        const int64_t col = c + __ffs(bad) - 1;
        if (col >= N) return;
        float sum = 0.0f;
#pragma unroll 1
        for (int i = 0; i < t.tokens; ++i) sum = fmaf(to_float<T>(t.a[i * t.lda + row]), to_float<T>(t.b[i * t.ldb + col]), sum);
        C[row * ldc + col] = from_float<T>(sum);
    }
}

// C = accumulators, rounded once; of each product of a launch.  REST: all of
// them weight gradients with remainders.
template <typename T, int NT_, int P, bool ALIGNED, bool REST>
struct EpiStore {
    static constexpr int NT = NT_, GROUPS = 2;
    T* C[P];
    int64_t ldc[P], M[P], N[P];
    RoundedTerms<T> terms[REST ? P : 1];
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int p, int, int64_t row, int nt, int group, int lane, Release release) const {
        constexpr int STEPS = NT / GROUPS / 32;
#pragma unroll 1
        for (int j = 0; j < STEPS; ++j) {
            const int c = (group * STEPS + j) * 32;
            uint32_t v[32];
            tc5::ld32(acc + c, v);
            if (j == STEPS - 1) release();
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
            const int64_t col = (int64_t)nt * NT + c;
            const uint32_t bad = REST ? not_finite(f) : 0u;
            store_block<ALIGNED>(C[p], ldc[p], row - lane, M[p], col, N[p], f, lane);
            if (REST && __any_sync(~0u, bad != 0u)) store_rounded_terms(terms[p], bad, C[p], ldc[p], row, M[p], col, N[p]);
        }
    }
};

// The same where a tile is shared by several units: partial sums in 32 bits,
// planes of M rows of ld (N rounded up to 32) for each split.  Products of the
// launch that are not shared (no planes) go straight to their C.  REST: those are
// weight gradients with remainders.
template <typename T, int NT_, int P, bool REST>
struct EpiPartial {
    static constexpr int NT = NT_, GROUPS = 2;
    float* planes[P];
    T* C[P];
    int64_t ld[P], ldc[P], M[P], N[P];
    RoundedTerms<T> terms[REST ? P : 1];
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int p, int z, int64_t row, int nt, int group, int lane, Release release) const {
        constexpr int STEPS = NT / GROUPS / 32;
#pragma unroll 1
        for (int j = 0; j < STEPS; ++j) {
            const int c = (group * STEPS + j) * 32;
            uint32_t v[32];
            tc5::ld32(acc + c, v);
            if (j == STEPS - 1) release();
            const int64_t col = (int64_t)nt * NT + c;
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
            if (planes[p] == nullptr) {
                const uint32_t bad = REST ? not_finite(f) : 0u;
                store_block<false>(C[p], ldc[p], row - lane, M[p], col, N[p], f, lane);
                if (REST && __any_sync(~0u, bad != 0u)) store_rounded_terms(terms[p], bad, C[p], ldc[p], row, M[p], col, N[p]);
            } else if (row < M[p] && col < ld[p]) {
                store_row(planes[p] + ((int64_t)z * M[p] + row) * ld[p] + col, f);
            }
        }
    }
};

// C = the sum of the splits' planes, in their order, rounded once: a thread for
// four columns of a row (the planes hold few tiles: 32-bit indices do).  halves: a
// split has two planes of M rows, of rounded values and of what that leaves.
template <typename T>
struct PartialSums {
    const float* planes;
    T* C;
    int64_t ldc;
    int M, N, ld, splits;
    bool halves;
};
template <typename T, int P>
struct AllPartialSums {
    PartialSums<T> s[P];
};
template <typename T, int P>
__global__ void __launch_bounds__(256) add_partials_kernel(const __grid_constant__ AllPartialSums<T, P> all) {
    pdl_wait();
    pdl_launch_dependents();
    const PartialSums<T>& s = all.s[blockIdx.y];
    const uint32_t i = blockIdx.x * 256 + threadIdx.x, quads = (uint32_t)s.ld / 4, n = (uint32_t)s.M * quads;
    if (i >= n) return;
    const uint32_t row = i / quads, c = (i - row * quads) * 4;
    if (c >= (uint32_t)s.N) return;
    const float4* p = reinterpret_cast<const float4*>(s.planes) + i;
    const int splits = s.splits;
    const size_t step = s.halves ? 2 * (size_t)n : n;
    float4 sum = p[0], rest = s.halves ? p[n] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int z = 1; z < splits; ++z) {
        const float4 v = p[z * step];
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        if (s.halves) {
            const float4 w = p[z * step + n];
            rest.x += w.x, rest.y += w.y, rest.z += w.z, rest.w += w.w;
        }
    }
    if (s.halves) {
        sum.x = with_rest(sum.x, rest.x), sum.y = with_rest(sum.y, rest.y);
        sum.z = with_rest(sum.z, rest.z), sum.w = with_rest(sum.w, rest.w);
    }
    T* dst = s.C + row * s.ldc + c;
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (c + j < (uint32_t)s.N) dst[j] = from_float<T>(v[j]);
}
constexpr int kMaxSplits = 16;

// h = act(g) * u from accumulators of NT / 2 columns of g and as many of u,
// rounded to 16 bits (the operand of the next product); SAVE: a = act(g),
// b = u act'(g).
template <typename T, int NT_, bool SAVE>
struct EpiGate {
    static constexpr int NT = NT_, GROUPS = 2;
    T* h;
    KeepPlanes keep;
    int64_t M, N;  // N: F rounded up to 64, a row of every plane
    int act;
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int, int, int64_t row, int nt, int group, int, Release release) const {
        constexpr int STEPS = NT / 2 / GROUPS / 32;
#pragma unroll 1
        for (int j = 0; j < STEPS; ++j) {
            const int c = (group * STEPS + j) * 32;
            uint32_t g[32], u[32];
            tc5::ld32(acc + c, g);
            tc5::ld32(acc + NT / 2 + c, u);
            if (j == STEPS - 1) release();
            const int64_t col = (int64_t)nt * (NT / 2) + c;
            if (row >= M || col >= N) continue;
            float hv[32], av[32], bv[32];
            with_activation(act, [&](auto tag) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float da = 0.0f;
                    activation<decltype(tag)::value, SAVE>(__uint_as_float(g[i]), av[i], da);
                    hv[i] = av[i] * __uint_as_float(u[i]);
                    bv[i] = __uint_as_float(u[i]) * da;
                }
            });
            const int64_t at = row * N + col;
            store_row(h + at, hv);
            if (SAVE) {
                using V = typename Keep<T>::value;
                keep_row(static_cast<V*>(keep.a), keep.ea, at, av);
                keep_row(static_cast<V*>(keep.b), keep.eb, at, bv);
            }
        }
    }
};

// dg = dh b, du = dh a, rounded to 16 bits (operands of the next products);
// REST: and what that leaves, M rows further on.
template <typename T, int NT_, bool REST>
struct EpiGateBackward {
    static constexpr int NT = NT_, GROUPS = 2;
    KeepPlanes keep;
    T *dg, *du;
    int64_t M, N;  // N: F rounded up to 64, a row of every plane
    static __device__ __forceinline__ float rest(float v) { return remainder_of(v, from_float<T>(v)); }
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int, int, int64_t row, int nt, int group, int, Release release) const {
        constexpr int STEPS = NT / GROUPS / 32;
#pragma unroll 1
        for (int j = 0; j < STEPS; ++j) {
            const int c = (group * STEPS + j) * 32;
            uint32_t v[32];
            tc5::ld32(acc + c, v);
            if (j == STEPS - 1) release();
            const int64_t col = (int64_t)nt * NT + c;
            if (row >= M || col >= N) continue;
            using V = typename Keep<T>::value;
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
                const int64_t at = row * N + col + i;
                float a[16], b[16];
                kept16(static_cast<const V*>(keep.a), keep.ea, at, a);
                kept16(static_cast<const V*>(keep.b), keep.eb, at, b);
                uint32_t pg[8], pu[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float d0 = __uint_as_float(v[i + 2 * k]), d1 = __uint_as_float(v[i + 2 * k + 1]);
                    pg[k] = pack2<T>(d0 * b[2 * k], d1 * b[2 * k + 1]);
                    pu[k] = pack2<T>(d0 * a[2 * k], d1 * a[2 * k + 1]);
                }
                store_v8(dg + at, pg);
                store_v8(du + at, pu);
                if constexpr (REST) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float d0 = __uint_as_float(v[i + 2 * k]), d1 = __uint_as_float(v[i + 2 * k + 1]);
                        pg[k] = pack2<T>(rest(d0 * b[2 * k]), rest(d1 * b[2 * k + 1]));
                        pu[k] = pack2<T>(rest(d0 * a[2 * k]), rest(d1 * a[2 * k + 1]));
                    }
                    store_v8(dg + at + M * N, pg);
                    store_v8(du + at + M * N, pu);
                }
            }
        }
    }
};

// The same two epilogues for the split kernel: one value per lane.
template <typename T, int HALVES_>
struct EpiSplitStore {
    static constexpr int UNITS = 1, HALVES = HALVES_;
    T* C;
    int64_t ldc, N;
    __device__ __forceinline__ void emit(float v, float rest, int64_t m, int unit, int lane, int tile) const {
        const int64_t n = (int64_t)tile * 128 + unit * 32 + lane;
        if (n < N) C[m * ldc + n] = from_float<T>(HALVES == 2 ? with_rest(v, rest) : v);
    }
};

template <typename T>
struct EpiSplitGate {
    static constexpr int UNITS = 2, HALVES = 1;
    T* h;
    int64_t rest;     // rows from a value to what its rounding leaves; 0: not kept
    KeepPlanes keep;  // null: no backward pass follows
    int64_t N;        // F rounded up to 64, a row of every plane
    int act;
    __device__ __forceinline__ void emit(float g, float u, int64_t m, int unit, int lane, int tile) const {
        const int64_t n = (int64_t)tile * 64 + unit * 32 + lane;
        if (n >= N) return;  // whole warps
        float av = 0.0f, da = 0.0f;
        with_activation(act, [&](auto tag) { activation<decltype(tag)::value, true>(g, av, da); });
        const T hi = from_float<T>(av * u);
        h[m * N + n] = hi;
        if (rest != 0) h[(m + rest) * N + n] = from_float<T>(remainder_of(av * u, hi));
        if (keep.a != nullptr) {
            using V = typename Keep<T>::value;
            keep_lane(static_cast<V*>(keep.a), keep.ea, m * N + n, av, lane);
            keep_lane(static_cast<V*>(keep.b), keep.eb, m * N + n, u * da, lane);
        }
    }
};

// Rows of 16-bit elements to 128-byte aligned rows, up to five matrices in one
// launch: a warp takes 256 elements of a row, 8 loads of one element a lane in
// flight (the source may be aligned to its elements only), and stores 4 bytes a
// lane.
struct RealignAll {
    Matrix16 src[kRealignMax], dst[kRealignMax];
    int64_t end[kRealignMax];  // items up to and with each matrix
    int count;
};
__global__ void __launch_bounds__(256) realign_kernel(const __grid_constant__ RealignAll a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    for (int64_t i0 = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i0 < a.end[a.count - 1]; i0 += (int64_t)gridDim.x * 8) {
        int k = 0;
        while (i0 >= a.end[k]) ++k;
        const int64_t item = i0 - (k > 0 ? a.end[k - 1] : 0);
        const int64_t cols = a.src[k].cols, parts = (cols + 255) / 256;
        const int64_t r = item / parts, c0 = item % parts * 256 + lane * 2;
        const uint16_t* p = static_cast<const uint16_t*>(a.src[k].p) + r * a.src[k].ld;
        uint16_t* d = static_cast<uint16_t*>(a.dst[k].p) + r * a.dst[k].ld;
        uint16_t v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) v[i][j] = c0 + i * 64 + j < cols ? p[c0 + i * 64 + j] : (uint16_t)0;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // rows of cols rounded up to 64: a pair begun inside one lies in it
            if (c0 + i * 64 < cols)
                *reinterpret_cast<uint32_t*>(d + c0 + i * 64) = (uint32_t)v[i][0] | (uint32_t)v[i][1] << 16;
    }
}

cudaError_t map16(CUtensorMap* m, const Matrix16& x, int box_rows) {
    const int64_t ld = x.rows > 1 ? x.ld : round_up(x.cols, 8);
    return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, x.p, x.cols, x.rows, ld * 2, 64, box_rows, true);
}

int64_t pair_tiles(int64_t M, int64_t N, int64_t per_tile) { return (M + 255) / 256 * ((N + per_tile - 1) / per_tile); }

constexpr double kNarrow16 = 0.6;  // 128 columns for 256: 722 us against 642 for the forward of 4096 x 4096 x 12288
bool narrow16(int64_t M, int64_t N, int64_t wide) {
    return narrow_tiles(pair_tiles(M, N, wide), pair_tiles(M, N, wide / 2), kNarrow16);
}

// One product of a launch: C (M x N) = sum over segments of A_s B_s^T, depth K
// each; a_mn: A is stored K x M.
struct Product16 {
    Matrix16 A[2], B[2];
    int segs;
    bool a_mn;
    int64_t M, N, K;
    void* C;
    int64_t ldc;
    bool doubled;  // rows M / 2 and on of the product are added to the first ones
    int64_t stages() const { return (K + 63) / 64 * segs; }
    // of a sum over tokens with remainders: its first segment
    template <typename T> RoundedTerms<T> rounded() const {
        return {static_cast<const T*>(A[0].p), static_cast<const T*>(B[0].p), A[0].ld, B[0].ld, (int)K};
    }
};

// Tiles of `per_tile` columns (64 or 128 of each matrix if gated) and maps of
// products; b_box: rows of a box of B.
cudaError_t tile_args(const Product16* w, int count, int64_t per_tile, int b_maps, int b_box, TileArgs& g, TileMaps& maps) {
    memset(&maps, 0, sizeof(maps));
    g = TileArgs{};
    g.products = count;
    int map = 0;
    cudaError_t err = cudaSuccess;
    for (int p = 0; p < count; ++p) {
        TileProduct& q = g.p[p];
        q.mt = (int)((w[p].M + 255) / 256);
        q.nt = (int)((w[p].N + per_tile - 1) / per_tile);
        q.nk = (int)((w[p].K + 63) / 64);
        q.segs = w[p].segs;
        q.last_steps = (int)((w[p].K - (int64_t)(q.nk - 1) * 64 + 15) / 16);
        q.a_mn = w[p].a_mn;
        q.map = map;
        for (int s = 0; s < w[p].segs && err == cudaSuccess; ++s) err = map16(&maps.a[map + s], w[p].A[s], w[p].a_mn ? 64 : 128);
        for (int s = 0; s < std::max(w[p].segs, b_maps) && err == cudaSuccess; ++s) err = map16(&maps.b[map + s], w[p].B[s], b_box);
        map += w[p].segs;
    }
    return err;
}

// One product with an epilogue of its own; A with k contiguous.
template <int KIND, bool B_MN, bool GATED, class Epi>
cudaError_t product16(const Product16& w, const Epi& epi, cudaStream_t st) {
    TileArgs g;
    TileMaps maps;
    const cudaError_t err =
        tile_args(&w, 1, GATED ? Epi::NT / 2 : Epi::NT, GATED ? 2 : 1, B_MN ? 64 : Epi::NT / 2, g, maps);
    return err != cudaSuccess ? err : launch_tile_gemm<KIND, kMajorK, B_MN, GATED>(g, maps, epi, st);
}

// x (tokens x K) times the rows of W0 (and W1, 64 rows of each to a tile).
template <int KIND, bool PAIRED, class Epi>
cudaError_t split16(const Matrix16& x, const Matrix16& W0, const Matrix16& W1, bool early, const Epi& epi,
                    cudaStream_t st) {
    constexpr int ROWS = PAIRED ? 64 : 128;
    SplitMaps maps;
    memset(&maps, 0, sizeof(maps));
    cudaError_t err = map16(&maps.p[0], W0, ROWS);
    if (err == cudaSuccess && PAIRED) err = map16(&maps.p[1], W1, ROWS);
    if (err == cudaSuccess) err = map16(&maps.q, x, split_nq(x.rows));
    if (err != cudaSuccess) return err;
    SplitArgs g = {};
    g.nt = (int)((W0.rows + ROWS - 1) / ROWS);
    g.nk = (int)((x.cols + 63) / 64);
    g.last_steps = (int)((x.cols - (int64_t)(g.nk - 1) * 64 + 15) / 16);
    g.early = early;
    g.M = (int)x.rows / Epi::HALVES;
    return launch_split_gemm<KIND, PAIRED>(g, maps, epi, st);
}

// Products into their C, with wide or narrow tiles.
template <int KIND, typename T, int A_MAJOR, bool B_MN, bool REST, int NT, bool ALIGNED>
cudaError_t store16_sized(const Product16* w, int count, cudaStream_t st) {
    TileArgs g;
    TileMaps maps;
    const cudaError_t err = tile_args(w, count, NT, 1, B_MN ? 64 : NT / 2, g, maps);
    if (err != cudaSuccess) return err;
    EpiStore<T, NT, kMaxProducts, ALIGNED, REST> epi = {};
    for (int p = 0; p < count; ++p) {
        epi.C[p] = static_cast<T*>(w[p].C);
        epi.ldc[p] = w[p].ldc;
        epi.M[p] = w[p].M;
        epi.N[p] = w[p].N;
        if (REST) epi.terms[p] = w[p].rounded<T>();
    }
    return launch_tile_gemm<KIND, A_MAJOR, B_MN, false>(g, maps, epi, st);
}

// Products whose few tiles are shared by several units of `depth` stages:
// partial sums in the library's pool, and a launch that adds them up.
template <int KIND, typename T, int A_MAJOR, bool B_MN, bool REST, int NT>
cudaError_t store16_shared(const Product16* w, int count, int64_t depth, cudaStream_t st) {
    TileArgs g;
    TileMaps maps;
    cudaError_t err = tile_args(w, count, NT, 1, B_MN ? 64 : NT / 2, g, maps);
    if (err != cudaSuccess) return err;
    AllPartialSums<T, kMaxProducts> sums = {};
    EpiPartial<T, NT, kMaxProducts, REST> epi = {};
    int64_t total = 0, most = 0;
    int shared = 0, of[kMaxProducts];
    for (int p = 0; p < count; ++p) {
        const int64_t ld = round_up(w[p].N, 32), s = (w[p].stages() + depth - 1) / depth;
        const int64_t per = (w[p].stages() + s - 1) / s;
        g.p[p].splits = (int)((w[p].stages() + per - 1) / per);  // none empty
        epi.C[p] = static_cast<T*>(w[p].C);
        epi.ldc[p] = w[p].ldc;
        epi.M[p] = w[p].M;
        epi.N[p] = w[p].N;
        epi.ld[p] = ld;
        if (REST) epi.terms[p] = w[p].rounded<T>();
        if (g.p[p].splits == 1 && !w[p].doubled) continue;
        of[shared] = p;
        sums.s[shared++] = PartialSums<T>{nullptr, epi.C[p], w[p].ldc, (int)(w[p].doubled ? w[p].M / 2 : w[p].M), (int)w[p].N, (int)ld,
                                         g.p[p].splits, w[p].doubled};
        total += w[p].M * ld * g.p[p].splits;
        most = std::max(most, w[p].M * ld / 4);
    }
    void* ws = nullptr;
    err = pool_alloc(&ws, (size_t)total * 4, st);
    if (err != cudaSuccess) return err;
    float* at = static_cast<float*>(ws);
    for (int i = 0; i < shared; ++i) {
        sums.s[i].planes = epi.planes[of[i]] = at;
        at += w[of[i]].M * epi.ld[of[i]] * sums.s[i].splits;
    }
    err = launch_tile_gemm<KIND, A_MAJOR, B_MN, false>(g, maps, epi, st);
    if (err == cudaSuccess)
        err = launch_pdl(add_partials_kernel<T, kMaxProducts>, dim3((unsigned)((most + 255) / 256), (unsigned)shared), dim3(256),
                         0, st, sums);
    const cudaError_t freed = cudaFreeAsync(ws, st);
    return err == cudaSuccess ? freed : err;
}

// How wide the tiles of a launch with few of them had best be and how deep its
// units, from dealing them out as the kernel does: a unit costs its stages (0.2
// us each, narrow ones kNarrow16 of that) and 8 more, adding partial sums up 20.
// Sharing wide tiles moves a third less through L2 than narrow ones of the same
// count (192 x 12288 -> 4096: 32 us narrow, 28 wide).
struct Share {
    int nt;         // 0: too many tiles for that to matter
    int64_t depth;  // of a unit, at most
    bool split;     // some tile is shared
};
Share best_share(const Product16* w, int count) {
    constexpr int kMaxPairs = 256;
    const int64_t pairs = std::min(kMaxPairs, std::max(1, device_sms() / 2));
    int64_t deepest = 0, tiles = 0;
    for (int p = 0; p < count; ++p) {
        deepest = std::max(deepest, w[p].stages());
        tiles += pair_tiles(w[p].M, w[p].N, 128);
    }
    Share best{0, deepest, false};
    if (count == 0 || tiles > 2 * pairs) return best;
    double best_cost = 1e30;
    for (const int nt : {128, 256}) {
        for (int64_t depth = deepest; depth >= 12; depth = depth * 3 / 4) {
            double load[kMaxPairs] = {0};
            int64_t t = 0, units = 0;
            bool fits = true;
            for (int p = 0; p < count && fits; ++p) {
                const int64_t s = (w[p].stages() + depth - 1) / depth;
                const int64_t n = pair_tiles(w[p].M, w[p].N, nt) * s;
                const double each = (double)((w[p].stages() + s - 1) / s) * (nt == 128 ? kNarrow16 : 1.0) + 8;
                units += n;
                fits = s <= kMaxSplits && units <= 4 * pairs;
                for (int64_t i = 0; i < n && fits; ++i, t = t + 1 == pairs ? 0 : t + 1) load[t] += each;
            }
            if (!fits) break;
            const double cost = *std::max_element(load, load + pairs) + (depth < deepest ? 20 : 0);
            if (cost < best_cost) {
                best_cost = cost;
                best = Share{nt, depth, depth < deepest};
            }
        }
    }
    if (best.nt == 0) best = Share{128, deepest, false};  // all shallower than 12
    return best;
}

// Products of one launch: shared if they are few and deep, else with the tiles
// whose rounds are the shorter.  REST: dx doubled, if it is among them, and weight
// gradients of a few tokens (two stages each: never shared).
template <int KIND, typename T, int A_MAJOR, bool B_MN, bool REST>
cudaError_t store16(const Product16* w, int count, const Share& share, cudaStream_t st) {
    if (count == 0) return cudaSuccess;
    int64_t wide = 0, few = 0;
    bool aligned = true;
    for (int p = 0; p < count; ++p) {
        wide += pair_tiles(w[p].M, w[p].N, 256);
        few += pair_tiles(w[p].M, w[p].N, 128);
        aligned = aligned && aligned_rows<T>(w[p].C, w[p].ldc);
    }
    if (share.split || w[0].doubled)
        return share.nt == 128 ? store16_shared<KIND, T, A_MAJOR, B_MN, REST, 128>(w, count, share.depth, st)
                               : store16_shared<KIND, T, A_MAJOR, B_MN, REST, 256>(w, count, share.depth, st);
    const bool narrow = share.nt != 0 ? share.nt == 128 : narrow_tiles(wide, few, kNarrow16);
    auto f = narrow ? (aligned ? store16_sized<KIND, T, A_MAJOR, B_MN, REST, 128, true>
                               : store16_sized<KIND, T, A_MAJOR, B_MN, REST, 128, false>)
                    : (aligned ? store16_sized<KIND, T, A_MAJOR, B_MN, REST, 256, true>
                               : store16_sized<KIND, T, A_MAJOR, B_MN, REST, 256, false>);
    return f(w, count, st);
}

template <int KIND, typename T, int NT, bool SAVE>
cudaError_t gate16(const FfForward& f, cudaStream_t st) {
    return product16<KIND, false, true>(
        Product16{{f.x}, {f.wg, f.wu}, 1, false, f.T, f.F, f.D, nullptr, 0, false},
        EpiGate<T, NT, SAVE>{static_cast<T*>(f.h), KeepPlanes{f.a, f.b, f.ea, f.eb}, f.T, f.ld, f.act}, st);
}

template <int KIND, typename T>
cudaError_t forward_typed(const FfForward& f, cudaStream_t st) {
    const int64_t rest = f.T <= kFullTokens ? f.T : 0;
    const Matrix16 h{f.h, f.T + rest, f.F, f.ld};
    cudaError_t err;
    if (f.T <= kSplitTokens16) {
        err = split16<KIND, true>(f.x, f.wg, f.wu, false,
                                  EpiSplitGate<T>{static_cast<T*>(f.h), rest, KeepPlanes{f.a, f.b, f.ea, f.eb}, f.ld, f.act}, st);
    } else {
        const bool narrow = narrow16(f.T, f.F, 128), save = f.a != nullptr;
        err = narrow ? (save ? gate16<KIND, T, 128, true>(f, st) : gate16<KIND, T, 128, false>(f, st))
                     : (save ? gate16<KIND, T, 256, true>(f, st) : gate16<KIND, T, 256, false>(f, st));
    }
    if (err != cudaSuccess) return err;
    // Wd was complete before the launch above could end its own wait
    if (rest != 0)
        return split16<KIND, false>(h, f.wd, f.wd, true, EpiSplitStore<T, 2>{static_cast<T*>(f.y), f.ldy, f.D}, st);
    if (f.T <= kSplitTokens16)
        return split16<KIND, false>(h, f.wd, f.wd, true, EpiSplitStore<T, 1>{static_cast<T*>(f.y), f.ldy, f.D}, st);
    const Product16 y{{h}, {f.wd}, 1, false, f.T, f.D, f.F, f.y, f.ldy, false};
    return store16<KIND, T, kMajorK, false, false>(&y, 1, best_share(&y, 1), st);
}

template <int KIND, typename T, int NT, bool REST>
cudaError_t gate_backward16(const FfBackward& f, cudaStream_t st) {
    return product16<KIND, true, false>(
        Product16{{f.dy}, {f.wd}, 1, false, f.T, f.F, f.D, nullptr, 0, false},
        EpiGateBackward<T, NT, REST>{KeepPlanes{const_cast<void*>(f.a), const_cast<void*>(f.b), const_cast<uint8_t*>(f.ea),
                                           const_cast<uint8_t*>(f.eb)},
                                static_cast<T*>(f.dg), static_cast<T*>(f.du), f.T, f.ld}, st);
}

template <int KIND, typename T>
cudaError_t backward_typed(const FfBackward& f, cudaStream_t st) {
    const bool full = f.T <= kFullTokens;
    const int segs = full ? 2 : 1;
    Matrix16 h[2], dg[2], du[2];  // and what their roundings leave
    for (int i = 0; i < 2; ++i) {
        const int64_t from = i * f.T * f.ld;
        h[i] = Matrix16{static_cast<T*>(const_cast<void*>(f.h)) + from, f.T, f.F, f.ld};
        dg[i] = Matrix16{static_cast<T*>(f.dg) + from, f.T, f.F, f.ld};
        du[i] = Matrix16{static_cast<T*>(f.du) + from, f.T, f.F, f.ld};
    }
    cudaError_t err = cudaSuccess;
    // dh = dy Wd (B is Wd, D x F: K x N), unless only dWd is wanted
    if (f.dx != nullptr || f.dwg != nullptr || f.dwu != nullptr)
        err = narrow16(f.T, f.F, 256)
                  ? (full ? gate_backward16<KIND, T, 128, true>(f, st) : gate_backward16<KIND, T, 128, false>(f, st))
                  : (full ? gate_backward16<KIND, T, 256, true>(f, st) : gate_backward16<KIND, T, 256, false>(f, st));
    if (err != cudaSuccess) return err;
    // dx = dg Wg + du Wu; the weights' gradients are sums over the T rows of both
    // operands.  All in one launch where the tiles are few (best_share); else dx
    // by itself (its tiles are of another depth: dealt out with the others, some
    // pairs would have one more of the deep ones).
    Product16 w[kMaxProducts];
    int count = 0;
    if (f.dx != nullptr) {
        const int64_t rows = f.T * segs;
        const Matrix16 g{f.dg, rows, f.F, f.ld}, u{f.du, rows, f.F, f.ld};
        w[count++] = Product16{{g, u}, {f.wg, f.wu}, 2, false, rows, f.D, f.F, f.dx, f.lddx, full};
    }
    const int others = count;
    if (f.dwg != nullptr) w[count++] = Product16{{dg[0], dg[1]}, {f.x, f.x}, segs, true, f.F, f.D, f.T, f.dwg, f.lddwg, false};
    if (f.dwu != nullptr) w[count++] = Product16{{du[0], du[1]}, {f.x, f.x}, segs, true, f.F, f.D, f.T, f.dwu, f.lddwu, false};
    if (f.dwd != nullptr) w[count++] = Product16{{f.dy, f.dy}, {h[0], h[1]}, segs, true, f.D, f.F, f.T, f.dwd, f.lddwd, false};
    const auto store = full ? store16<KIND, T, kMajorAny, true, true> : store16<KIND, T, kMajorAny, true, false>;
    const Share all = best_share(w, count);
    if (all.nt != 0) return store(w, count, all, st);
    err = store(w, others, best_share(w, others), st);
    if (err != cudaSuccess) return err;
    return store(w + others, count - others, best_share(w + others, count - others), st);
}

}  // namespace

cudaError_t launch_realign(const Matrix16* src, const Matrix16* dst, int count, cudaStream_t st) {
    RealignAll a = {};
    int64_t items = 0;
    for (int i = 0; i < count; ++i) {
        a.src[i] = src[i];
        a.dst[i] = dst[i];
        items += src[i].rows * ((src[i].cols + 255) / 256);
        a.end[i] = items;
    }
    a.count = count;
    if (items == 0) return cudaSuccess;
    const unsigned blocks = (unsigned)std::min<int64_t>((items + 7) / 8, 1 << 20);
    return launch_pdl(realign_kernel, dim3(blocks), dim3(256), 0, st, a);
}

cudaError_t launch_ff_forward(const FfForward& f, cudaStream_t st) {
    return f.type == DDGEMM_BF16 ? forward_typed<kKindBF16, __nv_bfloat16>(f, st)
                                 : forward_typed<kKindF16, __half>(f, st);
}

cudaError_t launch_ff_backward(const FfBackward& f, cudaStream_t st) {
    return f.type == DDGEMM_BF16 ? backward_typed<kKindBF16, __nv_bfloat16>(f, st)
                                 : backward_typed<kKindF16, __half>(f, st);
}

cudaError_t read_and_reset_wait_timeouts_ff(unsigned int* count) { return reset_tile_timeouts(count); }

}  // namespace ddg
