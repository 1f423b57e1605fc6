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

// C = accumulators, rounded once; of one product, or of each of three.
template <typename T, int NT_, int P, bool ALIGNED>
struct EpiStore {
    static constexpr int NT = NT_, GROUPS = 2;
    T* C[P];
    int64_t ldc[P], M[P], N[P];
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int p, int64_t row, int nt, int group, int lane, Release release) const {
        if (P == 1) p = 0;
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
            store_block<ALIGNED>(C[p], ldc[p], row - lane, M[p], (int64_t)nt * NT + c, N[p], f, lane);
        }
    }
};

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
    __device__ __forceinline__ void run(uint32_t acc, int, int64_t row, int nt, int group, int, Release release) const {
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

// dg = dh b, du = dh a, rounded to 16 bits (operands of the next products).
template <typename T, int NT_>
struct EpiGateBackward {
    static constexpr int NT = NT_, GROUPS = 2;
    KeepPlanes keep;
    T *dg, *du;
    int64_t M, N;  // N: F rounded up to 64, a row of every plane
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int, int64_t row, int nt, int group, int, Release release) const {
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
            }
        }
    }
};

// The same two epilogues for the split kernel: one value per lane.
template <typename T>
struct EpiSplitStore {
    static constexpr int UNITS = 1;
    T* C;
    int64_t ldc, N;
    __device__ __forceinline__ void emit(float v, float, int64_t m, int unit, int lane, int tile) const {
        const int64_t n = (int64_t)tile * 128 + unit * 32 + lane;
        if (n < N) C[m * ldc + n] = from_float<T>(v);
    }
};

template <typename T>
struct EpiSplitGate {
    static constexpr int UNITS = 2;
    T* h;
    KeepPlanes keep;  // null: no backward pass follows
    int64_t N;        // F rounded up to 64, a row of every plane
    int act;
    __device__ __forceinline__ void emit(float g, float u, int64_t m, int unit, int lane, int tile) const {
        const int64_t n = (int64_t)tile * 64 + unit * 32 + lane;
        if (n >= N) return;  // whole warps
        float av = 0.0f, da = 0.0f;
        with_activation(act, [&](auto tag) { activation<decltype(tag)::value, true>(g, av, da); });
        h[m * N + n] = from_float<T>(av * u);
        if (keep.a != nullptr) {
            using V = typename Keep<T>::value;
            keep_lane(static_cast<V*>(keep.a), keep.ea, m * N + n, av, lane);
            keep_lane(static_cast<V*>(keep.b), keep.eb, m * N + n, u * da, lane);
        }
    }
};

// Rows of `cols` 16-bit elements to 128-byte aligned rows: a warp takes 256
// elements of a row, 8 loads of one element a lane in flight (the source may be
// aligned to its elements only), and stores 4 bytes a lane.
__global__ void __launch_bounds__(256) realign_kernel(const uint16_t* src, int64_t ld, int64_t rows, int64_t cols,
                                                      uint16_t* dst, int64_t ldd) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t parts = (cols + 255) / 256;
    for (int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); item < rows * parts; item += (int64_t)gridDim.x * 8) {
        const int64_t r = item / parts, c0 = item % parts * 256 + lane * 2;
        const uint16_t* p = src + r * ld;
        uint16_t v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) v[i][j] = c0 + i * 64 + j < cols ? p[c0 + i * 64 + j] : (uint16_t)0;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // ldd is cols rounded up to 64: a pair begun inside a row lies in it
            if (c0 + i * 64 < cols)
                *reinterpret_cast<uint32_t*>(dst + r * ldd + c0 + i * 64) = (uint32_t)v[i][0] | (uint32_t)v[i][1] << 16;
    }
}

cudaError_t map16(CUtensorMap* m, const Matrix16& x, int box_rows) {
    const int64_t ld = x.rows > 1 ? x.ld : round_up(x.cols, 8);
    return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, x.p, x.cols, x.rows, ld * 2, 64, box_rows, true);
}

// A product's depth and tiles; PER: columns of B under a tile (64 or 128 of
// each matrix if gated).
TileArgs tile_args(int64_t M, int64_t N, int64_t per_tile, int64_t K, int segs) {
    TileArgs g = {};
    g.products = 1;
    g.mt[0] = (int)((M + 255) / 256);
    g.nt[0] = (int)((N + per_tile - 1) / per_tile);
    g.nk = (int)((K + 63) / 64);
    g.segs = segs;
    g.last_steps = (int)((K - (int64_t)(g.nk - 1) * 64 + 15) / 16);
    return g;
}

int64_t pair_tiles(int64_t M, int64_t N, int64_t per_tile) { return (M + 255) / 256 * ((N + per_tile - 1) / per_tile); }

constexpr double kNarrow16 = 0.6;  // see narrow_tiles
bool narrow16(int64_t M, int64_t N, int64_t wide) {
    return narrow_tiles(pair_tiles(M, N, wide), pair_tiles(M, N, wide / 2), kNarrow16);
}

// sum over segments of A_s B_s^T; A_MN: A is K x M, B_MN: B is K x N.
template <int KIND, bool A_MN, bool B_MN, bool GATED, class Epi>
cudaError_t product16(int64_t M, int64_t N, int64_t K, int segs, const Matrix16& A0, const Matrix16& A1,
                      const Matrix16& B0, const Matrix16& B1, const Epi& epi, cudaStream_t st) {
    TileMaps maps;
    memset(&maps, 0, sizeof(maps));
    constexpr int A_BOX = A_MN ? 64 : 128, B_BOX = B_MN ? 64 : Epi::NT / 2;
    cudaError_t err = map16(&maps.a[0], A0, A_BOX);
    if (err == cudaSuccess) err = map16(&maps.b[0], B0, B_BOX);
    if (err == cudaSuccess && segs == 2) err = map16(&maps.a[1], A1, A_BOX);
    if (err == cudaSuccess && (segs == 2 || GATED)) err = map16(&maps.b[1], B1, B_BOX);
    if (err != cudaSuccess) return err;
    return launch_tile_gemm<KIND, A_MN, B_MN, GATED>(tile_args(M, N, GATED ? Epi::NT / 2 : Epi::NT, K, segs), maps, epi, st);
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
    g.M = x.rows;
    return launch_split_gemm<KIND, PAIRED>(g, maps, epi, st);
}

template <class Epi>
void set_store(Epi& epi, int p, void* C, int64_t ldc, int64_t M, int64_t N) {
    epi.C[p] = static_cast<decltype(epi.C[p] + 0)>(C);
    epi.ldc[p] = ldc;
    epi.M[p] = M;
    epi.N[p] = N;
}

// C = sum over segments, with wide or narrow tiles.
template <int KIND, typename T, bool B_MN, int NT, bool ALIGNED>
cudaError_t store16_sized(int64_t M, int64_t N, int64_t K, int segs, const Matrix16& A0, const Matrix16& A1,
                          const Matrix16& B0, const Matrix16& B1, void* C, int64_t ldc, cudaStream_t st) {
    EpiStore<T, NT, 1, ALIGNED> epi;
    set_store(epi, 0, C, ldc, M, N);
    return product16<KIND, false, B_MN, false>(M, N, K, segs, A0, A1, B0, B1, epi, st);
}
template <int KIND, typename T, bool B_MN>
cudaError_t store16(int64_t M, int64_t N, int64_t K, int segs, const Matrix16& A0, const Matrix16& A1,
                    const Matrix16& B0, const Matrix16& B1, void* C, int64_t ldc, cudaStream_t st) {
    const bool narrow = narrow16(M, N, 256), aligned = aligned_rows<T>(C, ldc);
    auto f = narrow ? (aligned ? store16_sized<KIND, T, B_MN, 128, true> : store16_sized<KIND, T, B_MN, 128, false>)
                    : (aligned ? store16_sized<KIND, T, B_MN, 256, true> : store16_sized<KIND, T, B_MN, 256, false>);
    return f(M, N, K, segs, A0, A1, B0, B1, C, ldc, st);
}

template <int KIND, typename T, int NT, bool SAVE>
cudaError_t gate16(const FfForward& f, cudaStream_t st) {
    return product16<KIND, false, false, true>(
        f.T, f.F, f.D, 1, f.x, f.x, f.wg, f.wu,
        EpiGate<T, NT, SAVE>{static_cast<T*>(f.h), KeepPlanes{f.a, f.b, f.ea, f.eb}, f.T, f.ld, f.act}, st);
}

template <int KIND, typename T>
cudaError_t forward_typed(const FfForward& f, cudaStream_t st) {
    const Matrix16 h{f.h, f.T, f.F, f.ld};
    cudaError_t err;
    if (f.T <= kSplitTokens16) {
        err = split16<KIND, true>(f.x, f.wg, f.wu, false,
                                  EpiSplitGate<T>{static_cast<T*>(f.h), KeepPlanes{f.a, f.b, f.ea, f.eb}, f.ld, f.act}, st);
    } else {
        const bool narrow = narrow16(f.T, f.F, 128), save = f.a != nullptr;
        err = narrow ? (save ? gate16<KIND, T, 128, true>(f, st) : gate16<KIND, T, 128, false>(f, st))
                     : (save ? gate16<KIND, T, 256, true>(f, st) : gate16<KIND, T, 256, false>(f, st));
    }
    if (err != cudaSuccess) return err;
    // Wd was complete before the launch above could end its own wait
    if (f.T <= kSplitTokens16)
        return split16<KIND, false>(h, f.wd, f.wd, true, EpiSplitStore<T>{static_cast<T*>(f.y), f.ldy, f.D}, st);
    return store16<KIND, T, false>(f.T, f.D, f.F, 1, h, h, f.wd, f.wd, f.y, f.ldy, st);
}

template <int KIND, typename T, int NT>
cudaError_t gate_backward16(const FfBackward& f, cudaStream_t st) {
    return product16<KIND, false, true, false>(
        f.T, f.F, f.D, 1, f.dy, f.dy, f.wd, f.wd,
        EpiGateBackward<T, NT>{KeepPlanes{const_cast<void*>(f.a), const_cast<void*>(f.b), const_cast<uint8_t*>(f.ea),
                                           const_cast<uint8_t*>(f.eb)},
                                static_cast<T*>(f.dg), static_cast<T*>(f.du), f.T, f.ld}, st);
}

// The weights' gradients that are wanted, in one launch: sums over the T rows
// of both operands.
template <int KIND, typename T, int NT, bool ALIGNED>
cudaError_t weights16(const FfBackward& f, const Matrix16& h, const Matrix16& dg, const Matrix16& du, cudaStream_t st) {
    TileMaps maps;
    memset(&maps, 0, sizeof(maps));
    EpiStore<T, NT, kMaxProducts, ALIGNED> epi = {};
    TileArgs g = tile_args(f.F, f.D, NT, f.T, 1);
    g.products = 0;
    cudaError_t err = cudaSuccess;
    auto add = [&](const Matrix16& A, const Matrix16& B, void* C, int64_t ldc) {
        if (C == nullptr || err != cudaSuccess) return;
        const int p = g.products++;
        err = map16(&maps.a[p], A, 64);
        if (err == cudaSuccess) err = map16(&maps.b[p], B, 64);
        g.mt[p] = (int)((A.cols + 255) / 256);
        g.nt[p] = (int)((B.cols + NT - 1) / NT);
        set_store(epi, p, C, ldc, A.cols, B.cols);
    };
    add(dg, f.x, f.dwg, f.lddwg);
    add(du, f.x, f.dwu, f.lddwu);
    add(f.dy, h, f.dwd, f.lddwd);
    if (err != cudaSuccess || g.products == 0) return err;
    return launch_tile_gemm<KIND, true, true, false>(g, maps, epi, st);
}

template <int KIND, typename T>
cudaError_t backward_typed(const FfBackward& f, cudaStream_t st) {
    const Matrix16 h{const_cast<void*>(f.h), f.T, f.F, f.ld}, dg{f.dg, f.T, f.F, f.ld}, du{f.du, f.T, f.F, f.ld};
    cudaError_t err = cudaSuccess;
    // dh = dy Wd (B is Wd, D x F: K x N), unless only dWd is wanted
    if (f.dx != nullptr || f.dwg != nullptr || f.dwu != nullptr)
        err = narrow16(f.T, f.F, 256) ? gate_backward16<KIND, T, 128>(f, st) : gate_backward16<KIND, T, 256>(f, st);
    // dx = dg Wg + du Wu
    if (err == cudaSuccess && f.dx != nullptr)
        err = store16<KIND, T, true>(f.T, f.D, f.F, 2, dg, du, f.wg, f.wu, f.dx, f.lddx, st);
    if (err != cudaSuccess) return err;
    const int64_t wide = 2 * pair_tiles(f.F, f.D, 256) + pair_tiles(f.D, f.F, 256);
    const int64_t narrow = 2 * pair_tiles(f.F, f.D, 128) + pair_tiles(f.D, f.F, 128);
    const bool aligned = (f.dwg == nullptr || aligned_rows<T>(f.dwg, f.lddwg)) &&
                         (f.dwu == nullptr || aligned_rows<T>(f.dwu, f.lddwu)) &&
                         (f.dwd == nullptr || aligned_rows<T>(f.dwd, f.lddwd));
    return narrow_tiles(wide, narrow, kNarrow16)
               ? (aligned ? weights16<KIND, T, 128, true>(f, h, dg, du, st) : weights16<KIND, T, 128, false>(f, h, dg, du, st))
               : (aligned ? weights16<KIND, T, 256, true>(f, h, dg, du, st) : weights16<KIND, T, 256, false>(f, h, dg, du, st));
}

}  // namespace

cudaError_t launch_realign(const Matrix16& src, const Matrix16& dst, cudaStream_t st) {
    const int64_t items = src.rows * ((src.cols + 255) / 256);
    if (items == 0) return cudaSuccess;
    const unsigned blocks = (unsigned)std::min<int64_t>((items + 7) / 8, 1 << 20);
    return launch_pdl(realign_kernel, dim3(blocks), dim3(256), 0, st, static_cast<const uint16_t*>(src.p), src.ld,
                      src.rows, src.cols, static_cast<uint16_t*>(dst.p), dst.ld);
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
