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
    __device__ __forceinline__ void run(uint32_t acc, int p, int, int64_t row, int nt, int group, int lane, Release release) const {
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

// The same where a tile is shared by several units: partial sums in 32 bits,
// planes of M rows of ld (N rounded up to 32) for each split.
template <int NT_, int P>
struct EpiPartial {
    static constexpr int NT = NT_, GROUPS = 2;
    float* planes[P];
    int64_t ld[P], M[P];
    template <class Release>
    __device__ __forceinline__ void run(uint32_t acc, int p, int z, int64_t row, int nt, int group, int, Release release) const {
        if (P == 1) p = 0;
        constexpr int STEPS = NT / GROUPS / 32;
#pragma unroll 1
        for (int j = 0; j < STEPS; ++j) {
            const int c = (group * STEPS + j) * 32;
            uint32_t v[32];
            tc5::ld32(acc + c, v);
            if (j == STEPS - 1) release();
            const int64_t col = (int64_t)nt * NT + c;
            if (row >= M[p] || col >= ld[p]) continue;
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
            store_row(planes[p] + ((int64_t)z * M[p] + row) * ld[p] + col, f);
        }
    }
};

// C = the sum of the splits' planes, in their order, rounded once.
template <typename T, int P>
struct PartialSums {
    const float* planes[P];
    T* C[P];
    int64_t ld[P], ldc[P], M[P], N[P];
    int splits;
};
template <typename T, int P>
__global__ void __launch_bounds__(256) add_partials_kernel(const __grid_constant__ PartialSums<T, P> s) {
    pdl_wait();
    pdl_launch_dependents();
    const int p = P == 1 ? 0 : blockIdx.z;
    const int64_t n = s.M[p] * s.ld[p];
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / s.ld[p], c = i - row * s.ld[p];
        if (c >= s.N[p]) continue;
        float v[16];
#pragma unroll
        for (int z = 0; z < 16; ++z) v[z] = z < s.splits ? s.planes[p][z * n + i] : 0.0f;
        float sum = v[0];
#pragma unroll
        for (int z = 1; z < 16; ++z)
            if (z < s.splits) sum += v[z];
        s.C[p][row * s.ldc[p] + c] = from_float<T>(sum);
    }
}

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

// dg = dh b, du = dh a, rounded to 16 bits (operands of the next products).
template <typename T, int NT_>
struct EpiGateBackward {
    static constexpr int NT = NT_, GROUPS = 2;
    KeepPlanes keep;
    T *dg, *du;
    int64_t M, N;  // N: F rounded up to 64, a row of every plane
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

constexpr double kNarrow16 = 0.6;  // 128 columns for 256: 783 us against 683 for the forward of 4096 x 4096 x 12288
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

// Products whose few tiles are shared by several units: the partial sums in the
// library's pool, and the launch that adds them up.
template <typename T, int P>
class Partials {
public:
    void add(void* C, int64_t ldc, int64_t M, int64_t N) {
        const int p = count_++;
        sums_.C[p] = static_cast<T*>(C);
        sums_.ldc[p] = ldc;
        sums_.M[p] = M;
        sums_.N[p] = N;
        sums_.ld[p] = round_up(N, 32);
        total_ += M * sums_.ld[p];
        most_ = std::max(most_, M * sums_.ld[p]);
    }
    template <int KIND, bool A_MN, bool B_MN>
    cudaError_t run(TileArgs g, int splits, const TileMaps& maps, cudaStream_t st) {
        void* ws = nullptr;
        cudaError_t err = pool_alloc(&ws, (size_t)(total_ * splits * 4), st);
        if (err != cudaSuccess) return err;
        EpiPartial<128, P> epi = {};
        float* at = static_cast<float*>(ws);
        for (int p = 0; p < count_; ++p) {
            epi.planes[p] = at;
            sums_.planes[p] = at;
            epi.ld[p] = sums_.ld[p];
            epi.M[p] = sums_.M[p];
            at += sums_.M[p] * sums_.ld[p] * splits;
        }
        g.splits = splits;
        sums_.splits = splits;
        err = launch_tile_gemm<KIND, A_MN, B_MN, false>(g, maps, epi, st);
        if (err == cudaSuccess)
            err = launch_pdl(add_partials_kernel<T, P>, dim3((unsigned)std::min<int64_t>((most_ + 255) / 256, 1 << 20), 1, (unsigned)count_),
                             dim3(256), 0, st, sums_);
        const cudaError_t freed = cudaFreeAsync(ws, st);
        return err == cudaSuccess ? freed : err;
    }

private:
    PartialSums<T, P> sums_ = {};
    int count_ = 0;
    int64_t total_ = 0, most_ = 0;
};

// C = sum over segments, with wide or narrow tiles, or narrow ones shared.
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
    const int splits = tile_splits(pair_tiles(M, N, 128), (K + 63) / 64 * segs);
    if (splits > 1) {
        Partials<T, 1> parts;
        parts.add(C, ldc, M, N);
        TileMaps maps;
        memset(&maps, 0, sizeof(maps));
        cudaError_t err = map16(&maps.a[0], A0, 128);
        if (err == cudaSuccess) err = map16(&maps.b[0], B0, 64);
        if (err == cudaSuccess && segs == 2) err = map16(&maps.a[1], A1, 128);
        if (err == cudaSuccess && segs == 2) err = map16(&maps.b[1], B1, 64);
        if (err != cudaSuccess) return err;
        return parts.template run<KIND, false, B_MN>(tile_args(M, N, 128, K, segs), splits, maps, st);
    }
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
struct WeightProduct {
    Matrix16 A, B;
    void* C;
    int64_t ldc;
};
template <int NT>
cudaError_t weight_args(const WeightProduct* w, int count, int64_t T, TileArgs& g, TileMaps& maps) {
    memset(&maps, 0, sizeof(maps));
    g = tile_args(0, 0, NT, T, 1);
    g.products = count;
    cudaError_t err = cudaSuccess;
    for (int p = 0; p < count && err == cudaSuccess; ++p) {
        err = map16(&maps.a[p], w[p].A, 64);
        if (err == cudaSuccess) err = map16(&maps.b[p], w[p].B, 64);
        g.mt[p] = (int)((w[p].A.cols + 255) / 256);
        g.nt[p] = (int)((w[p].B.cols + NT - 1) / NT);
    }
    return err;
}
template <int KIND, typename T, int NT, bool ALIGNED>
cudaError_t weights16_sized(const WeightProduct* w, int count, int64_t tokens, cudaStream_t st) {
    TileArgs g;
    TileMaps maps;
    const cudaError_t err = weight_args<NT>(w, count, tokens, g, maps);
    if (err != cudaSuccess) return err;
    EpiStore<T, NT, kMaxProducts, ALIGNED> epi = {};
    for (int p = 0; p < count; ++p) set_store(epi, p, w[p].C, w[p].ldc, w[p].A.cols, w[p].B.cols);
    return launch_tile_gemm<KIND, true, true, false>(g, maps, epi, st);
}
template <int KIND, typename T>
cudaError_t weights16(const FfBackward& f, const Matrix16& h, const Matrix16& dg, const Matrix16& du, cudaStream_t st) {
    WeightProduct w[kMaxProducts];
    int count = 0;
    if (f.dwg != nullptr) w[count++] = WeightProduct{dg, f.x, f.dwg, f.lddwg};
    if (f.dwu != nullptr) w[count++] = WeightProduct{du, f.x, f.dwu, f.lddwu};
    if (f.dwd != nullptr) w[count++] = WeightProduct{f.dy, h, f.dwd, f.lddwd};
    if (count == 0) return cudaSuccess;
    int64_t wide = 0, narrow = 0;
    bool aligned = true;
    for (int p = 0; p < count; ++p) {
        wide += pair_tiles(w[p].A.cols, w[p].B.cols, 256);
        narrow += pair_tiles(w[p].A.cols, w[p].B.cols, 128);
        aligned = aligned && aligned_rows<T>(w[p].C, w[p].ldc);
    }
    const int splits = tile_splits(narrow, (f.T + 63) / 64);
    if (splits > 1) {
        Partials<T, kMaxProducts> parts;
        for (int p = 0; p < count; ++p) parts.add(w[p].C, w[p].ldc, w[p].A.cols, w[p].B.cols);
        TileArgs g;
        TileMaps maps;
        const cudaError_t err = weight_args<128>(w, count, f.T, g, maps);
        return err != cudaSuccess ? err : parts.template run<KIND, true, true>(g, splits, maps, st);
    }
    auto run = narrow_tiles(wide, narrow, kNarrow16)
                   ? (aligned ? weights16_sized<KIND, T, 128, true> : weights16_sized<KIND, T, 128, false>)
                   : (aligned ? weights16_sized<KIND, T, 256, true> : weights16_sized<KIND, T, 256, false>);
    return run(w, count, f.T, st);
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
    return weights16<KIND, T>(f, h, dg, du, st);
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
