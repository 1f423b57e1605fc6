// lm_api.cu -- the C entry points of the 4-bit microscaled matrices and of the
// gated feed-forward block (declarations in ddgemm.h): argument checks,
// workspaces, launch sequences.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "launch.cuh"
#include "mx4.cuh"

using namespace ddg;

namespace {

constexpr int64_t kAlign = 256;

bool known_format(int f) { return f == DDGEMM_MXFP4 || f == DDGEMM_NVFP4; }
bool known_type(int t) { return t == DDGEMM_F32 || t == DDGEMM_BF16 || t == DDGEMM_F16; }
bool known_type16(int t) { return t == DDGEMM_BF16 || t == DDGEMM_F16; }
bool known_activation(int a) { return a >= DDGEMM_ACT_SILU && a <= DDGEMM_ACT_RELU; }
int64_t type_bytes(int t) { return t == DDGEMM_F32 ? 4 : 2; }
bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// Bytes from the first to the last element of a matrix.
int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
    return rows == 0 || cols == 0 ? 0 : ((rows - 1) * ld + cols) * elem;
}
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    if (a == nullptr || b == nullptr || na <= 0 || nb <= 0) return false;
    return (uintptr_t)a < (uintptr_t)b + (uintptr_t)nb && (uintptr_t)b < (uintptr_t)a + (uintptr_t)na;
}

ddgemm_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return DDGEMM_OK;
    (void)cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? DDGEMM_ERR_ALLOC : DDGEMM_ERR_CUDA;
}

// Sizes of a 4-bit matrix: within the limits, and its scale tiles and row
// tiles within the coordinates of tensor copies and grids.
ddgemm_status check_mx4_size(int format, int64_t rows, int64_t K) {
    if (!known_format(format) || rows < 0 || K < 0) return DDGEMM_ERR_INVALID_ARG;
    if (K > DDGEMM_MX4_MAX_K || rows > DDGEMM_MX4_MAX_ROWS) return DDGEMM_ERR_UNSUPPORTED;
    const int64_t tiles = (rows + 127) / 128 * mx4_scale_tiles(format, K);
    const int64_t items = rows * ((K + MX4_TILE_K - 1) / MX4_TILE_K) / 8;
    if (tiles >= (1LL << 31) || items >= (1LL << 31) - 1) return DDGEMM_ERR_UNSUPPORTED;
    return DDGEMM_OK;
}

ddgemm_status check_mx4(int format, const Mx4Matrix& m) {
    ddgemm_status s = check_mx4_size(format, m.rows, m.K);
    if (s != DDGEMM_OK) return s;
    if (m.rows == 0 || m.K == 0) return DDGEMM_OK;
    if (m.codes == nullptr || m.scales == nullptr || !aligned16(m.codes) || !aligned16(m.scales))
        return DDGEMM_ERR_INVALID_ARG;
    if (m.ldq % 16 != 0 || m.ldq < mx4_code_bytes(m.K)) return DDGEMM_ERR_INVALID_ARG;
    if (format == DDGEMM_NVFP4 && (m.exponents == nullptr || (uintptr_t)m.exponents % 4 != 0)) return DDGEMM_ERR_INVALID_ARG;
    return DDGEMM_OK;
}

bool overlaps_mx4(int format, const Mx4Matrix& m, const void* p, int64_t bytes) {
    return overlap(m.codes, span(m.rows, mx4_code_bytes(m.K), m.ldq, 1), p, bytes) ||
           overlap(m.scales, mx4_scale_bytes(format, m.rows, m.K), p, bytes) ||
           (format == DDGEMM_NVFP4 && overlap(m.exponents, m.rows * 4, p, bytes));
}

// One block of the library's pool, handed out in 256-byte aligned pieces and
// returned, in stream order, when the call ends.
class Workspace {
public:
    explicit Workspace(cudaStream_t st) : st_(st) {}
    ~Workspace() {
        if (base_ != nullptr) (void)cudaFreeAsync(base_, st_);
    }
    Workspace(const Workspace&) = delete;
    Workspace& operator=(const Workspace&) = delete;
    int64_t reserve(int64_t bytes) {
        const int64_t at = total_;
        total_ = round_up(total_ + bytes, kAlign);
        return at;
    }
    bool allocate() {
        if (total_ == 0) return true;
        if (pool_alloc(&base_, (size_t)total_, st_) == cudaSuccess) return true;
        (void)cudaGetLastError();
        base_ = nullptr;
        return false;
    }
    template <typename T> T* at(int64_t offset) const { return reinterpret_cast<T*>(static_cast<char*>(base_) + offset); }

private:
    cudaStream_t st_;
    void* base_ = nullptr;
    int64_t total_ = 0;
};

// A 16-bit operand as the tensor copies need it (16-byte aligned rows): itself,
// or a copy in the workspace with whole 128-byte rows.  Rows that are not a
// multiple of 128 bytes apart also make every copied row touch a line more (1009
// tokens, 2056 -> 5400 -> 2056: 65 us, with 2048 for 2056 54 us), which grows with
// the tokens; a copy costs the weights' bytes.  Forward, us, as they lie and
// copied: 2049 tokens 129 and 146, 4096 191 and 202, 6144 279 and 278, 8192 368
// and 361; 4104 -> 12296 -> 4104: 475 and 533, 806 and 829, 1208 and 1199, 1632 and
// 1559.
constexpr int64_t kRealignTokens = 6000;
struct Aligned16 {
    Matrix16 m;
    bool copy;
    int64_t offset;
    Aligned16(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t tokens, Workspace& ws)
        : m{const_cast<void*>(p), rows, cols, ld},
          copy(rows > 0 && cols > 0 &&
               (!aligned16(p) || (rows > 1 && (ld % 8 != 0 || (tokens > kRealignTokens && ld % 64 != 0))))),
          offset(copy ? ws.reserve(rows * round_up(cols, 64) * 2) : 0) {}
};

// Makes the copies that are needed, in one launch, and points to them.
cudaError_t resolve(Aligned16* const* operands, int count, const Workspace& ws, cudaStream_t st) {
    Matrix16 src[kRealignMax], dst[kRealignMax];
    int n = 0;
    for (int i = 0; i < count; ++i) {
        Aligned16& a = *operands[i];
        if (!a.copy) continue;
        src[n] = a.m;
        a.m = Matrix16{ws.at<void>(a.offset), a.m.rows, a.m.cols, round_up(a.m.cols, 64)};
        dst[n++] = a.m;
    }
    return n > 0 ? launch_realign(src, dst, n, st) : cudaSuccess;
}

ddgemm_status check_ff_size(int64_t T, int64_t D, int64_t F) {
    if (T < 0 || D < 0 || F < 0) return DDGEMM_ERR_INVALID_ARG;
    if (T > DDGEMM_FF_MAX || D > DDGEMM_FF_MAX || F > DDGEMM_FF_MAX) return DDGEMM_ERR_UNSUPPORTED;
    return DDGEMM_OK;
}

struct Span16 {
    const void* p;
    int64_t rows, cols, ld;
};
bool bad_operand(const Span16& x) {
    return x.ld < std::max<int64_t>(1, x.cols) || (x.rows > 0 && x.cols > 0 && (x.p == nullptr || (uintptr_t)x.p % 2));
}
int64_t bytes_of(const Span16& x) { return span(x.rows, x.cols, x.ld, 2); }

cudaError_t zero16(void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem, cudaStream_t st) {
    if (p == nullptr || rows == 0 || cols == 0) return cudaSuccess;
    return cudaMemset2DAsync(p, (size_t)(ld * elem), 0, (size_t)(cols * elem), (size_t)rows, st);
}

// Planes of the training form: h, a and b, exponent bytes of a and b.
struct SavedLayout {
    int64_t ld, off_a, off_b, off_ea, off_eb, total;
    SavedLayout(int type, int64_t T, int64_t F) {
        const int64_t elem = type == DDGEMM_BF16 ? 2 : 4, bytes = type == DDGEMM_BF16 ? 1 : 0;
        ld = round_up(F, 64);
        off_a = round_up(ff_rows(T) * ld * 2, kAlign);
        off_b = off_a + round_up(T * ld * elem, kAlign);
        off_ea = off_b + round_up(T * ld * elem, kAlign);
        off_eb = off_ea + round_up(T * ld / 32 * bytes, kAlign);
        total = off_eb + round_up(T * ld / 32 * bytes, kAlign);
    }
};

// Arguments packed as 64-bit words (of any alignment).
class Words {
public:
    explicit Words(const void* p) : p_(static_cast<const char*>(p)) {}
    template <typename T> T number(int i) const { return (T)word(i); }
    template <typename T> T* pointer(int i) const { return reinterpret_cast<T*>((uintptr_t)word(i)); }
    double real(int i) const {
        double v;
        memcpy(&v, p_ + 8 * i, 8);
        return v;
    }

private:
    int64_t word(int i) const {
        int64_t v;
        memcpy(&v, p_ + 8 * i, 8);
        return v;
    }
    const char* p_;
};
// formats, types and flags are small: anything else is no valid one
template <> int Words::number<int>(int i) const {
    const int64_t v = word(i);
    return v >= 0 && v < (1 << 30) ? (int)v : -1;
}

}  // namespace

extern "C" {

ddgemm_status dd_mx4_layout(int format, int64_t rows, int64_t K, int64_t* code_row_bytes, int64_t* scale_bytes) {
    const ddgemm_status s = check_mx4_size(format, rows, K);
    if (s != DDGEMM_OK) return s;
    if (code_row_bytes) *code_row_bytes = mx4_code_bytes(K);
    if (scale_bytes) *scale_bytes = mx4_scale_bytes(format, rows, K);
    return DDGEMM_OK;
}

ddgemm_status dd_mx4_quantize(int format, int type, int columns, int64_t rows, int64_t K, const void* X, int64_t ldx,
                              uint8_t* codes, int64_t ldq, uint8_t* scales, int32_t* exponents, void* stream) {
    if (!known_type(type) || (columns != 0 && columns != 1)) return DDGEMM_ERR_INVALID_ARG;
    const Mx4Matrix q{codes, ldq, scales, exponents, rows, K};
    const ddgemm_status s = check_mx4(format, q);
    if (s != DDGEMM_OK) return s;
    const int64_t xr = columns ? K : rows, xc = columns ? rows : K;
    if (ldx < std::max<int64_t>(1, xc)) return DDGEMM_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) return DDGEMM_OK;
    if (K == 0)
        return format == DDGEMM_NVFP4 && exponents ? status_of(cudaMemsetAsync(exponents, 0, (size_t)rows * 4, st))
                                                   : DDGEMM_OK;
    if (X == nullptr || (uintptr_t)X % type_bytes(type) != 0) return DDGEMM_ERR_INVALID_ARG;
    if (overlaps_mx4(format, q, X, span(xr, xc, ldx, type_bytes(type)))) return DDGEMM_ERR_INVALID_ARG;
    Workspace ws(st);
    const bool maxima = columns && format == DDGEMM_NVFP4;
    if (maxima) ws.reserve(rows * mx4_scale_tiles(format, K) / 4 * 17 * 4);
    if (!ws.allocate()) return DDGEMM_ERR_ALLOC;
    return status_of(launch_mx4_quantize(Mx4Quantize{format, type, columns == 1, rows, K, X, ldx, codes, ldq, scales,
                                                     exponents, maxima ? ws.at<float>(0) : nullptr},
                                         st));
}

ddgemm_status dd_mx4_dequantize(int format, int type, int64_t rows, int64_t K, const uint8_t* codes, int64_t ldq,
                                const uint8_t* scales, const int32_t* exponents, void* X, int64_t ldx, void* stream) {
    if (!known_type(type)) return DDGEMM_ERR_INVALID_ARG;
    const Mx4Matrix q{codes, ldq, scales, exponents, rows, K};
    const ddgemm_status s = check_mx4(format, q);
    if (s != DDGEMM_OK) return s;
    if (ldx < std::max<int64_t>(1, K)) return DDGEMM_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return DDGEMM_OK;
    if (X == nullptr || (uintptr_t)X % type_bytes(type) != 0) return DDGEMM_ERR_INVALID_ARG;
    if (overlaps_mx4(format, q, X, span(rows, K, ldx, type_bytes(type)))) return DDGEMM_ERR_INVALID_ARG;
    return status_of(launch_mx4_dequantize(format, type, rows, K, codes, ldq, scales, exponents, X, ldx,
                                           static_cast<cudaStream_t>(stream)));
}

ddgemm_status dd_mx4_gemm(int format, int64_t M, int64_t N, int64_t K, const uint8_t* A_codes, int64_t lda,
                          const uint8_t* A_scales, const int32_t* A_exponents, const uint8_t* B_codes, int64_t ldb,
                          const uint8_t* B_scales, const int32_t* B_exponents, float alpha, int type, void* C,
                          int64_t ldc, void* stream) {
    if (!known_type(type)) return DDGEMM_ERR_INVALID_ARG;
    const Mx4Matrix A{A_codes, lda, A_scales, A_exponents, M, K}, B{B_codes, ldb, B_scales, B_exponents, N, K};
    ddgemm_status s = check_mx4_size(format, M, K);
    if (s == DDGEMM_OK) s = check_mx4_size(format, N, K);
    if (s != DDGEMM_OK) return s;
    if (ldc < std::max<int64_t>(1, N)) return DDGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return DDGEMM_OK;  // nothing to write: no pointer is read
    s = check_mx4(format, A);
    if (s == DDGEMM_OK) s = check_mx4(format, B);
    if (s != DDGEMM_OK) return s;
    const int64_t es = type_bytes(type), cb = span(M, N, ldc, es);
    if (C == nullptr || (uintptr_t)C % es != 0) return DDGEMM_ERR_INVALID_ARG;
    if (overlaps_mx4(format, A, C, cb) || overlaps_mx4(format, B, C, cb)) return DDGEMM_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) return status_of(zero16(C, M, N, ldc, es, st));
    return status_of(launch_mx4_gemm(Mx4Gemm{format, type, A, B, alpha, C, ldc, false}, st));
}

ddgemm_status dd_ff_gated_saved_size(int type, int64_t T, int64_t F, size_t* bytes) {
    if (bytes == nullptr || !known_type16(type)) return DDGEMM_ERR_INVALID_ARG;
    const ddgemm_status s = check_ff_size(T, 0, F);
    if (s != DDGEMM_OK) return s;
    *bytes = (size_t)SavedLayout(type, T, F).total;
    return DDGEMM_OK;
}

ddgemm_status dd_ff_gated(int type, int activation, int64_t T, int64_t D, int64_t F, const void* x, int64_t ldx,
                          const void* Wg, int64_t ldwg, const void* Wu, int64_t ldwu, const void* Wd, int64_t ldwd,
                          void* y, int64_t ldy, void* saved, size_t saved_bytes, void* stream) {
    if (!known_type16(type) || !known_activation(activation)) return DDGEMM_ERR_INVALID_ARG;
    ddgemm_status s = check_ff_size(T, D, F);
    if (s != DDGEMM_OK) return s;
    const Span16 in[4] = {{x, T, D, ldx}, {Wg, F, D, ldwg}, {Wu, F, D, ldwu}, {Wd, D, F, ldwd}};
    const Span16 out{y, T, D, ldy};
    if (ldy < std::max<int64_t>(1, D)) return DDGEMM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return DDGEMM_OK;
    if (bad_operand(out)) return DDGEMM_ERR_INVALID_ARG;
    const SavedLayout L(type, T, F);
    if (saved != nullptr && ((uintptr_t)saved % kAlign != 0 || saved_bytes < (size_t)L.total))
        return DDGEMM_ERR_INVALID_ARG;
    for (const Span16& m : in) {
        if (bad_operand(m)) return DDGEMM_ERR_INVALID_ARG;
        if (overlap(m.p, bytes_of(m), y, bytes_of(out)) || (saved && overlap(m.p, bytes_of(m), saved, L.total)))
            return DDGEMM_ERR_INVALID_ARG;
    }
    if (saved != nullptr && overlap(saved, L.total, y, bytes_of(out))) return DDGEMM_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (F == 0) return status_of(zero16(y, T, D, ldy, 2, st));
    Workspace ws(st);
    Aligned16 ax(x, T, D, ldx, T, ws), ag(Wg, F, D, ldwg, T, ws), au(Wu, F, D, ldwu, T, ws), ad(Wd, D, F, ldwd, T, ws);
    const int64_t h = saved ? 0 : ws.reserve(ff_rows(T) * L.ld * 2);
    if (!ws.allocate()) return DDGEMM_ERR_ALLOC;
    Aligned16* const operands[] = {&ax, &ag, &au, &ad};
    cudaError_t err = resolve(operands, 4, ws, st);
    if (err != cudaSuccess) return status_of(err);
    char* sv = static_cast<char*>(saved);
    FfForward f{type, activation, T, D, F, ax.m, ag.m, au.m, ad.m, saved ? saved : ws.at<void>(h),
                saved ? sv + L.off_a : nullptr, saved ? sv + L.off_b : nullptr,
                saved ? reinterpret_cast<uint8_t*>(sv + L.off_ea) : nullptr,
                saved ? reinterpret_cast<uint8_t*>(sv + L.off_eb) : nullptr, L.ld, y, ldy};
    return status_of(launch_ff_forward(f, st));
}

ddgemm_status dd_ff_gated_backward(int type, int64_t T, int64_t D, int64_t F, const void* dy, int64_t lddy,
                                   const void* x, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu,
                                   int64_t ldwu, const void* Wd, int64_t ldwd, const void* saved, size_t saved_bytes,
                                   void* dx, int64_t lddx, void* dWg, int64_t lddwg, void* dWu, int64_t lddwu,
                                   void* dWd, int64_t lddwd, void* stream) {
    if (!known_type16(type)) return DDGEMM_ERR_INVALID_ARG;
    ddgemm_status s = check_ff_size(T, D, F);
    if (s != DDGEMM_OK) return s;
    const Span16 in[5] = {{dy, T, D, lddy}, {x, T, D, ldx}, {Wg, F, D, ldwg}, {Wu, F, D, ldwu}, {Wd, D, F, ldwd}};
    const Span16 out[4] = {{dx, T, D, lddx}, {dWg, F, D, lddwg}, {dWu, F, D, lddwu}, {dWd, D, F, lddwd}};
    const SavedLayout L(type, T, F);
    for (const Span16& m : in)
        if (bad_operand(m)) return DDGEMM_ERR_INVALID_ARG;
    if (T > 0 && F > 0 && D > 0 &&
        (saved == nullptr || (uintptr_t)saved % kAlign != 0 || saved_bytes < (size_t)L.total))
        return DDGEMM_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i) {
        const Span16& o = out[i];
        if (o.p == nullptr) continue;
        if (bad_operand(o)) return DDGEMM_ERR_INVALID_ARG;
        for (const Span16& m : in)
            if (overlap(m.p, bytes_of(m), o.p, bytes_of(o))) return DDGEMM_ERR_INVALID_ARG;
        if (overlap(saved, L.total, o.p, bytes_of(o))) return DDGEMM_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[j].p, bytes_of(out[j]), o.p, bytes_of(o))) return DDGEMM_ERR_INVALID_ARG;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0 || D == 0 || F == 0) {  // empty sums
        cudaError_t err = cudaSuccess;
        for (const Span16& o : out)
            if (err == cudaSuccess) err = zero16(const_cast<void*>(o.p), o.rows, o.cols, o.ld, 2, st);
        return status_of(err);
    }
    Workspace ws(st);
    Aligned16 ay(dy, T, D, lddy, T, ws), ax(x, T, D, ldx, T, ws), ag(Wg, F, D, ldwg, T, ws), au(Wu, F, D, ldwu, T, ws),
        ad(Wd, D, F, ldwd, T, ws);
    const int64_t og = ws.reserve(ff_rows(T) * L.ld * 2), ou = ws.reserve(ff_rows(T) * L.ld * 2);
    if (!ws.allocate()) return DDGEMM_ERR_ALLOC;
    Aligned16* const operands[] = {&ay, &ax, &ag, &au, &ad};
    cudaError_t err = resolve(operands, 5, ws, st);
    if (err != cudaSuccess) return status_of(err);
    const char* sv = static_cast<const char*>(saved);
    FfBackward f{type, T, D, F, ay.m, ax.m, ag.m, au.m, ad.m, saved,
                 sv + L.off_a, sv + L.off_b, reinterpret_cast<const uint8_t*>(sv + L.off_ea),
                 reinterpret_cast<const uint8_t*>(sv + L.off_eb), ws.at<void>(og), ws.at<void>(ou), L.ld, dx, lddx, dWg, lddwg, dWu, lddwu, dWd, lddwd};
    return status_of(launch_ff_backward(f, st));
}

ddgemm_status dd_mx4_ff_gated(int format, int type, int activation, int64_t T, int64_t D, int64_t F, const void* x,
                              int64_t ldx, const uint8_t* in_codes, int64_t ld_in, const uint8_t* in_scales,
                              const int32_t* in_exponents, const uint8_t* out_codes, int64_t ld_out,
                              const uint8_t* out_scales, const int32_t* out_exponents, void* y, int64_t ldy,
                              void* stream) {
    if (!known_format(format) || !known_type(type) || !known_activation(activation)) return DDGEMM_ERR_INVALID_ARG;
    ddgemm_status s = check_ff_size(T, D, F);
    if (s != DDGEMM_OK) return s;
    const int64_t F32 = round_up(F, 32), es = type_bytes(type);
    const Mx4Matrix W1{in_codes, ld_in, in_scales, in_exponents, 2 * F32, D};
    const Mx4Matrix W2{out_codes, ld_out, out_scales, out_exponents, D, F};
    s = check_mx4(format, W1);
    if (s == DDGEMM_OK) s = check_mx4(format, W2);
    if (s == DDGEMM_OK) s = check_mx4_size(format, T, D);
    if (s == DDGEMM_OK) s = check_mx4_size(format, T, F);
    if (s != DDGEMM_OK) return s;
    if (ldx < std::max<int64_t>(1, D) || ldy < std::max<int64_t>(1, D)) return DDGEMM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return DDGEMM_OK;
    const int64_t xb = span(T, D, ldx, es), yb = span(T, D, ldy, es);
    if (x == nullptr || y == nullptr || (uintptr_t)x % es != 0 || (uintptr_t)y % es != 0) return DDGEMM_ERR_INVALID_ARG;
    if (overlap(x, xb, y, yb) || overlaps_mx4(format, W1, y, yb) || overlaps_mx4(format, W2, y, yb))
        return DDGEMM_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (F == 0) return status_of(zero16(y, T, D, ldy, es, st));
    const bool nv = format == DDGEMM_NVFP4;
    Workspace ws(st);
    const int64_t xl = round_up(mx4_code_bytes(D), 128), hl = round_up(mx4_code_bytes(F), 128);
    const int64_t xc = ws.reserve(T * xl), xs = ws.reserve(mx4_scale_bytes(format, T, D)), xe = ws.reserve(T * 4);
    const int64_t hc = ws.reserve(T * hl), hs = ws.reserve(mx4_scale_bytes(format, T, F)), he = ws.reserve(T * 4);
    const int64_t hm = nv ? ws.reserve(T * mx4_scale_tiles(format, F) * 4 * 4) : 0;
    if (!ws.allocate()) return DDGEMM_ERR_ALLOC;
    const Mx4Matrix xq{ws.at<uint8_t>(xc), xl, ws.at<uint8_t>(xs), ws.at<int32_t>(xe), T, D};
    const Mx4Matrix hq{ws.at<uint8_t>(hc), hl, ws.at<uint8_t>(hs), ws.at<int32_t>(he), T, F};
    float* most = nv ? ws.at<float>(hm) : nullptr;
    cudaError_t err = launch_mx4_quantize(Mx4Quantize{format, type, false, T, D, x, ldx, ws.at<uint8_t>(xc), xl,
                                                      ws.at<uint8_t>(xs), ws.at<int32_t>(xe), nullptr},
                                          st);
    if (err == cudaSuccess) err = launch_mx4_gate(Mx4Gate{format, activation, xq, W1, hq, most, F}, st);
    if (err == cudaSuccess && nv)
        err = launch_nvfp4_finish(most, T, F, ws.at<uint8_t>(hc), hl, ws.at<uint8_t>(hs), ws.at<int32_t>(he), st);
    if (err == cudaSuccess) err = launch_mx4_gemm(Mx4Gemm{format, type, hq, W2, 1.0f, y, ldy, true}, st);
    return status_of(err);
}

ddgemm_status dd_call_packed(int call, const void* words) {
    if (words == nullptr) return DDGEMM_ERR_INVALID_ARG;
    const Words w(words);
    switch (call) {
        case DDGEMM_CALL_MX4_QUANTIZE:
            return dd_mx4_quantize(w.number<int>(0), w.number<int>(1), w.number<int>(2), w.number<int64_t>(3),
                                   w.number<int64_t>(4), w.pointer<const void>(5), w.number<int64_t>(6),
                                   w.pointer<uint8_t>(7), w.number<int64_t>(8), w.pointer<uint8_t>(9),
                                   w.pointer<int32_t>(10), w.pointer<void>(11));
        case DDGEMM_CALL_MX4_DEQUANTIZE:
            return dd_mx4_dequantize(w.number<int>(0), w.number<int>(1), w.number<int64_t>(2),
                                     w.number<int64_t>(3), w.pointer<const uint8_t>(4), w.number<int64_t>(5),
                                     w.pointer<const uint8_t>(6), w.pointer<const int32_t>(7), w.pointer<void>(8),
                                     w.number<int64_t>(9), w.pointer<void>(10));
        case DDGEMM_CALL_MX4_GEMM:
            return dd_mx4_gemm(w.number<int>(0), w.number<int64_t>(1), w.number<int64_t>(2), w.number<int64_t>(3),
                               w.pointer<const uint8_t>(4), w.number<int64_t>(5), w.pointer<const uint8_t>(6),
                               w.pointer<const int32_t>(7), w.pointer<const uint8_t>(8), w.number<int64_t>(9),
                               w.pointer<const uint8_t>(10), w.pointer<const int32_t>(11), (float)w.real(12),
                               w.number<int>(13), w.pointer<void>(14), w.number<int64_t>(15), w.pointer<void>(16));
        case DDGEMM_CALL_MX4_FF_GATED:
            return dd_mx4_ff_gated(w.number<int>(0), w.number<int>(1), w.number<int>(2), w.number<int64_t>(3),
                                   w.number<int64_t>(4), w.number<int64_t>(5), w.pointer<const void>(6),
                                   w.number<int64_t>(7), w.pointer<const uint8_t>(8), w.number<int64_t>(9),
                                   w.pointer<const uint8_t>(10), w.pointer<const int32_t>(11),
                                   w.pointer<const uint8_t>(12), w.number<int64_t>(13),
                                   w.pointer<const uint8_t>(14), w.pointer<const int32_t>(15), w.pointer<void>(16),
                                   w.number<int64_t>(17), w.pointer<void>(18));
        case DDGEMM_CALL_FF_GATED:
            return dd_ff_gated(w.number<int>(0), w.number<int>(1), w.number<int64_t>(2), w.number<int64_t>(3),
                               w.number<int64_t>(4), w.pointer<const void>(5), w.number<int64_t>(6),
                               w.pointer<const void>(7), w.number<int64_t>(8), w.pointer<const void>(9),
                               w.number<int64_t>(10), w.pointer<const void>(11), w.number<int64_t>(12),
                               w.pointer<void>(13), w.number<int64_t>(14), w.pointer<void>(15),
                               w.number<size_t>(16), w.pointer<void>(17));
        case DDGEMM_CALL_FF_GATED_BACKWARD:
            return dd_ff_gated_backward(w.number<int>(0), w.number<int64_t>(1), w.number<int64_t>(2),
                                        w.number<int64_t>(3), w.pointer<const void>(4), w.number<int64_t>(5),
                                        w.pointer<const void>(6), w.number<int64_t>(7), w.pointer<const void>(8),
                                        w.number<int64_t>(9), w.pointer<const void>(10), w.number<int64_t>(11),
                                        w.pointer<const void>(12), w.number<int64_t>(13),
                                        w.pointer<const void>(14), w.number<size_t>(15), w.pointer<void>(16),
                                        w.number<int64_t>(17), w.pointer<void>(18), w.number<int64_t>(19),
                                        w.pointer<void>(20), w.number<int64_t>(21), w.pointer<void>(22),
                                        w.number<int64_t>(23), w.pointer<void>(24));
        default: return DDGEMM_ERR_INVALID_ARG;
    }
}

}  // extern "C"
