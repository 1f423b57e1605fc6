// kv_cache.cu -- the 4-bit cache: new tokens' keys and values quantised into their
// places, and rows read back.
//
// Both move their bytes once (2 to 4 bytes a value on one side, 0.54 to 0.58 on the
// other), small batches in their launch.  A lane holds 8 consecutive values of a row; a
// row is 8, 16 or 32 lanes, so that a block's largest value takes one or two exchanges
// between lanes.  Keys may be rotated on the way in: in 32 bits and what they leave
// (rotary.cuh), so that a value is rounded once, to its code.
//
// A prompt of 8192 tokens, 8 heads of 128, bfloat16, mxfp4: written with rotation 29 us,
// without 20, read back 13 (42 MB each way, 6.3 us of a copy).  Bound by instructions: 22
// million for a written batch, of which the rotation and what it leaves are 10 us; at 78
// registers three blocks share an SM.  32 single tokens, nvfp4: 3.7 us written with rotation, 2.7 read.
#include "eight.cuh"
#include "kv_cache.cuh"
#include "rotary.cuh"

namespace ddg {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 16;  // of a block

// Eight values of a row from element d on, 0 beyond `dim`.
template <typename T>
__device__ __forceinline__ void load_values(const T* row, int d, int dim, bool vec, Eight<T>& x) {
    if (vec && d + 8 <= dim) {
        load8(row + d, x);
    } else {
        T* t = reinterpret_cast<T*>(x.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = d + i < dim ? row[d + i] : from_float<T>(0.0f);
    }
}

// A thread's rows of a block's tokens, one after the other: token, keys or values (0 or
// 1) and head, `step` rows apart.
struct Rows {
    int t, row, heads, dt, dr;
    __device__ __forceinline__ Rows(int first, int step, int heads_) : heads(heads_) {
        const int of_token = 2 * heads;
        t = first / of_token;
        row = first - t * of_token;
        dt = step / of_token;
        dr = step - dt * of_token;
    }
    __device__ __forceinline__ int kv() const { return row >= heads; }
    __device__ __forceinline__ int head() const { return row >= heads ? row - heads : row; }
    __device__ __forceinline__ void next() {
        t += dt;
        row += dr;
        if (row >= 2 * heads) {
            row -= 2 * heads;
            ++t;
        }
    }
};

// The places of a block's tokens.  The starts go to shared memory where they fit: the
// search's steps wait for one another.
constexpr int kStarts = 512;
__device__ __forceinline__ void find_places(const CacheView& c, const BatchView& b, int64_t t0, int here, Place* places) {
    __shared__ int32_t starts[kStarts + 1];
    const bool fit = b.batch <= kStarts;
    if (fit) {
        for (int i = threadIdx.x; i <= b.batch; i += kThreads) starts[i] = b.starts[i];
        __syncthreads();
    }
    if ((int)threadIdx.x < here) places[threadIdx.x] = place_of(c, b, fit ? starts : b.starts, t0 + threadIdx.x);
    __syncthreads();
}

template <typename T>
struct Append {
    CacheView c;
    BatchView b;
    const T *k, *v;
    int64_t kt, kh, vt, vh;  // strides of tokens and heads
    bool vec_k, vec_v;
    const uint64_t* turns;  // null: keys are not rotated
    int half;
    float m, ml;
    bool interleaved;
};

template <typename T, int FMT, int WIDTH>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 3) append_kernel(const Append<T> a, int tokens) {
    constexpr int LANES = WIDTH / 8, BLOCK = mx4_block(FMT), SHARE = BLOCK / 8, BLOCKS = WIDTH / BLOCK;
    // [tokens][8 stride]: pair 8 i + k of a token at k stride + i, so that neighbouring lanes read neighbouring words
    extern __shared__ float4 turns[];
    const int stride = (a.half + 7) / 8;
    __shared__ Place places[kMostTokens];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int here = (int)min((int64_t)tokens, a.b.tokens - t0);
    find_places(a.c, a.b, t0, here, places);
    if (a.turns != nullptr) {
        for (int i = threadIdx.x; i < here * a.half; i += kThreads) {
            const int k = i / a.half, pair = i - k * a.half;
            const Turn t = times(turn_of((uint64_t)(int64_t)places[k].position * a.turns[pair]), a.m, a.ml);
            turns[(k * 8 + pair % 8) * stride + pair / 8] = make_float4(t.c, t.cl, t.s, t.sl);
        }
        __syncthreads();
    }
    const int lane = threadIdx.x % LANES, d = lane * 8;
    // whole warps take part in the exchanges below; a thread has its next row's values on the way
    const int rows = here * 2 * a.c.heads, whole = (int)round_up(rows, 32 / LANES);
    Rows at(threadIdx.x / LANES, kThreads / LANES, a.c.heads);
    const auto source = [&](const Rows& r) {
        return r.kv() == 0 ? a.k + (t0 + r.t) * a.kt + r.head() * a.kh : a.v + (t0 + r.t) * a.vt + r.head() * a.vh;
    };
    Eight<T> now, following{};
    if (at.t < here) load_values(source(at), d, a.c.dim, at.kv() == 0 ? a.vec_k : a.vec_v, following);
    for (int row = threadIdx.x / LANES; row < whole; row += kThreads / LANES) {
        now = following;
        const Rows r = at;
        at.next();
        if (row + kThreads / LANES < rows) load_values(source(at), d, a.c.dim, at.kv() == 0 ? a.vec_k : a.vec_v, following);
        const int t = min(r.t, here - 1), kv = r.kv(), head = r.head();
        const Place p = places[t];
        const int page = p.page;
        const bool store = row < rows && page >= 0;
        float x[8];
        unpack8(now, x);
        // lanes whose values are turned: whole rows' first lanes
        const uint32_t turning = __ballot_sync(~0u, kv == 0 && a.turns != nullptr && d < 2 * a.half);
        if (kv == 0) {
            const T* src = a.k + (t0 + t) * a.kt + head * a.kh;
            if (a.turns != nullptr && d < 2 * a.half) {
                const auto turn = [&](int pair) { return turns[(t * 8 + pair % 8) * stride + pair / 8]; };
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        if (d + i < 2 * a.half) {
                            const float4 w = turn((d + i) / 2);
                            const float u = x[i], v = x[i + 1];
                            x[i] = sum_of_products(u, w.x, w.y, -v, w.z, w.w);
                            x[i + 1] = sum_of_products(u, w.z, w.w, v, w.x, w.y);
                        }
                    }
                } else if (a.half % 8 == 0) {
                    // the partners are another lane's
                    const bool second = d >= a.half;
                    const int from = (threadIdx.x & 31) + (second ? -a.half : a.half) / 8;
                    const float4* at_pair = turns + t * 8 * stride + (second ? d - a.half : d) / 8;
                    Eight<T> partner;
#pragma unroll
                    for (int i = 0; i < (int)sizeof(T) * 2; ++i) partner.w[i] = __shfl_sync(turning, now.w[i], from);
                    float other[8];
                    unpack8(partner, other);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 w = at_pair[i * stride];
                        x[i] = sum_of_products(x[i], w.x, w.y, second ? other[i] : -other[i], w.z, w.w);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {  // (first, second) of a pair: first cos - second sin, second cos + first sin
                        const int e = d + i;
                        if (e >= 2 * a.half) break;
                        const bool second = e >= a.half;
                        const int pair = second ? e - a.half : e;
                        const float4 w = turn(pair);
                        const float other = to_float<T>(src[second ? pair : e + a.half]);
                        x[i] = sum_of_products(x[i], w.x, w.y, second ? other : -other, w.z, w.w);
                    }
                }
            }
        }
        uint32_t most = 0, finite = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = __float_as_uint(x[i]) & 0x7fffffffu;
            most = max(most, bits);
            if (FMT == kNvfp4) finite = max(finite, bits < kInfBits ? bits : 0u);
        }
#pragma unroll
        for (int s = 1; s < SHARE; s *= 2) most = max(most, __shfl_xor_sync(~0u, most, s));
        float y[8];
        uint32_t byte;
        int e;
        if (FMT == kMxfp4) {
            byte = mxfp4_scale_byte(most);
            const float inverse = mxfp4_inverse(byte);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i] * inverse;
            uint32_t top = byte == 255u ? 0u : byte;
#pragma unroll
            for (int s = SHARE; s < LANES; s *= 2) top = max(top, __shfl_xor_sync(~0u, top, s));
            e = (int)top - 127;
        } else {
#pragma unroll
            for (int s = 1; s < LANES; s *= 2) finite = max(finite, __shfl_xor_sync(~0u, finite, s));
            e = nvfp4_row_exponent(finite);
            byte = nvfp4_scale_byte(most, exp2_int(-e));
            const float step = nvfp4_step(byte, e), inverse = nvfp4_inverse(byte, step);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = quotient(x[i], step, inverse);
        }
        if (store) {
            const int64_t to = cache_row(a.c, page, kv, head, p.position & (a.c.page_size - 1));
            *reinterpret_cast<uint32_t*>(a.c.codes + to * (WIDTH / 2) + lane * 4) = e2m1_pack8(y);
            if (lane % SHARE == 0) a.c.scales[to * BLOCKS + lane / SHARE] = (uint8_t)byte;
            if (lane == 0) a.c.exponents[to] = (int8_t)(FMT == kNvfp4 && finite == 0u ? -127 : e);
        }
    }
}

template <typename T>
struct Read {
    CacheView c;
    BatchView b;
    T *k, *v;
    int64_t kt, kh, vt, vh;
    bool vec_k, vec_v;
};

template <typename T, int FMT, int WIDTH>
__global__ void __launch_bounds__(kThreads) read_kernel(const Read<T> a, int tokens) {
    constexpr int LANES = WIDTH / 8, BLOCK = mx4_block(FMT), SHARE = BLOCK / 8, BLOCKS = WIDTH / BLOCK;
    __shared__ Place places[kMostTokens];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int here = (int)min((int64_t)tokens, a.b.tokens - t0);
    find_places(a.c, a.b, t0, here, places);
    const int lane = threadIdx.x % LANES, d = lane * 8;
    const int rows = here * 2 * a.c.heads;
    Rows r(threadIdx.x / LANES, kThreads / LANES, a.c.heads);
#pragma unroll 2
    for (int row = threadIdx.x / LANES; row < rows; row += kThreads / LANES, r.next()) {
        const int t = r.t, kv = r.kv(), head = r.head();
        const Place p = places[t];
        if (p.sequence < 0 || d >= a.c.dim) continue;
        const int page = p.page;
        float y[8];
        if (page < 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(0x7fc00000u);
        } else {
            const int64_t at = cache_row(a.c, page, kv, head, p.position & (a.c.page_size - 1));
            const uint32_t byte = a.c.scales[at * BLOCKS + lane / SHARE];
            const uint32_t word = *reinterpret_cast<const uint32_t*>(a.c.codes + at * (WIDTH / 2) + lane * 4);
            e2m1_unpack8(word, y);
            if (FMT == kMxfp4) {
                const float scale = mxfp4_scale(byte);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= scale;
            } else {
                const float scale = e4m3_value(byte);
                const float2 f = exp2_factors(a.c.exponents[at]);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = y[i] * scale * f.x * f.y;
            }
        }
        T* out = kv == 0 ? a.k + (t0 + t) * a.kt + head * a.kh : a.v + (t0 + t) * a.vt + head * a.vh;
        if ((kv == 0 ? a.vec_k : a.vec_v) && d + 8 <= a.c.dim) {
            pack8(out + d, y);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (d + i < a.c.dim) out[d + i] = from_float<T>(y[i]);
        }
    }
}

// Whether rows of T start at whole 16 bytes.
template <typename T>
bool whole_rows(const void* p, int64_t tokens, int64_t per_token, int64_t heads, int64_t per_head) {
    constexpr int64_t per = 16 / sizeof(T);
    return (uintptr_t)p % 16 == 0 && (tokens <= 1 || per_token % per == 0) && (heads <= 1 || per_head % per == 0);
}

// As many tokens to a block as leave each SM several blocks: a block's start (places,
// angles) costs more than its rows.
inline int tokens_of_block(const CacheView& c, int64_t tokens) {
    int n = 1;
    while (n < kMostTokens && tokens >= 12LL * n * device_sms()) n *= 2;
    return n;
}

template <typename T, int FMT, int WIDTH>
cudaError_t append(const CacheAppend& g, cudaStream_t st) {
    Append<T> a{g.cache, g.batch, static_cast<const T*>(g.k), static_cast<const T*>(g.v), g.kt, g.kh, g.vt, g.vh,
                whole_rows<T>(g.k, g.batch.tokens, g.kt, g.cache.heads, g.kh),
                whole_rows<T>(g.v, g.batch.tokens, g.vt, g.cache.heads, g.vh), g.turns, g.half, g.m, g.ml, g.interleaved};
    const int tokens = tokens_of_block(g.cache, g.batch.tokens);
    const size_t smem = g.turns ? (size_t)tokens * round_up(g.half, 8) * sizeof(float4) : 0;
    return launch_pdl(append_kernel<T, FMT, WIDTH>, dim3((unsigned)((g.batch.tokens + tokens - 1) / tokens)), dim3(kThreads), smem, st, a, tokens);
}

template <typename T, int FMT, int WIDTH>
cudaError_t read(const CacheRead& g, cudaStream_t st) {
    Read<T> a{g.cache, g.batch, static_cast<T*>(g.k), static_cast<T*>(g.v), g.kt, g.kh, g.vt, g.vh,
              whole_rows<T>(g.k, g.batch.tokens, g.kt, g.cache.heads, g.kh),
              whole_rows<T>(g.v, g.batch.tokens, g.vt, g.cache.heads, g.vh)};
    const int tokens = tokens_of_block(g.cache, g.batch.tokens);
    return launch_pdl(read_kernel<T, FMT, WIDTH>, dim3((unsigned)((g.batch.tokens + tokens - 1) / tokens)), dim3(kThreads), 0, st, a, tokens);
}

template <typename T, int FMT, class G>
cudaError_t by_width(const G& g, cudaStream_t st) {
    if constexpr (std::is_same_v<G, CacheAppend>) {
        return g.cache.width == 64 ? append<T, FMT, 64>(g, st) : g.cache.width == 128 ? append<T, FMT, 128>(g, st) : append<T, FMT, 256>(g, st);
    } else {
        return g.cache.width == 64 ? read<T, FMT, 64>(g, st) : g.cache.width == 128 ? read<T, FMT, 128>(g, st) : read<T, FMT, 256>(g, st);
    }
}

template <class G>
cudaError_t by_type(const G& g, cudaStream_t st) {
    if (g.batch.tokens == 0 || g.cache.heads == 0) return cudaSuccess;
    const bool mx = g.cache.fmt == kMxfp4;
    switch (g.type) {
        case DDGEMM_F32: return mx ? by_width<float, kMxfp4>(g, st) : by_width<float, kNvfp4>(g, st);
        case DDGEMM_BF16: return mx ? by_width<__nv_bfloat16, kMxfp4>(g, st) : by_width<__nv_bfloat16, kNvfp4>(g, st);
        default: return mx ? by_width<__half, kMxfp4>(g, st) : by_width<__half, kNvfp4>(g, st);
    }
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppend& g, cudaStream_t st) { return by_type(g, st); }
cudaError_t launch_cache_read(const CacheRead& g, cudaStream_t st) { return by_type(g, st); }

}  // namespace ddg
