// rotary.cu -- rotary positions: every pair of a head's first elements turned by its
// position's angle (rotary.cuh), forward or back.
//
// Bound by HBM: each value is read once and written once.  The angles of a block's
// tokens are computed once, a thread for a pair, and shared by all its heads: one for
// each head would be more arithmetic than the turning itself.  8192 x 40 x 128 bfloat16,
// there (from rows of 48 heads) and back: 61 us, 5.5 TB/s, 0.82 of a copy; 2.2 us of one
// token.  Where a half is not whole pieces of 16 bytes, a thread turns single pairs: 1009
// x 25 x 80 in 32 bits, 20 elements turned, 10 us each way for 16 MB, by its latency.
#include "eight.cuh"
#include "launch.cuh"
#include "rotary.cuh"

namespace ddg {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // tokens of a block where there are many

__device__ __forceinline__ void turn_pair(float& a, float& b, float2 t) {
    const float x = a, y = b;
    a = fmaf(x, t.x, -(y * t.y));
    b = fmaf(x, t.y, y * t.x);
}

// A unit of work is 8 elements of a head and their partners (kHalf, kInterleaved: all in
// 16-byte pieces), or a pair (kSingle), or what lies behind the turned part.  Threads: x
// units of a head, y heads.
enum Mode { kSingle, kHalf, kInterleaved };
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const Rotary r, int tokens, int heads) {
    constexpr int PER = MODE == kSingle ? 1 : MODE == kHalf ? 8 : 4;  // pairs of a unit
    constexpr int ROWS = MODE == kHalf ? 2 : 4;                       // heads whose loads a thread has in flight
    // [tokens][half], pair u PER + i of a token at i half / PER + u: neighbouring threads read neighbouring words (as
    // they lie a warp's reads would meet in a few banks, half of the time of 8192 x 40 x 128)
    extern __shared__ float2 turns[];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int here = (int)min((int64_t)tokens, r.T - t0);
    const int h0 = blockIdx.y * heads, hs = min(heads, r.H - h0), stride = r.half / PER;
    const int thread = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    for (int i = thread; i < here * r.half; i += threads) {
        const int k = i / r.half, pair = i - k * r.half;
        const int64_t t = t0 + k;
        const int64_t p = r.wide ? static_cast<const int64_t*>(r.positions)[t] : static_cast<const int32_t*>(r.positions)[t];
        const Turn a = times(turn_of((uint64_t)p * r.turns[pair]), r.m, r.ml);
        turns[k * r.half + pair % PER * stride + pair / PER] = make_float2(a.c, r.inverse ? -a.s : a.s);
    }
    __syncthreads();
    const T* x0 = static_cast<const T*>(r.x) + t0 * r.xt + (int64_t)h0 * r.xh;
    T* y0 = static_cast<T*>(r.y) + t0 * r.yt + (int64_t)h0 * r.yh;
    if constexpr (MODE != kSingle) {
        const int64_t xs = (int64_t)blockDim.y * r.xh, ys = (int64_t)blockDim.y * r.yh;
        for (int u = threadIdx.x; u < r.units; u += blockDim.x) {
            const bool copied = u * 8 >= (MODE == kHalf ? r.half : 2 * r.half);
            const int d = u * 8 + (copied && MODE == kHalf ? r.half : 0);
            const T* xt = x0 + threadIdx.y * r.xh + d;
            T* yt = y0 + threadIdx.y * r.yh + d;
            for (int t = 0; t < here; ++t, xt += r.xt, yt += r.yt) {
                float2 turn[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) turn[i] = copied ? make_float2(1.0f, 0.0f) : turns[t * r.half + u + i * stride];
                const T* x = xt;
                T* y = yt;
                for (int h = threadIdx.y; h < hs; h += ROWS * blockDim.y, x += ROWS * xs, y += ROWS * ys) {
                    Eight<T> a[ROWS], b[MODE == kHalf ? ROWS : 1];
#pragma unroll
                    for (int k = 0; k < ROWS; ++k) {
                        if (h + k * (int)blockDim.y >= hs) break;
                        load8(x + k * xs, a[k]);
                        if (MODE == kHalf && !copied) load8(x + k * xs + r.half, b[k]);
                    }
#pragma unroll
                    for (int k = 0; k < ROWS; ++k) {
                        if (h + k * (int)blockDim.y >= hs) break;
                        if (copied) {
                            float v[8];
                            unpack8(a[k], v);
                            pack8(y + k * ys, v);
                            continue;
                        }
                        float v[8], w[8];
                        unpack8(a[k], v);
                        if (MODE == kHalf) {
                            unpack8(b[k], w);
#pragma unroll
                            for (int i = 0; i < 8; ++i) turn_pair(v[i], w[i], turn[i % PER]);
                            pack8(y + k * ys + r.half, w);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) turn_pair(v[2 * i], v[2 * i + 1], turn[i % PER]);
                        }
                        pack8(y + k * ys, v);
                    }
                }
            }
        }
    } else {
        // units of all heads of all tokens, one after the other
        const int all = here * hs * r.units, step = threads / r.units, rest = threads - step * r.units;
        int row = thread / r.units, u = thread - row * r.units, t = row / hs, h = row - t * hs;
        const int dt = step / hs, dh = step - dt * hs;
        for (int i = thread; i < all; i += threads) {
            const T* x = x0 + t * r.xt + h * r.xh;
            T* y = y0 + t * r.yt + h * r.yh;
            if (u < r.half) {
                const int j = r.interleaved ? 2 * u : u, k = r.interleaved ? 2 * u + 1 : u + r.half;
                float a = to_float<T>(x[j]), b = to_float<T>(x[k]);
                turn_pair(a, b, turns[t * r.half + u]);
                y[j] = from_float<T>(a);
                y[k] = from_float<T>(b);
            } else {
                y[u + r.half] = x[u + r.half];
            }
            u += rest;
            h += dh;
            t += dt;
            if (u >= r.units) {
                u -= r.units;
                ++h;
            }
            while (h >= hs) {
                h -= hs;
                ++t;
            }
        }
    }
}

template <typename T>
cudaError_t launch(Rotary r, cudaStream_t st) {
    const int64_t per = 16 / sizeof(T);
    const auto whole = [&](const void* p, int64_t a, int64_t b) { return (uintptr_t)p % 16 == 0 && a % per == 0 && b % per == 0; };
    const bool vec = r.D % 8 == 0 && r.half % (r.interleaved ? 4 : 8) == 0 && whole(r.x, r.T > 1 ? r.xt : 0, r.H > 1 ? r.xh : 0) &&
                     whole(r.y, r.T > 1 ? r.yt : 0, r.H > 1 ? r.yh : 0);
    // in place what is not turned stays
    const int end = r.x == r.y ? 2 * r.half : r.D;
    r.units = vec ? (r.interleaved ? end : end - r.half) / 8 : end - r.half;
    const int ux = r.units < 64 ? r.units : 64, uy = kThreads / ux > 0 ? kThreads / ux : 1;
    // few tokens: a block for as many heads as it has rows of threads; many: several heads for a thread, which share
    // the token's angles
    const bool many = r.T >= 8 * device_sms();
    const int tokens = many && r.half <= 1024 ? kTokens : 1;  // 32 KB of angles at most
    const int heads = r.T >= 2 * device_sms() || r.H <= uy ? r.H : uy;
    const int most = many ? (uy + 1) / 2 : uy, rounds = (heads + most - 1) / most, rows = (heads + rounds - 1) / rounds;
    const int64_t blocks = (r.T + tokens - 1) / tokens;
    const dim3 grid((unsigned)blocks, (unsigned)((r.H + heads - 1) / heads)), block(vec ? (unsigned)ux : kThreads, vec ? (unsigned)rows : 1);
    const size_t smem = (size_t)tokens * r.half * sizeof(float2);
    return !vec ? launch_pdl(rotary_kernel<T, kSingle>, grid, block, smem, st, r, tokens, heads)
                : r.interleaved ? launch_pdl(rotary_kernel<T, kInterleaved>, grid, block, smem, st, r, tokens, heads)
                                : launch_pdl(rotary_kernel<T, kHalf>, grid, block, smem, st, r, tokens, heads);
}

}  // namespace

cudaError_t launch_rotary(const Rotary& r, cudaStream_t st) {
    if (r.T == 0 || r.H == 0) return cudaSuccess;
    if (r.x == r.y && r.half == 0) return cudaSuccess;
    switch (r.type) {
        case DDGEMM_F32: return launch<float>(r, st);
        case DDGEMM_BF16: return launch<__nv_bfloat16>(r, st);
        default: return launch<__half>(r, st);
    }
}

}  // namespace ddg
