// rotary.cu -- rotary positions: every pair of a head's first elements turned by its
// position's angle (rotary.cuh), forward or back.
//
// Bound by HBM: each value is read once and written once.  The angles of a block's
// tokens are computed once, a thread for a pair, and shared by all its heads.
#include "launch.cuh"
#include "mx4.cuh"
#include "rotary.cuh"

namespace ddg {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // tokens of a block where there are many

// Eight elements from a 16-byte aligned address on.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    constexpr int W = sizeof(T) * 8 / 16;
    uint4 raw[W];
#pragma unroll
    for (int i = 0; i < W; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
    const T* t = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float<T>(t[i]);
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float2 t) {
    const float x = a, y = b;
    a = fmaf(x, t.x, -(y * t.y));
    b = fmaf(x, t.y, y * t.x);
}

// A unit of work is 8 elements of a head and their partners (VEC: everything in
// 16-byte pieces), or a pair, or what lies behind the turned part.  Threads:
// x units of a head, y rows (token, head).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const Rotary r, int tokens, int heads) {
    extern __shared__ float2 turns[];  // [tokens][half]
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int here = (int)min((int64_t)tokens, r.T - t0);
    const int h0 = blockIdx.y * heads, hs = min(heads, r.H - h0);
    const int thread = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    for (int i = thread; i < here * r.half; i += threads) {
        const int64_t t = t0 + i / r.half;
        const int64_t p = r.wide ? static_cast<const int64_t*>(r.positions)[t] : static_cast<const int32_t*>(r.positions)[t];
        const Turn a = times(turn_of((uint64_t)p * r.turns[i % r.half]), r.m, r.ml);
        turns[i] = make_float2(a.c, r.inverse ? -a.s : a.s);
    }
    __syncthreads();
    const int rows = here * hs;
    int t = 0, h = threadIdx.y;
    const T* x0 = static_cast<const T*>(r.x) + t0 * r.xt + h0 * r.xh;
    T* y0 = static_cast<T*>(r.y) + t0 * r.yt + h0 * r.yh;
    for (int row = threadIdx.y; row < rows; row += blockDim.y, h += blockDim.y) {
        while (h >= hs) {
            h -= hs;
            ++t;
        }
        const T* x = x0 + t * r.xt + h * r.xh;
        T* y = y0 + t * r.yt + h * r.yh;
        const float2* turn = turns + t * r.half;
        for (int u = threadIdx.x; u < r.units; u += blockDim.x) {
            if (VEC) {
                float a[8], b[8];
                if (u * 8 >= (r.interleaved ? 2 * r.half : r.half)) {
                    const int d = u * 8 + (r.interleaved ? 0 : r.half);
                    load8(x + d, a);
                    store8(y + d, a);
                } else if (r.interleaved) {
                    load8(x + u * 8, a);
#pragma unroll
                    for (int i = 0; i < 4; ++i) turn_pair(a[2 * i], a[2 * i + 1], turn[u * 4 + i]);
                    store8(y + u * 8, a);
                } else {
                    load8(x + u * 8, a);
                    load8(x + r.half + u * 8, b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], turn[u * 8 + i]);
                    store8(y + u * 8, a);
                    store8(y + r.half + u * 8, b);
                }
            } else if (u < r.half) {
                const int i = r.interleaved ? 2 * u : u, j = r.interleaved ? 2 * u + 1 : u + r.half;
                float a = to_float<T>(x[i]), b = to_float<T>(x[j]);
                turn_pair(a, b, turn[u]);
                y[i] = from_float<T>(a);
                y[j] = from_float<T>(b);
            } else {
                y[u + r.half] = x[u + r.half];
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
    // few tokens: a block for as many heads as it has rows of threads
    const int tokens = r.T >= 8 * device_sms() ? kTokens : 1;
    const int heads = r.T >= 2 * device_sms() || r.H <= uy ? r.H : uy;
    const int64_t blocks = (r.T + tokens - 1) / tokens;
    const dim3 grid((unsigned)blocks, (unsigned)((r.H + heads - 1) / heads)), block((unsigned)ux, (unsigned)uy);
    const size_t smem = (size_t)tokens * r.half * sizeof(float2);
    return vec ? launch_pdl(rotary_kernel<T, true>, grid, block, smem, st, r, tokens, heads)
               : launch_pdl(rotary_kernel<T, false>, grid, block, smem, st, r, tokens, heads);
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
