// split_gemm.cuh -- matrix products of few rows (tokens) with a large matrix
// (weights), for the 4-bit products and the gated block: bound by the bytes of
// the weights, so the work is split over k as well until it covers the SMs.
//
// One CTA multiplies 128 rows of the weights (the M side of the MMA, so that
// no tensor-core row is idle however few tokens there are) with NQ tokens over
// its share of k; a cluster of CTAs shares one such tile, each with its own
// part of k.  The partial sums meet in shared memory: every output has an
// owner among the CTAs, all CTAs write their sums of it into the owner's memory
// (remote stores, nobody waits for a remote load), and after a cluster barrier
// the owner adds them in the CTAs' order (no atomics: results do not depend on
// timing).  Warps: 0 copies, 1 issues MMAs, 2-9 read the accumulators (four for
// every other 16 tokens); all take part in the final sums.  Two CTAs fit an SM.
//
// The wait for the launch before this one: the next stages of a CTA's weights
// are fetched into L2 ahead of it (kAhead of them: all would not stay there),
// and if the weights are EARLY (nothing that the launch before this one
// writes), the ring is filled with them ahead of it.
//
// Weights of 37.7 MB from HBM (8192 x 8192 nvfp4) with one token: 9.1 us, 4.1
// TB/s; the 16-bit block of 302 MB: 51 us, 5.9 TB/s, 0.88 of the copy rate.  A
// launch by itself has 6 us in which HBM is idle (launch, first copies, barriers,
// store); each further token costs about 0.05 us, in the epilogue.
#pragma once

#include "mx4.cuh"
#include "tile_gemm.cuh"

namespace ddg {
namespace {

constexpr int kSplitThreads = 320;
constexpr int kSplitSmem = 108 * 1024;  // of the ring: two CTAs on an SM
constexpr int kMaxCluster = 8;
constexpr int kAhead = 6;

template <int KIND, int NQ>
struct SplitShape {
    static constexpr bool F4 = kind_is_4bit(KIND);
    static constexpr int P_BYTES = 128 * 128, Q_BYTES = NQ * 128;
    static constexpr int SCALE_TILES = F4 ? (KIND == kKindMx ? 2 : 4) : 0;
    static constexpr int SCALE_BYTES = SCALE_TILES * 512;  // of each operand
    static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES + 2 * SCALE_BYTES;
    static constexpr int STAGES = kSplitSmem / STAGE_BYTES;
    static constexpr int SMEM = STAGES * STAGE_BYTES + 1024;
    static constexpr uint32_t ACC_COLS = NQ < 32 ? 32 : NQ;
    static constexpr uint32_t TMEM_COLS = !F4 ? ACC_COLS : 128;  // with two sets of 32 columns of scales
    static_assert(!F4 || NQ <= 64, "tensor memory");
    static_assert(STAGE_BYTES % 1024 == 0 && STAGES >= 2, "ring");
    static_assert(128 * NQ * 4 + kMaxCluster * kMaxCluster * 256 <= STAGES * STAGE_BYTES, "partial sums fit the ring");
};

struct SplitMaps {
    CUtensorMap p[2], q;  // weights (gated 16-bit: Wg and Wu, 64 rows each), tokens
};

struct SplitArgs {
    int nt;            // tiles of 128 weight rows
    int nk, per;       // stages along k, and of one CTA
    int last_steps;    // MMAs in the last stage
    int tiles_k;       // 4-bit kinds: scale tiles in a row of 128
    const uint8_t *sp, *sq;  // scales of the weights and of the tokens
    int splits;        // CTAs of a cluster
    int early;         // the weights may be read before the wait
    int M;             // tokens
};

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float ld_shared(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Epi: UNITS (1: a unit of work is 32 weight rows of one token, 4 units to a
// tile and token; 2: it is 32 rows of g and 32 of u, 2 units) and
// emit(v0, v1, token, unit, lane, tile): the whole warp, one row per lane.
// HALVES = 2: the tokens' matrix holds two rows for each of M tokens, all first
// ones, then all second ones; v0 and v1 are the sums of each.
template <int KIND, int NQ, bool PAIRED16, class Epi>
__global__ void __launch_bounds__(kSplitThreads, 2) split_gemm_kernel(const __grid_constant__ SplitArgs g,
                                                                   const __grid_constant__ SplitMaps maps,
                                                                   const __grid_constant__ Epi epi) {
    using S = SplitShape<KIND, NQ>;
    constexpr int STAGES = S::STAGES;
    constexpr bool F4 = S::F4;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * STAGES + 1];
    __shared__ uint32_t tmem_slot;

    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int z = (int)cluster_ctarank();
    const int nt = blockIdx.x / g.splits;
    const int k0 = z * g.per, count = min(g.per, g.nk - k0);
    const uint32_t full0 = smem_addr(&bars[0]), empty0 = smem_addr(&bars[STAGES]), done_bar = smem_addr(&bars[2 * STAGES]);

    constexpr int ROW = F4 ? 128 : 64;
    auto load_weights = [&](int i, uint32_t dst, uint32_t bar) {
        const int kb = k0 + i;
        if (PAIRED16) {
            tma_load_2d(dst, &maps.p[0], kb * ROW, nt * 64, bar);
            tma_load_2d(dst + S::P_BYTES / 2, &maps.p[1], kb * ROW, nt * 64, bar);
        } else {
            tma_load_2d(dst, &maps.p[0], kb * ROW, nt * 128, bar);
        }
        if (F4)  // tiles of scales lie one after the other along k
            bulk_load_at(dst + S::P_BYTES + S::Q_BYTES, g.sp + ((int64_t)nt * g.tiles_k + kb * S::SCALE_TILES) * 512,
                         S::SCALE_BYTES, bar);
    };
    const int ahead = g.early ? min(count, STAGES) : 0;
    if (warp == 0) {
        if (elect_one()) {
            for (int i = 0; i < STAGES; ++i) {
                mbar_init(full0 + 8 * i, 1);
                mbar_init(empty0 + 8 * i, 1);
            }
            mbar_init(done_bar, 1);
            fence_barrier_init();
            for (int i = ahead; i < min(count, ahead + kAhead); ++i) {
                const int kb = k0 + i;
                tma_prefetch_2d(&maps.p[0], kb * ROW, nt * (PAIRED16 ? 64 : 128));
                if (PAIRED16) tma_prefetch_2d(&maps.p[1], kb * ROW, nt * 64);
            }
            for (int i = 0; i < ahead; ++i) {
                mbar_expect_tx(full0 + 8 * i, S::STAGE_BYTES);
                load_weights(i, ring + i * S::STAGE_BYTES, full0 + 8 * i);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        tc5::tmem_alloc(smem_addr(&tmem_slot), S::TMEM_COLS);
        tc5::tmem_relinquish();
    }
    tc5::fence_before_sync();
    __syncthreads();
    tc5::fence_after_sync();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        pdl_wait();
        pdl_launch_dependents();
        uint32_t stage = 0, phase = 0;
        int issued = ahead;
        bool ok = true;
        for (int i = 0; i < count; ++i) {
            ok = warp_wait(empty0 + 8 * stage, phase ^ 1, kTileWaitNs);
            if (!ok) break;
            if (elect_one()) {
                const uint32_t dst = ring + stage * S::STAGE_BYTES, bar = full0 + 8 * stage;
                if (i >= ahead) {
                    mbar_expect_tx(bar, S::STAGE_BYTES);
                    load_weights(i, dst, bar);
                }
                const int kb = k0 + i;
                tma_load_2d(dst + S::P_BYTES, &maps.q, kb * ROW, 0, bar);
                if (F4)
                    bulk_load_at(dst + S::P_BYTES + S::Q_BYTES + S::SCALE_BYTES, g.sq + (int64_t)kb * S::SCALE_TILES * 512,
                                 S::SCALE_BYTES, bar);
            }
            __syncwarp();
            issued = max(issued, i + 1);
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        // copies still in flight land before the CTA exits
        for (int j = max(0, issued - STAGES); j < issued; ++j) {
            const bool landed = warp_wait(full0 + 8 * (uint32_t)(j % STAGES), (uint32_t)(j / STAGES & 1), kTileWaitNs);
            ok = ok && landed;
            if (!landed) break;
        }
        if (!ok && lane == 0) tile_timeout();
    } else if (warp == 1) {
        constexpr uint32_t IDESC = F4 ? tc5::idesc_e2m1(KIND == kKindMx, 128, NQ)
                                      : tc5::idesc_f16(KIND == kKindBF16, false, false, 128, NQ);
        const uint64_t pd0 = tc5::desc_kmajor_sw128(ring), qd0 = tc5::desc_kmajor_sw128(ring + S::P_BYTES);
        const uint64_t sd0 = tc5::desc_scale_tile(ring + S::P_BYTES + S::Q_BYTES);
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        for (int i = 0; i < count; ++i) {
            ok = warp_wait(full0 + 8 * stage, phase, kTileWaitNs);
            if (!ok) break;
            tc5::fence_after_sync();
            if (elect_one()) {
                const uint64_t off = (uint64_t)((stage * S::STAGE_BYTES) >> 4);
                const int steps = k0 + i == g.nk - 1 ? g.last_steps : 4;
                if constexpr (F4) {
                    const uint32_t sc = tmem + S::ACC_COLS + (i & 1) * 32;
                    const uint64_t sd = sd0 + off;
#pragma unroll
                    for (int t = 0; t < S::SCALE_TILES; ++t) {
                        tc5::cp_scales_single(sc + t * 4, sd + t * 32);
                        tc5::cp_scales_single(sc + 16 + t * 4, sd + (S::SCALE_TILES + t) * 32);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= steps) break;
                        const uint32_t acc = (i | j) != 0 ? 1u : 0u;
                        if (KIND == kKindMx)
                            tc5::mma_mx_single(tmem, pd0 + off + 2 * j, qd0 + off + 2 * j,
                                               tc5::idesc_scale_byte(IDESC, (j & 1) * 2), sc + (j / 2) * 4,
                                               sc + 16 + (j / 2) * 4, acc);
                        else
                            tc5::mma_nv_single(tmem, pd0 + off + 2 * j, qd0 + off + 2 * j, IDESC, sc + j * 4,
                                               sc + 16 + j * 4, acc);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= steps) break;
                        tc5::mma_f16_single(tmem, pd0 + off + 2 * j, qd0 + off + 2 * j, IDESC, (i | j) != 0 ? 1u : 0u);
                    }
                }
                tc5::commit(empty0 + 8 * stage);
                if (i == count - 1) tc5::commit(done_bar);
            }
            __syncwarp();
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) {  // what was issued still has to finish
            if (elect_one()) tc5::commit(done_bar);
            __syncwarp();
            if (lane == 0) tile_timeout();
        }
    }
    __syncwarp();

    // Units of outputs: 32 weight rows of one token, or (UNITS = 2) 32 rows of g
    // and the 32 of u that go with them.  Unit w belongs to CTA w % splits, at
    // slot w / splits of its memory; a slot holds a row of 32 for each CTA.
    // Once every MMA of the cluster has finished, the rings hold nothing more.
    constexpr int HALVES = Epi::HALVES, PARTS = Epi::UNITS * HALVES, PER_TOKEN = 4 / Epi::UNITS;
    static_assert(PARTS <= 2, "two sums of a unit at most");
    const int tokens = g.M, units = tokens * PER_TOKEN, splits = g.splits, columns = tokens * HALVES;
    if (!warp_wait(done_bar, 0, 2 * kTileWaitNs) && lane == 0) tile_timeout();
    tc5::fence_after_sync();
    cluster_sync();
    if (warp >= 2) {
        const int q = warp & 3;  // 32 rows of the tile: of which unit, and which of its parts
        const int unit = Epi::UNITS == 1 ? q : PAIRED16 ? q % 2 : q / 2;
        const int part = Epi::UNITS == 1 ? 0 : PAIRED16 ? q / 2 : q % 2;
        const uint32_t mine = ring + (uint32_t)(z * PARTS + part) * 128 + lane * 4, pitch = (uint32_t)(splits * PARTS) * 128;
        const uint32_t inverse = 65536u / (uint32_t)splits + 1u;  // w / splits = w * inverse >> 16 for w < 4096
#pragma unroll 1
        for (int c = (warp - 2) / 4 * 16; c < columns; c += 32) {
            uint32_t v[16];
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
                "tcgen05.wait::ld.sync.aligned;\n"
                : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                  "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                : "r"(tmem + ((uint32_t)(q * 32) << 16) + c)
                : "memory");
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool second = HALVES == 2 && c + i >= tokens;
                const uint32_t w = (uint32_t)((c + i - (second ? tokens : 0)) * PER_TOKEN + unit), slot = w * inverse >> 16;
                if (c + i < columns)
                    st_cluster(cluster_addr(mine + slot * pitch + (second ? 128 : 0), w - slot * splits), v[i]);
            }
        }
    }
    tc5::fence_before_sync();
    cluster_sync();
    tc5::fence_after_sync();
    if (warp == 1) tc5::tmem_dealloc(tmem, S::TMEM_COLS);

    pdl_wait();  // the other warps' first access to global memory
    for (int slot = warp; slot * splits + z < units; slot += kSplitThreads / 32) {
        const int w = slot * splits + z;
        const uint32_t at = ring + (uint32_t)(slot * splits * PARTS) * 128 + lane * 4;
        float p0[kMaxCluster], p1[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            p0[c] = c < splits ? ld_shared(at + c * PARTS * 128) : 0.0f;
            if (PARTS == 2) p1[c] = c < splits ? ld_shared(at + c * PARTS * 128 + 128) : 0.0f;
        }
        float v0 = p0[0], v1 = PARTS == 2 ? p1[0] : 0.0f;
#pragma unroll
        for (int c = 1; c < kMaxCluster; ++c) {
            if (c >= splits) break;
            v0 += p0[c];
            if (PARTS == 2) v1 += p1[c];
        }
        epi.emit(v0, v1, w / PER_TOKEN, w % PER_TOKEN, lane, nt);
    }
}

template <int KIND, int NQ, bool PAIRED16, class Epi>
cudaError_t launch_split_sized(SplitArgs g, const SplitMaps& maps, const Epi& epi, cudaStream_t st) {
    using S = SplitShape<KIND, NQ>;
    static std::atomic<uint64_t> ready{0};  // devices whose attribute is set
    auto* kernel = split_gemm_kernel<KIND, NQ, PAIRED16, Epi>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (err != cudaSuccess) return err;
        ready.fetch_or(1ULL << dev, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)g.nt * g.splits));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)g.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, g, maps, epi);
}

// Tokens that a CTA multiplies: the least of 16, 32, 64 and 128 that holds them all.
inline int split_nq(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// CTAs along k: as many as two to an SM give each tile, at most a cluster,
// with at least two stages each.
inline int split_count(int64_t tiles, int nk) {
    const int64_t slots = 2 * (int64_t)device_sms();
    int64_t s = std::min<int64_t>(kMaxCluster, std::max<int64_t>(1, slots / std::max<int64_t>(1, tiles)));
    s = std::min<int64_t>(s, std::max(1, nk / 2));
    const int per = (int)((nk + s - 1) / s);
    return (nk + per - 1) / per;
}

// Up to how many tokens the split kernel takes a product; beyond, the pairs'
// tiles are faster although they leave SMs idle.  Weights from HBM, us:
//                          33 tokens         64 tokens        128 tokens
//                        split    pairs    split    pairs    split    pairs
//   8192 x 8192 nvfp4     10.7     12.9     12.0     13.0     15.5     13.3
//   8192 x 8192 mxfp4      9.7     10.9     10.8     11.1
//   4096 x 12288 mxfp4     8.4     12.9      9.6     13.0     12.6     13.4
//   2048 x 16384 mxfp4     8.2     15.4      9.5     15.6
//   512 x 16384 nvfp4      6.3     16.2      7.3     16.3
//   12288 x 4096 mxfp4     9.1     10.4     10.0      9.4     13.6      9.8
//   8192 x 1024 mxfp4      5.2      4.8      6.3      5.1
//   2048 x 1024 nvfp4      5.4      5.3      6.9      5.5
//   16-bit block 4096 x 12288               59.9     79.0     68.9     80.4
// Short sums are the exception from 33 tokens on, by up to 1.4 us.
constexpr int kSplitTokens4 = 64, kSplitTokens16 = 128;

template <int KIND, bool PAIRED16, class Epi>
cudaError_t launch_split_gemm(SplitArgs g, const SplitMaps& maps, const Epi& epi, cudaStream_t st) {
    // rows of the tokens' matrix: what the callers send here at most
    constexpr int MOST = Epi::HALVES == 2 ? 2 * (int)kFullTokens : kind_is_4bit(KIND) ? kSplitTokens4 : kSplitTokens16;
    const int rows = g.M * Epi::HALVES;
    if (rows > MOST) return cudaErrorInvalidValue;
    g.splits = split_count(g.nt, g.nk);
    g.per = (g.nk + g.splits - 1) / g.splits;
    const int nq = split_nq(rows);
    if (nq == 16) return launch_split_sized<KIND, 16, PAIRED16>(g, maps, epi, st);
    if constexpr (MOST >= 64) {
        if (nq == 64) return launch_split_sized<KIND, 64, PAIRED16>(g, maps, epi, st);
    }
    if constexpr (MOST >= 128) {
        if (nq == 128) return launch_split_sized<KIND, 128, PAIRED16>(g, maps, epi, st);
    }
    return launch_split_sized<KIND, 32, PAIRED16>(g, maps, epi, st);
}

}  // namespace
}  // namespace ddg
