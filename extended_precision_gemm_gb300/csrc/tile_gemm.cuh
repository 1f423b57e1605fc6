// tile_gemm.cuh -- matrix products on CTA pairs (tcgen05 cta_group::2) for the
// 4-bit products and the gated feed-forward block: one persistent kernel,
// templated on what its operands are and on the epilogue that takes the
// accumulators.  Everything is in an unnamed namespace, so each including file
// has its own count of bounded waits that gave up.
//
// D = sum over k of A[m, k] B[n, k], for up to four products in one launch.  A
// pair of CTAs on two SMs owns a tile of 256 m by NT n: each CTA holds 128 rows
// of A, one half of the rows of B, and 128 rows of the accumulators (f32, in
// tensor memory, twice: the MMAs of a tile overlap the epilogue of the one
// before).  A stage of the shared-memory ring is 128 bytes of k.  Warps: 0 copies
// (TMA), 1 issues the MMAs (even CTA only), the others run the epilogue, four
// warps (128 rows) for each group of columns.
//
// Where the tiles are few and deep, the stages of a tile are shared out among
// several units of work (splits), whose partial sums an epilogue leaves in
// planes of their own to be added afterwards.
//
// 16-bit operands: NT = 256 (128 where that fills the SMs better), 64 k to a
// stage, either operand with k contiguous or with its row index contiguous
// (64 x 64 blocks, the same swizzle); the sum may run over two segments
// (A0 B0^T + A1 B1^T).
// 4-bit operands: NT = 192 (or 128), 256 k to a stage; two accumulators of 192
// columns leave 128 columns of tensor memory to the scales (16 for A's 128
// rows, 32 for two tiles of 128 rows of B, twice).  192 rows of B start at a
// multiple of 64 rows of a scale tile: their scales begin two columns into it
// for every other tile.
//
// Bound by the tensor pipe (16 bits: 94 to 98% busy, 1.69 to 1.93 PF/s at 4096 x
// 4096 x 8192, and the power cap in a loop; 4 bits: 83% busy, 6.5 P/s at 4096 x
// 4096 x 16384; 8192^3 nvfp4 161 us and mxfp4 151, in a loop, at the power cap, 187
// and 168).  A pair's tile of 256
// by NT is the largest whose accumulators fit tensor memory twice: an epilogue
// costs up to 3 us, which one accumulator would add to every tile.  Short sums
// are bound by their epilogue all the same (depth 1280, gelu: 3 us a tile against
// 1.2 us of MMAs).
#pragma once

#include <algorithm>

#include "launch.cuh"
#include "umma.cuh"

namespace ddg {
namespace {

constexpr unsigned long long kTileWaitNs = 2000000000ULL;  // bounded waits: 2 s
constexpr int kTileGroup = 8;  // m tiles that share their n tiles while these are in L2

__device__ unsigned int g_tile_timeouts = 0;

__device__ __forceinline__ void tile_timeout() { atomicAdd(&g_tile_timeouts, 1u); }

constexpr int kMaxProducts = 4, kMaxMaps = 2 * kMaxProducts;

struct TileMaps {
    CUtensorMap a[kMaxMaps], b[kMaxMaps];  // by product and segment, or (gated) b by CTA
    CUtensorMap sa, sb;                    // scales (4-bit kinds): tiles of 128 words
};

struct TileProduct {
    int mt, nt;       // tiles along m and n
    int nk, segs;     // stages of a segment, segments
    int last_steps;   // MMAs in a segment's last stage
    int map;          // its first maps
    int a_mn;         // A stored with m contiguous (kernels that take either)
    int splits, per;  // units that share a tile, stages of one (the last may have fewer)
    int64_t first;    // first unit
};

struct TileArgs {
    TileProduct p[kMaxProducts];
    int64_t units;  // of all products
    int products;
    int pairs;      // CTA pairs in the grid
    int tiles_k;    // 4-bit kinds: scale tiles in a row of 128
};

template <int KIND, int NT_>
struct TileShape {
    static constexpr bool F4 = kind_is_4bit(KIND);
    static constexpr int NT = NT_;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = NT / 2 * 128;
    static constexpr int SCALE_TILES = F4 ? (KIND == kKindMx ? 2 : 4) : 0;  // per stage and 128 rows
    static constexpr int SB_BLOCKS = NT % 128 == 0 ? NT / 128 : 2;          // 128-row blocks under a tile of B
    static constexpr int SA_BYTES = SCALE_TILES * 512, SB_BYTES = SB_BLOCKS * SA_BYTES;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
    static constexpr int STAGES = 208 * 1024 / STAGE_BYTES;  // the rest is L1, for the epilogue's loads
    static constexpr int SMEM = STAGES * STAGE_BYTES + 1024;
    static constexpr uint32_t SCALE_COL = 2 * NT, SCALE_COLS = 64;  // two sets
    static_assert(STAGE_BYTES % 1024 == 0 && SMEM + 1024 <= 227 * 1024, "shared memory");
    static_assert(!F4 || SCALE_COL + 2 * SCALE_COLS <= 512, "tensor memory");
};

// Unit t: split z of tile (m, n) of product p.
__device__ __forceinline__ void tile_of(const TileArgs& g, int64_t t, int& z, int& p, int& m, int& n) {
    p = 0;
#pragma unroll
    for (int i = 1; i < kMaxProducts; ++i)
        if (i < g.products && t >= g.p[i].first) p = i;
    const TileProduct& q = g.p[p];
    t -= q.first;
    const int64_t tiles = (int64_t)q.mt * q.nt;
    z = q.splits > 1 ? (int)(t / tiles) : 0;
    t -= z * tiles;
    const int64_t per_group = (int64_t)kTileGroup * q.nt;
    const int64_t group = t / per_group;
    const int first = (int)group * kTileGroup, size = min(kTileGroup, q.mt - first);
    m = first + (int)((t % per_group) % size);
    n = (int)((t % per_group) / size);
}

// How A is stored: k contiguous, or k or m as each product says.
enum Major { kMajorK = 0, kMajorAny = 1 };

// Epi: NT, GROUPS, and run(acc, product, split, m row, n tile, group, lane, release): takes this
// warp's 32 rows of the accumulators from column `acc` on (all lanes, also for
// rows beyond the matrix) and calls release() after its last read of them.
template <int KIND, int A_MAJOR, bool B_MN, bool GATED, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(64 + 128 * Epi::GROUPS, 1)
    tile_gemm_kernel(const __grid_constant__ TileArgs g, const __grid_constant__ TileMaps maps,
                     const __grid_constant__ Epi epi) {
    using S = TileShape<KIND, Epi::NT>;
    constexpr int STAGES = S::STAGES, NT = S::NT;
    constexpr bool F4 = S::F4;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * STAGES + 5];
    __shared__ uint32_t tmem_slot;

    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int64_t pair = blockIdx.x >> 1;
    const int64_t units = g.units;

    const uint32_t full0 = smem_addr(&bars[0]), empty0 = smem_addr(&bars[STAGES]);
    const uint32_t accf0 = smem_addr(&bars[2 * STAGES]), acce0 = smem_addr(&bars[2 * STAGES + 2]);
    const uint32_t done_bar = smem_addr(&bars[2 * STAGES + 4]);

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, 2 * 4 * Epi::GROUPS);
        }
        mbar_init(done_bar, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tc5::tmem_alloc_pair(smem_addr(&tmem_slot), 512);
        tc5::tmem_relinquish_pair();
    }
    tc5::fence_before_sync();
    cluster_sync();
    tc5::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        // ---- copies; both CTAs' complete on the even CTA's barriers ----
        const uint32_t full_lead0 = cluster_addr(full0, 0);
        uint32_t stage = 0, phase = 0;
        int64_t issued = 0;
        bool ok = true;
        for (int64_t t = pair; t < units && ok; t += g.pairs) {
            int z, p, mt, nt;
            tile_of(g, t, z, p, mt, nt);
            const TileProduct& q = g.p[p];
            const int it0 = z * q.per, per_tile = min(q.per, q.nk * q.segs - it0);
            const bool a_mn = A_MAJOR == kMajorAny && q.a_mn != 0;
            const int a_row = (mt * 2 + (int)rank) * 128;
            const int b_row = GATED ? nt * (NT / 2) : nt * NT + (int)rank * (NT / 2);
            int seg = it0 / q.nk, kb = it0 % q.nk;
            for (int it = 0; it < per_tile; ++it) {
                ok = warp_wait(empty0 + 8 * stage, phase ^ 1, kTileWaitNs);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t dst = ring + stage * S::STAGE_BYTES, bar = full_lead0 + 8 * stage;
                    const CUtensorMap* ma = &maps.a[q.map + seg];
                    const CUtensorMap* mb = &maps.b[GATED ? rank : q.map + seg];
                    if (leader) mbar_expect_tx(full0 + 8 * stage, 2u * S::STAGE_BYTES);
                    constexpr int ROW = F4 ? 128 : 64;  // elements (bytes of codes) of a 128-byte row
                    if (!a_mn) {
                        tma_load_2d_group(dst, ma, kb * ROW, a_row, bar);
                    } else {
                        tma_load_2d_group(dst, ma, a_row, kb * 64, bar);
                        tma_load_2d_group(dst + 8192, ma, a_row + 64, kb * 64, bar);
                    }
                    const uint32_t db = dst + S::A_BYTES;
                    if (!B_MN) {
                        tma_load_2d_group(db, mb, kb * ROW, b_row, bar);
                    } else {
                        static_assert(!B_MN || NT % 128 == 0, "whole blocks of 64");
#pragma unroll
                        for (int i = 0; i < NT / 128; ++i)
                            tma_load_2d_group(db + i * 8192, mb, b_row + i * 64, kb * 64, bar);
                    }
                    if (F4) {
                        const uint32_t ds = db + S::B_BYTES;
                        const int t0 = kb * S::SCALE_TILES, rb = nt * NT / 128;
                        tma_load_2d_group(ds, &maps.sa, 0, (mt * 2 + (int)rank) * g.tiles_k + t0, bar);
                        tma_load_2d_group(ds + S::SA_BYTES, &maps.sb, 0, rb * g.tiles_k + t0, bar);
                        if (S::SB_BLOCKS == 2)
                            tma_load_2d_group(ds + 2 * S::SA_BYTES, &maps.sb, 0, (rb + 1) * g.tiles_k + t0, bar);
                    }
                }
                __syncwarp();
                if (++kb == q.nk) { kb = 0; ++seg; }
                ++issued;
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
        }
        // copies still in flight land before the CTA exits: the even CTA
        // waits for its last stages to fill, the odd CTA (whose copies
        // complete on the even CTA's barriers) for them to be consumed
        const int64_t first = issued > STAGES ? issued - STAGES : 0;
        for (int64_t j = first; j < issued; ++j) {
            const uint32_t bar = (leader ? full0 : empty0) + 8 * (uint32_t)(j % STAGES);
            const bool landed = warp_wait(bar, (uint32_t)((j / STAGES) & 1), kTileWaitNs);
            ok = ok && landed;
            if (!landed) break;
        }
        if (!ok && lane == 0) tile_timeout();
    } else if (warp == 1) {
        bool ok = true;
        if (leader) {
            // ---- MMAs ----
            constexpr uint32_t IDESC = F4 ? tc5::idesc_e2m1(KIND == kKindMx, 256, NT)
                                          : tc5::idesc_f16(KIND == kKindBF16, false, B_MN, 256, NT);
            constexpr uint64_t B_STEP = B_MN ? 2048 / 16 : 2;
            const uint64_t bd0 = B_MN ? tc5::desc_mnmajor_sw128(ring + S::A_BYTES, 8192)
                                      : tc5::desc_kmajor_sw128(ring + S::A_BYTES);
            const uint64_t sd0 = tc5::desc_scale_tile(ring + S::A_BYTES + S::B_BYTES);
            uint32_t stage = 0, phase = 0, count = 0;
            for (int64_t t = pair; t < units && ok; t += g.pairs, ++count) {
                int z, p, mt, nt;
                tile_of(g, t, z, p, mt, nt);
                const TileProduct& q = g.p[p];
                const int it0 = z * q.per, per_tile = min(q.per, q.nk * q.segs - it0), nk = q.nk, last_steps = q.last_steps;
                const bool a_mn = A_MAJOR == kMajorAny && q.a_mn != 0;
                const uint64_t ad0 = a_mn ? tc5::desc_mnmajor_sw128(ring, 8192) : tc5::desc_kmajor_sw128(ring);
                const uint64_t a_step = a_mn ? 2048 / 16 : 2;
                const uint32_t idesc = IDESC | (a_mn ? 1u << 15 : 0u);
                const uint32_t buf = count & 1;
                const uint32_t d = tmem + buf * NT;
                ok = warp_wait(acce0 + 8 * buf, ((count >> 1) & 1) ^ 1, kTileWaitNs);
                if (!ok) break;
                tc5::fence_after_sync();
                int kb = it0 % nk;
                for (int it = 0; it < per_tile; ++it) {
                    ok = warp_wait(full0 + 8 * stage, phase, kTileWaitNs);
                    if (!ok) break;
                    tc5::fence_after_sync();
                    if (elect_one()) {
                        const uint64_t off = (uint64_t)((stage * S::STAGE_BYTES) >> 4);
                        const uint64_t ad = ad0 + off, bd = bd0 + off;
                        const int steps = kb == nk - 1 ? last_steps : 4;
                        if constexpr (F4) {
                            const uint32_t sc = tmem + S::SCALE_COL + (it & 1) * S::SCALE_COLS;
                            const uint64_t sd = sd0 + off;
                            constexpr int SB = 4 * S::SB_BLOCKS;  // columns of B's scales for 4 blocks of k
#pragma unroll
                            for (int i = 0; i < S::SCALE_TILES; ++i) {
                                tc5::cp_scales_pair(sc + i * 4, sd + i * 32);
                                tc5::cp_scales_pair(sc + 16 + i * SB, sd + (S::SCALE_TILES + i) * 32);
                                if (S::SB_BLOCKS == 2)
                                    tc5::cp_scales_pair(sc + 16 + i * SB + 4, sd + (2 * S::SCALE_TILES + i) * 32);
                            }
                            const uint32_t sbo = NT == 192 ? (uint32_t)(nt & 1) * 2 : 0u;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (j >= steps) break;
                                const uint32_t acc = (it | j) != 0 ? 1u : 0u;
                                if (KIND == kKindMx)
                                    tc5::mma_mx_pair(d, ad + 2 * j, bd + B_STEP * j,
                                                     tc5::idesc_scale_byte(IDESC, (j & 1) * 2), sc + (j / 2) * 4,
                                                     sc + 16 + (j / 2) * SB + sbo, acc);
                                else
                                    tc5::mma_nv_pair(d, ad + 2 * j, bd + B_STEP * j, IDESC, sc + j * 4,
                                                     sc + 16 + j * SB + sbo, acc);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (j >= steps) break;
                                tc5::mma_f16_pair(d, ad + a_step * j, bd + B_STEP * j, idesc, (it | j) != 0 ? 1u : 0u);
                            }
                        }
                        tc5::commit_pair(empty0 + 8 * stage, 0x3);
                        if (it == per_tile - 1) tc5::commit_pair(accf0 + 8 * buf, 0x3);
                    }
                    __syncwarp();
                    if (++kb == nk) kb = 0;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
            if (pair < units) {
                if (elect_one()) tc5::commit_pair(done_bar, 0x3);
                __syncwarp();
            }
        }
        // every MMA has finished before either CTA gives up its shared or
        // tensor memory
        if (pair < units) ok = warp_wait(done_bar, 0, leader ? kTileWaitNs : kTileWaitNs * 4) && ok;
        if (!ok && lane == 0) tile_timeout();
    } else {
        // ---- epilogue ----
        const int q = warp & 3, group = (warp - 2) >> 2;
        uint32_t count = 0;
        for (int64_t t = pair; t < units; t += g.pairs, ++count) {
            int z, p, mt, nt;
            tile_of(g, t, z, p, mt, nt);
            const uint32_t buf = count & 1;
            if (!warp_wait(accf0 + 8 * buf, (count >> 1) & 1, kTileWaitNs)) {
                if (lane == 0) tile_timeout();
                break;
            }
            tc5::fence_after_sync();
            const int64_t row = ((int64_t)mt * 2 + rank) * 128 + q * 32 + lane;
            epi.run(tmem + buf * NT + ((uint32_t)(q * 32) << 16), p, z, row, nt, group, lane, [&]() {
                tc5::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(acce0 + 8 * buf);
                    else mbar_arrive_remote(acce0 + 8 * buf, 0);
                }
            });
            __syncwarp();
        }
    }

    // neither CTA leaves while its peer may still touch its shared memory
    tc5::fence_before_sync();
    cluster_sync();
    tc5::fence_after_sync();
    if (warp == 1) {
        __syncwarp();
        tc5::tmem_dealloc_pair(tmem, 512);
    }
}

// Launch on as many CTA pairs as can be resident (never more than tiles).
template <int KIND, int A_MAJOR, bool B_MN, bool GATED, class Epi>
cudaError_t launch_tile_gemm(TileArgs g, const TileMaps& maps, const Epi& epi, cudaStream_t st) {
    using S = TileShape<KIND, Epi::NT>;
    static std::atomic<int> cached[64];  // resident pairs per device; 0 = not asked yet
    auto* kernel = tile_gemm_kernel<KIND, A_MAJOR, B_MN, GATED, Epi>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(64 + 128 * Epi::GROUPS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    int pairs = cached[dev].load(std::memory_order_relaxed);
    if (pairs <= 0) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (err != cudaSuccess) return err;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)(2 * std::max(1, device_sms() / 2)));
        if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs <= 0) {
            (void)cudaGetLastError();
            pairs = std::max(1, device_sms() / 2);
        } else {
            cached[dev].store(pairs, std::memory_order_relaxed);
        }
    }
    g.units = 0;
    for (int p = 0; p < g.products; ++p) {
        TileProduct& q = g.p[p];
        if (q.splits < 1) q.splits = 1;
        q.per = (q.nk * q.segs + q.splits - 1) / q.splits;
        q.first = g.units;
        g.units += (int64_t)q.mt * q.nt * q.splits;
    }
    if (g.units <= 0) return cudaSuccess;
    g.pairs = (int)std::min<int64_t>(pairs, g.units);
    cfg.numAttrs = 2;
    cfg.gridDim = dim3((unsigned)(2 * g.pairs));
    return cudaLaunchKernelEx(&cfg, kernel, g, maps, epi);
}

cudaError_t reset_tile_timeouts(unsigned int* count) {
    cudaError_t err = cudaDeviceSynchronize();
    if (err != cudaSuccess) return err;
    err = cudaMemcpyFromSymbol(count, g_tile_timeouts, sizeof(unsigned int));
    if (err != cudaSuccess) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_tile_timeouts, &zero, sizeof(unsigned int));
}

// Tiles of 128 columns instead of `wide` (256 or 192) where the pairs' rounds
// over the narrow ones are shorter: a narrow tile takes `narrow_cost` of a wide
// one's time, more than its share (its rows of A are read for fewer columns).
inline bool narrow_tiles(int64_t wide_tiles, int64_t narrow_count, double narrow_cost) {
    const int64_t pairs = std::max(1, device_sms() / 2);
    const int64_t wide_rounds = (wide_tiles + pairs - 1) / pairs, rounds = (narrow_count + pairs - 1) / pairs;
    return (double)rounds * narrow_cost < (double)wide_rounds;
}

// ---- pieces of epilogues ----

__device__ __forceinline__ void store_v8(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void load_v8(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}

// Whether the rows of a matrix begin at whole 32-byte sectors.
template <typename T>
inline bool aligned_rows(const void* C, int64_t ldc) {
    return ((uintptr_t)C | (uintptr_t)(ldc * (int64_t)sizeof(T))) % 32 == 0;
}

// Blocks of N x N words, one in each N lanes of a warp: lane l holds row l of
// its block on entry, column l on return.
template <int N, typename W>
__device__ __forceinline__ void turn(W (&v)[N], int lane) {
#pragma unroll
    for (int s = N / 2; s > 0; s >>= 1) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i & s) continue;
            const W got = __shfl_xor_sync(~0u, up ? v[i] : v[i | s], s);
            v[i] = up ? got : v[i];
            v[i | s] = up ? v[i | s] : got;
        }
    }
}

// A warp's 32 rows by 32 columns of C from (row0, c) on; lane l holds row
// row0 + l.  Rows and columns beyond M and N are left out.  ALIGNED rows leave
// in whole 32-byte sectors.  Others are turned first, so that a warp's stores
// are contiguous: 32 elements of a row, or, of 16-bit elements whose rows are
// 4-byte aligned, 16 words of each of two.  (A thread storing its own row
// element by element made a product of 333 x 2050 x 4100 take 27 us instead of
// 14.  8192 x N x 1024 mxfp4, in bf16: 39 us for N = 8192, 51 for 8190, 87 for
// 8191, 84 for 8190 without the words; in f32 84 for 8188, 175 with each row
// stored by its thread in 16-byte pieces, 107 for 8191.  A variant of the kernel
// for each: both paths in one cost the aligned one registers, 12% of a 4096^3
// nvfp4 product.)
template <bool ALIGNED, typename T>
__device__ __forceinline__ void store_block(T* C, int64_t ldc, int64_t row0, int64_t M, int64_t c, int64_t N,
                                            float (&v)[32], int lane) {
    if constexpr (ALIGNED) {
        if (row0 + lane >= M) return;
        T* p = C + (row0 + lane) * ldc + c;
        constexpr int PER = 32 / sizeof(T);
        if (c + 32 <= N) {
#pragma unroll
            for (int i = 0; i < 32; i += PER) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(v[i + j]);
                    else w[j] = pack2<T>(v[i + 2 * j], v[i + 2 * j + 1]);
                }
                store_v8(p + i, w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i < N) p[i] = from_float<T>(v[i]);
        }
    } else {
        if (c >= N || row0 >= M) return;
        if constexpr (sizeof(T) == 2) {
            if (((uintptr_t)C | (uintptr_t)(ldc * 2)) % 4 == 0) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
                turn<16>(w, lane);  // word i: row (lane & 16) + i, columns 2 (lane & 15) and the next
                const int64_t row = row0 + (lane & 16), col = c + 2 * (lane & 15);
                const int rows = (int)min((int64_t)16, max((int64_t)0, M - row));
                T* p = C + row * ldc + col;
                if (col + 1 < N) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < rows) *reinterpret_cast<uint32_t*>(p + i * ldc) = w[i];
                } else if (col < N) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < rows) reinterpret_cast<uint16_t*>(p)[i * ldc] = (uint16_t)w[i];
                }
                return;
            }
        }
        turn<32>(v, lane);
        const int rows = (int)min((int64_t)32, M - row0);
        T* p = C + row0 * ldc + c + lane;
        if (c + lane < N) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < rows) p[i * ldc] = from_float<T>(v[i]);
        }
    }
}

// 32 values of a row of one of the library's own planes (32-byte aligned rows).
template <typename T>
__device__ __forceinline__ void store_row(T* p, const float (&v)[32]) {
    constexpr int PER = 32 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 32; i += PER) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(v[i + j]);
            else w[j] = pack2<T>(v[i + 2 * j], v[i + 2 * j + 1]);
        }
        store_v8(p + i, w);
    }
}

}  // namespace
}  // namespace ddg
