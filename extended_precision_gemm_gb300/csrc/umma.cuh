// umma.cuh -- tcgen05 forms beyond those of tcgen05.cuh: operands stored with
// their row or column index contiguous, f16 operands, the block-scaled 4-bit
// products with their scales in tensor memory, and tensor maps.
#pragma once

#include <cuda.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "async_copy.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace ddg {

// True in one lane of a converged warp, always the same one.  The roles below
// that issue copies and MMAs run as whole warps and elect the issuing lane at
// the instructions: their loops then stay warp-uniform, and addresses and
// descriptors live in uniform registers, where these instructions want them.
// With the loop itself inside a single lane's branch every instruction first
// moves its operands over (measured: about 30 ns per copy or MMA; an 8192^3
// nvfp4 product takes 452 us so, 176 us with elected lanes).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " elect.sync _|p, 0xffffffff;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(p));
    return p != 0;
}

// The warp's index as a warp-uniform value.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(~0u, (int)(threadIdx.x >> 5), 0); }

// A bounded wait of a whole warp: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned long long budget) {
    return __all_sync(~0u, mbar_wait_bounded(bar, parity, budget));
}

// What a product's operands are: 16-bit floating point, or 4-bit codes with
// scales (mx4.cuh).
enum Kind { kKindF16 = 0, kKindBF16 = 1, kKindMx = 2, kKindNv = 3 };
__host__ __device__ constexpr bool kind_is_4bit(int kind) { return kind >= kKindMx; }

namespace tc5 {

// Shared-memory matrix descriptor of an operand whose row index (m or n) is
// contiguous, 128-byte swizzle: blocks of 64 (m or n) by 64 k, k rows of 128
// bytes in groups of 8 (1024 bytes, the stride byte offset), the next 64 of m
// or n `block_bytes` further on (the leading byte offset).  16 k are 2048
// bytes.
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t saddr, uint32_t block_bytes) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(block_bytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Descriptor of a 512-byte scale tile for tcgen05.cp 32x128b: 32 rows of 16
// bytes, 8 rows (128 bytes) to a core matrix, no swizzle.
__device__ __forceinline__ uint64_t desc_scale_tile(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) |
           ((uint64_t)1 << 46);
}

// Instruction descriptor of kind::f16, f32 accumulator; bits 15 and 16 say
// that A or B is stored with m or n contiguous.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, bool a_mn, bool b_mn, int M, int N) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Instruction descriptor of the block-scaled kinds with E2M1 operands (format
// 1); bit 23: E8M0 scales (else E4M3).  Bits 4-5 and 29-30 take the byte of a
// 32-bit scale word at which B's and A's scales of this MMA begin.
__host__ __device__ constexpr uint32_t idesc_e2m1(bool e8m0, int M, int N) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_scale_byte(uint32_t idesc, uint32_t byte) {
    return idesc | (byte << 4) | (byte << 29);
}

#define DDG_MMA_16(name, group)                                                                                    \
    __device__ __forceinline__ void name(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) { \
        asm volatile(                                                                                              \
            "{\n"                                                                                                  \
            " .reg .pred p;\n"                                                                                     \
            " setp.ne.b32 p, %4, 0;\n"                                                                             \
            " tcgen05.mma.cta_group::" group ".kind::f16 [%0], %1, %2, %3, p;\n"                                   \
            "}\n" ::"r"(d),                                                                                        \
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                                                            \
            : "memory");                                                                                           \
    }
DDG_MMA_16(mma_f16_single, "1")
DDG_MMA_16(mma_f16_pair, "2")
#undef DDG_MMA_16

#define DDG_MMA_4(name, group, kind, vec)                                                                           \
    __device__ __forceinline__ void name(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, \
                                         uint32_t accumulate) {                                                     \
        asm volatile(                                                                                               \
            "{\n"                                                                                                   \
            " .reg .pred p;\n"                                                                                      \
            " setp.ne.b32 p, %6, 0;\n"                                                                              \
            " tcgen05.mma.cta_group::" group ".kind::" kind ".block_scale.scale_vec::" vec                          \
            " [%0], %1, %2, %3, [%4], [%5], p;\n"                                                                   \
            "}\n" ::"r"(d),                                                                                         \
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                                           \
            : "memory");                                                                                            \
    }
DDG_MMA_4(mma_mx_single, "1", "mxf4", "2X")
DDG_MMA_4(mma_nv_single, "1", "mxf4nvf4", "4X")
DDG_MMA_4(mma_mx_pair, "2", "mxf4", "2X")
DDG_MMA_4(mma_nv_pair, "2", "mxf4nvf4", "4X")
#undef DDG_MMA_4

// A 512-byte scale tile into four tensor memory columns, repeated in each 32
// lanes.  Runs in order with the MMAs of the issuing thread.
__device__ __forceinline__ void cp_scales_single(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

}  // namespace tc5

// Tensor copy of a 2-D box into this CTA's shared memory, completing on its
// own barrier.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d_group(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Plain copy of `bytes` (a multiple of 16, both sides 16-byte aligned) into this
// CTA's shared memory.
__device__ __forceinline__ void bulk_load_at(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// The box at (x, y) into L2 only.  Safe before the wait for earlier work on the
// stream: whoever writes the box later writes it in L2 as well.
__device__ __forceinline__ void tma_prefetch_2d(const void* tmap, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tmap), "r"(x), "r"(y) : "memory");
}

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled tensor_map_encoder() {
    static std::atomic<EncodeTiled> cached{nullptr};
    EncodeTiled fn = cached.load(std::memory_order_acquire);
    if (fn == nullptr) {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<EncodeTiled>(ptr);
            cached.store(fn, std::memory_order_release);
        } else {
            (void)cudaGetLastError();
        }
    }
    return fn;
}

// A row-major matrix of `rows` rows of `cols` elements, `ld_bytes` apart, read
// in boxes of box_cols x box_rows; what lies outside reads as zero.  The base
// and ld_bytes are multiples of 16.
cudaError_t make_map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t cols,
                        int64_t rows, int64_t ld_bytes, int box_cols, int box_rows, bool swizzle) {
    const EncodeTiled fn = tensor_map_encoder();
    if (fn == nullptr) return cudaErrorNotSupported;
    if (cols <= 0 || rows <= 0 || cols >= (1LL << 31) || rows >= (1LL << 31)) return cudaErrorInvalidValue;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t elem[2] = {1, 1};
    const CUresult r = fn(m, type, 2, const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace
}  // namespace ddg
