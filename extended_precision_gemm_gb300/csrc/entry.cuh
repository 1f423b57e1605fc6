// entry.cuh -- pieces of the C entry points of the 4-bit, feed-forward and
// attention calls: argument checks, workspaces, packed arguments.
#pragma once

#include <cstdint>
#include <cstring>

#include "launch.cuh"

namespace ddg {
namespace {

constexpr int64_t kAlign = 256;

inline bool known_format(int f) { return f == DDGEMM_MXFP4 || f == DDGEMM_NVFP4; }
inline bool known_type(int t) { return t == DDGEMM_F32 || t == DDGEMM_BF16 || t == DDGEMM_F16; }
inline bool known_type16(int t) { return t == DDGEMM_BF16 || t == DDGEMM_F16; }
inline bool known_activation(int a) { return a >= DDGEMM_ACT_SILU && a <= DDGEMM_ACT_RELU; }
inline int64_t type_bytes(int t) { return t == DDGEMM_F32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// Bytes from the first to the last element of a matrix.
inline int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
    return rows == 0 || cols == 0 ? 0 : ((rows - 1) * ld + cols) * elem;
}
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    if (a == nullptr || b == nullptr || na <= 0 || nb <= 0) return false;
    return (uintptr_t)a < (uintptr_t)b + (uintptr_t)nb && (uintptr_t)b < (uintptr_t)a + (uintptr_t)na;
}

inline ddgemm_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return DDGEMM_OK;
    (void)cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? DDGEMM_ERR_ALLOC : DDGEMM_ERR_CUDA;
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
template <> inline int Words::number<int>(int i) const {
    const int64_t v = word(i);
    return v >= 0 && v < (1 << 30) ? (int)v : -1;
}

}  // namespace
}  // namespace ddg
