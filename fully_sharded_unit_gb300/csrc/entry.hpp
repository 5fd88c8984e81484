// What the C entry points of the compute handle share: the handle itself, and the checks
// of callers' arguments.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <new>
#include <string>

#include "compute.hpp"
#include "fsdp_unit.h"

namespace fsdp {
// Records the calling thread's failure reason for fsdp_last_error (api.cu).
int record_error(int code, const std::string& why);
}  // namespace fsdp

constexpr int64_t kHeader = 256;

struct fsdp_compute {
    int device = 0;
    int sms = 0;
    fsdp_allocator allocator{nullptr, nullptr, nullptr};   // alloc == nullptr: cudaMalloc / cudaFree
    char* block = nullptr;        // status word, then the workspace
    int64_t workspace_bytes = 0;
    unsigned long long wait_ns = 10000000000ull;
    int withhold_next = 0;
    bool broken = false;          // a drain wait ran out: only destroy is accepted

    int32_t* status() const { return reinterpret_cast<int32_t*>(block); }
    char* workspace() const { return block + kHeader; }
};

namespace fsdp {

inline int fail(int code, const std::string& why) { return record_error(code, why); }

inline int cuda_fail(cudaError_t e, const char* what) {
    cudaGetLastError();   // reported here, not to whoever asks next
    return fail(FSDP_E_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// Runs an entry point's body; nothing it throws (a message that finds no
// memory) crosses the C boundary.
template <typename F>
int entry(F&& body) noexcept {
    try {
        return body();
    } catch (const std::bad_alloc&) {
        return FSDP_E_OOM;
    } catch (...) {
        return FSDP_E_STATE;
    }
}

class OnDevice {
public:
    explicit OnDevice(int device) : device_(device) {
        if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = -1;
        if (prev_ != device_) ok_ = cudaSetDevice(device_) == cudaSuccess;
    }
    ~OnDevice() {
        if (prev_ >= 0 && prev_ != device_) cudaSetDevice(prev_);
    }
    bool ok() const { return ok_; }

private:
    int device_;
    int prev_ = -1;
    bool ok_ = true;
};

#define TRY(expr)                 \
    do {                          \
        const int rc_ = (expr);   \
        if (rc_ != FSDP_OK) return rc_; \
    } while (0)

constexpr int64_t kMaxDim = int64_t(1) << 40;

enum Types { kFloats = 1, kBf16 = 2, kAct8 = 4 };   // kFloats: F32 and BF16

// Checks a caller's matrix against the shape and types an operand may have.
inline int take(const fsdp_matrix* m, const char* name, int64_t rows, int64_t cols, int types, Mat* out) {
    const std::string who(name);
    if (m == nullptr) return fail(FSDP_E_INVALID_ARG, who + " is null");
    const bool act8 = m->dtype == FSDP_DTYPE_ACT8;
    const bool known = (m->dtype == FSDP_DTYPE_F32 && (types & kFloats)) ||
                       (m->dtype == FSDP_DTYPE_BF16 && (types & (kFloats | kBf16))) || (act8 && (types & kAct8));
    if (!known) return fail(FSDP_E_INVALID_ARG, who + " has a dtype this operand cannot have");
    if (m->rows != rows || m->cols != cols)
        return fail(FSDP_E_INVALID_ARG, who + " is " + std::to_string(m->rows) + " x " + std::to_string(m->cols) +
                                            ", expected " + std::to_string(rows) + " x " + std::to_string(cols));
    if (act8 && m->ld != act8_groups(cols) * kGroup)
        return fail(FSDP_E_INVALID_ARG, who + ": ld of an ACT8 matrix is 32*ceil(cols/32)");
    if (m->ld < cols) return fail(FSDP_E_INVALID_ARG, who + ": ld is smaller than cols");
    if (m->ld > kMaxDim || (rows > 0 && m->ld > (int64_t(1) << 60) / rows))
        return fail(FSDP_E_INVALID_ARG, who + " is too large");
    if (rows > 0) {
        if (m->data == nullptr) return fail(FSDP_E_INVALID_ARG, who + ": data is null");
        const uintptr_t mask = act8 ? 15u : m->dtype == FSDP_DTYPE_F32 ? 3u : 1u;
        if (reinterpret_cast<uintptr_t>(m->data) & mask)
            return fail(FSDP_E_ALIGN, who + (act8 ? ": data is not 16-byte aligned" : ": data is not aligned to its element"));
        if (act8 && m->exps == nullptr) return fail(FSDP_E_INVALID_ARG, who + ": exps is null");
    }
    *out = Mat{m->data, act8 ? m->exps : nullptr, m->ld, act8 ? act8_groups(cols) : 0, m->dtype};
    return FSDP_OK;
}

inline int take_optional(const fsdp_matrix* m, const char* name, int64_t rows, int64_t cols, int types, Mat* out) {
    *out = Mat{};
    return m == nullptr ? FSDP_OK : take(m, name, rows, cols, types, out);
}

inline int take_vector(const void* p, const char* name, int dtype) {
    if (dtype != FSDP_DTYPE_F32 && dtype != FSDP_DTYPE_BF16)
        return fail(FSDP_E_INVALID_ARG, std::string(name) + ": dtype must be FSDP_DTYPE_F32 or FSDP_DTYPE_BF16");
    if (p == nullptr) return fail(FSDP_E_INVALID_ARG, std::string(name) + " is null");
    if (reinterpret_cast<uintptr_t>(p) & (dtype == FSDP_DTYPE_F32 ? 3u : 1u))
        return fail(FSDP_E_ALIGN, std::string(name) + " is not aligned to its element");
    return FSDP_OK;
}

inline int check_shape(int64_t rows, int64_t cols, const char* what) {
    if (rows < 0 || cols < 1 || rows > kMaxDim || cols > kMaxDim)
        return fail(FSDP_E_INVALID_ARG, std::string(what) + ": rows must be >= 0 and cols >= 1 (at most 2^40)");
    return FSDP_OK;
}

inline int check_handle(const fsdp_compute* c) {
    if (c == nullptr) return fail(FSDP_E_INVALID_ARG, "compute handle is null");
    if (c->broken)
        return fail(FSDP_E_STATE, "a kernel's copies may have landed after it ended (FSDP_KSTATUS_DRAIN_TIMEOUT); "
                                  "destroy the handle");
    return FSDP_OK;
}

inline int check_activation(int act) {
    if (act < FSDP_ACTIVATION_NONE || act > FSDP_ACTIVATION_GELU_ERF) return fail(FSDP_E_INVALID_ARG, "unknown activation");
    return FSDP_OK;
}

inline int check_workspace(const fsdp_compute* c, int64_t need) {
    if (need > c->workspace_bytes)
        return fail(FSDP_E_CAPACITY, "the call needs " + std::to_string(need) + " bytes of workspace, the handle has " +
                                         std::to_string(c->workspace_bytes));
    return FSDP_OK;
}

}  // namespace fsdp
