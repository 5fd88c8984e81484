// C entry points of the block operators (declared in include/fsdp_unit.h).
// Every argument is checked here, before anything is enqueued; the launchers
// in norm.cu, act8.cu and linear.cu take what passed.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>

#include "compute.hpp"
#include "entry.hpp"
#include "fsdp_unit.h"

using namespace fsdp;

namespace {

int64_t norm_bytes(int64_t rows, int64_t cols) { return std::min<int64_t>(rows, kSms) * 2 * cols * 4; }

// column_sum_partials() * cols floats is no more than this.
int64_t column_sum_bytes(int64_t cols) { return (int64_t(4) * kSms * 256 + cols + 256) * 4; }

// Workspace of a weight gradient or a product: sums of shared tiles, column
// sums, aligned copies of operands.
int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

int64_t copies_offset(int64_t out_features) { return fsdp::kPartialBytes + round256(column_sum_bytes(out_features)); }

int64_t copy_bytes(int64_t rows, int64_t cols) { return round256(rows * ((cols + 7) / 8 * 8) * 2); }

constexpr int64_t kMaxSide = (int64_t(1) << 31) - 512;   // tile coordinates are 32-bit

int check_linear(int64_t T, int64_t I, int64_t O, int weight_layout) {
    if (T < 0 || I < 1 || O < 1 || T > kMaxSide || I > kMaxSide || O > kMaxSide)
        return fail(FSDP_E_INVALID_ARG, "linear: tokens must be >= 0 and features >= 1 (each below 2^31 - 512)");
    if (std::max(T, std::min(I, O)) > (int64_t(1) << 60) / std::max(I, O))   // the largest of the three matrices
        return fail(FSDP_E_INVALID_ARG, "linear: a matrix of more than 2^60 elements");
    if (weight_layout != FSDP_WEIGHT_IN_OUT && weight_layout != FSDP_WEIGHT_OUT_IN)
        return fail(FSDP_E_INVALID_ARG, "unknown weight_layout");
    return FSDP_OK;
}

// Checks the workspace for a product and takes its room from it; products of a
// few rows use none.
int take_room(fsdp_compute* c, const fsdp::Product& p, int64_t out_features, fsdp::ProductRoom* r) {
    if (fsdp::few_rows(p)) return FSDP_OK;
    const int64_t copies = static_cast<int64_t>(
        fsdp::product_copy_bytes(p.a, p.a_trans ? p.K : p.M, p.a_trans ? p.M : p.K) +
        fsdp::product_copy_bytes(p.b, p.b_trans ? p.K : p.N, p.b_trans ? p.N : p.K));
    TRY(check_workspace(c, copies_offset(out_features) + copies));
    r->partials = reinterpret_cast<float*>(c->workspace());
    r->copies = c->workspace() + copies_offset(out_features);
    r->status = c->status();
    r->wait_ns = c->wait_ns;
    r->withhold = c->withhold_next;
    return FSDP_OK;
}

int run_product(fsdp_compute* c, const fsdp::Product& p, const fsdp::ProductRoom& r, cudaStream_t st, const char* what) {
    const cudaError_t e = fsdp::launch_product(p, r, c->sms, st);
    if (e != cudaSuccess) return cuda_fail(e, what);
    if (p.M > 0 && p.N > 0 && p.K > 0 && !fsdp::few_rows(p)) c->withhold_next = 0;   // it ran on staged tiles
    return FSDP_OK;
}

}  // namespace

extern "C" {

int fsdp_compute_create(int64_t workspace_bytes, const fsdp_allocator* alloc, fsdp_compute** out) {
    return entry([&]() -> int {
        if (out == nullptr) return fail(FSDP_E_INVALID_ARG, "out is null");
        *out = nullptr;
        if (workspace_bytes < 0) return fail(FSDP_E_INVALID_ARG, "workspace_bytes must be >= 0");
        if (alloc != nullptr && (alloc->alloc == nullptr || alloc->free == nullptr))
            return fail(FSDP_E_INVALID_ARG, "the allocator needs both alloc and free");
        int device = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
        if (e != cudaSuccess) return cuda_fail(e, "querying the device");
        fsdp_compute* c = new (std::nothrow) fsdp_compute;
        if (c == nullptr) return fail(FSDP_E_OOM, "out of host memory");
        c->device = device;
        c->sms = std::min(sms, kSms);
        c->workspace_bytes = workspace_bytes;
        const size_t bytes = kHeader + static_cast<size_t>(workspace_bytes);
        if (alloc != nullptr) {
            c->allocator = *alloc;
            void* p = alloc->alloc(bytes, alloc->ctx);
            if (p == nullptr) {
                delete c;
                return fail(FSDP_E_OOM, "the caller's allocator returned NULL");
            }
            if (reinterpret_cast<uintptr_t>(p) & 255u) {
                alloc->free(p, alloc->ctx);
                delete c;
                return fail(FSDP_E_ALIGN, "the caller's allocator returned a block not aligned to 256 bytes");
            }
            c->block = static_cast<char*>(p);
        } else {
            void* p = nullptr;
            e = cudaMalloc(&p, bytes);
            if (e != cudaSuccess) {
                cudaGetLastError();
                delete c;
                return fail(e == cudaErrorMemoryAllocation ? FSDP_E_OOM : FSDP_E_CUDA,
                            std::string("cudaMalloc: ") + cudaGetErrorString(e));
            }
            c->block = static_cast<char*>(p);
        }
        e = cudaMemset(c->block, 0, kHeader);
        if (e == cudaSuccess) e = cudaDeviceSynchronize();
        if (e != cudaSuccess) {
            fsdp_compute_destroy(c);
            return cuda_fail(e, "clearing the status word");
        }
        *out = c;
        return FSDP_OK;
    });
}

int fsdp_compute_destroy(fsdp_compute* c) {
    return entry([&]() -> int {
        if (c == nullptr) return FSDP_OK;
        OnDevice dev(c->device);
        const cudaError_t e = cudaDeviceSynchronize();
        if (c->block != nullptr) {
            if (c->allocator.alloc != nullptr) c->allocator.free(c->block, c->allocator.ctx);
            else cudaFree(c->block);
        }
        delete c;
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "synchronising the device");
    });
}

int fsdp_compute_status(fsdp_compute* c, int32_t* flags, void* stream) {
    return entry([&]() -> int {
        if (c == nullptr) return fail(FSDP_E_INVALID_ARG, "compute handle is null");
        if (flags == nullptr) return fail(FSDP_E_INVALID_ARG, "flags is null");
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        int32_t v = 0;
        cudaError_t e = cudaMemcpyAsync(&v, c->status(), sizeof(v), cudaMemcpyDeviceToHost, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(c->status(), 0, sizeof(v), st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
        if (e != cudaSuccess) return cuda_fail(e, "reading the status word");
        *flags = v;
        if (v & FSDP_KSTATUS_DRAIN_TIMEOUT) c->broken = true;
        return FSDP_OK;
    });
}

int fsdp_compute_set_wait_limit(fsdp_compute* c, double seconds, int withhold_next) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (!(seconds >= 1e-6 && seconds <= 60.0)) return fail(FSDP_E_INVALID_ARG, "seconds must be in [1e-6, 60]");
        if (withhold_next < 0 || withhold_next > 1) return fail(FSDP_E_INVALID_ARG, "withhold_next must be 0 or 1");
        c->wait_ns = static_cast<unsigned long long>(seconds * 1e9);
        c->withhold_next = withhold_next;
        return FSDP_OK;
    });
}

int fsdp_layer_norm_workspace_bytes(int64_t rows, int64_t cols, int64_t* bytes) {
    return entry([&]() -> int {
        if (bytes == nullptr) return fail(FSDP_E_INVALID_ARG, "bytes is null");
        TRY(check_shape(rows, cols, "layer norm"));
        *bytes = norm_bytes(rows, cols);
        return FSDP_OK;
    });
}

int fsdp_linear_workspace_bytes(int64_t tokens, int64_t in_features, int64_t out_features, int weight_aligned,
                                int64_t* bytes) {
    return entry([&]() -> int {
        if (bytes == nullptr) return fail(FSDP_E_INVALID_ARG, "bytes is null");
        TRY(check_linear(tokens, in_features, out_features, FSDP_WEIGHT_IN_OUT));
        int64_t copies = copy_bytes(tokens, in_features) + copy_bytes(tokens, out_features);
        if (!weight_aligned)
            copies += std::max(copy_bytes(in_features, out_features), copy_bytes(out_features, in_features));
        *bytes = copies_offset(std::max(in_features, out_features)) + copies;
        return FSDP_OK;
    });
}

int fsdp_act8_layout(int64_t rows, int64_t cols, int64_t* data_ld, int64_t* exps_ld) {
    return entry([&]() -> int {
        TRY(check_shape(rows, cols, "act8"));
        if (data_ld) *data_ld = fsdp::act8_groups(cols) * fsdp::kGroup;
        if (exps_ld) *exps_ld = fsdp::act8_groups(cols);
        return FSDP_OK;
    });
}

int fsdp_layer_norm_forward(fsdp_compute* c, const fsdp_matrix* x, const void* gamma, const void* beta, int param_dtype,
                            double eps, const fsdp_matrix* y, float* mean, float* rstd, const fsdp_matrix* ckpt,
                            void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (x == nullptr) return fail(FSDP_E_INVALID_ARG, "x is null");
        fsdp::NormForward a{};
        a.rows = x->rows;
        a.cols = x->cols;
        TRY(check_shape(a.rows, a.cols, "layer norm"));
        TRY(take(x, "x", a.rows, a.cols, kFloats, &a.x));
        TRY(take(y, "y", a.rows, a.cols, kFloats, &a.y));
        TRY(take_optional(ckpt, "ckpt", a.rows, a.cols, kAct8, &a.ckpt));
        TRY(take_vector(gamma, "gamma", param_dtype));
        TRY(take_vector(beta, "beta", param_dtype));
        if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(FSDP_E_INVALID_ARG, "eps must be finite and >= 0");
        if (a.rows > 0) {
            TRY(take_vector(mean, "mean", FSDP_DTYPE_F32));
            TRY(take_vector(rstd, "rstd", FSDP_DTYPE_F32));
        }
        a.gamma = gamma;
        a.beta = beta;
        a.param_dtype = param_dtype;
        a.eps = static_cast<float>(eps);
        a.mean = mean;
        a.rstd = rstd;
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e = fsdp::launch_norm_forward(a, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "layer norm forward launch");
    });
}

int fsdp_layer_norm_backward(fsdp_compute* c, const fsdp_matrix* dy, const fsdp_matrix* x, const void* gamma,
                             int param_dtype, const float* mean, const float* rstd, const fsdp_matrix* add,
                             const fsdp_matrix* dx, void* dgamma, void* dbeta, int grad_dtype, int accumulate,
                             void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (dy == nullptr) return fail(FSDP_E_INVALID_ARG, "dy is null");
        fsdp::NormBackward a{};
        a.rows = dy->rows;
        a.cols = dy->cols;
        TRY(check_shape(a.rows, a.cols, "layer norm"));
        TRY(take(dy, "dy", a.rows, a.cols, kFloats, &a.dy));
        TRY(take(x, "x", a.rows, a.cols, kFloats | kAct8, &a.x));
        TRY(take_optional(add, "add", a.rows, a.cols, kFloats, &a.add));
        TRY(take(dx, "dx", a.rows, a.cols, kFloats, &a.dx));
        TRY(take_vector(gamma, "gamma", param_dtype));
        if (a.rows > 0) {
            TRY(take_vector(mean, "mean", FSDP_DTYPE_F32));
            TRY(take_vector(rstd, "rstd", FSDP_DTYPE_F32));
        }
        TRY(take_vector(dgamma, "dgamma", grad_dtype));
        TRY(take_vector(dbeta, "dbeta", grad_dtype));
        TRY(check_workspace(c, norm_bytes(a.rows, a.cols)));
        a.gamma = gamma;
        a.param_dtype = param_dtype;
        a.mean = mean;
        a.rstd = rstd;
        a.dgamma = dgamma;
        a.dbeta = dbeta;
        a.grad_dtype = grad_dtype;
        a.accumulate = accumulate != 0;
        a.partials = reinterpret_cast<float*>(c->workspace());
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e = fsdp::launch_norm_backward(a, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "layer norm backward launch");
    });
}

int fsdp_linear_forward(fsdp_compute* c, const fsdp_matrix* x, const fsdp_matrix* w, int weight_layout, const void* bias,
                        int bias_dtype, int activation, const fsdp_matrix* residual, const fsdp_matrix* preact,
                        const fsdp_matrix* y, void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (x == nullptr || y == nullptr) return fail(FSDP_E_INVALID_ARG, x == nullptr ? "x is null" : "y is null");
        const int64_t T = x->rows, I = x->cols, O = y->cols;
        TRY(check_linear(T, I, O, weight_layout));
        const bool io = weight_layout == FSDP_WEIGHT_IN_OUT;
        fsdp::Product p{};
        p.M = T;
        p.N = O;
        p.K = I;
        TRY(take(x, "x", T, I, kBf16, &p.a));
        TRY(take(w, "w", io ? I : O, io ? O : I, kBf16, &p.b));
        p.b_trans = io;
        if (bias != nullptr) TRY(take_vector(bias, "bias", bias_dtype));
        TRY(check_activation(activation));
        TRY(take_optional(residual, "residual", T, O, kFloats, &p.add));
        TRY(take_optional(preact, "preact", T, O, kFloats | kAct8, &p.pre));
        TRY(take(y, "y", T, O, kFloats, &p.out));
        p.bias = bias;
        p.bias_dtype = bias_dtype;
        p.act = activation;
        fsdp::ProductRoom room{};
        TRY(take_room(c, p, p.N, &room));
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        return run_product(c, p, room, static_cast<cudaStream_t>(stream), "linear forward launch");
    });
}

int fsdp_linear_grad_input(fsdp_compute* c, const fsdp_matrix* dy, const fsdp_matrix* w, int weight_layout,
                           int activation, const fsdp_matrix* preact, const fsdp_matrix* add, const fsdp_matrix* dx,
                           void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (dy == nullptr || dx == nullptr) return fail(FSDP_E_INVALID_ARG, dy == nullptr ? "dy is null" : "dx is null");
        const int64_t T = dy->rows, O = dy->cols, I = dx->cols;
        TRY(check_linear(T, I, O, weight_layout));
        const bool io = weight_layout == FSDP_WEIGHT_IN_OUT;
        fsdp::Product p{};
        p.M = T;
        p.N = I;
        p.K = O;
        TRY(take(dy, "dy", T, O, kBf16, &p.a));
        TRY(take(w, "w", io ? I : O, io ? O : I, kBf16, &p.b));
        p.b_trans = !io;
        TRY(check_activation(activation));
        p.act = activation;
        if (activation != FSDP_ACTIVATION_NONE) {
            TRY(take(preact, "preact", T, I, kFloats | kAct8, &p.pre));
            p.slope = 1;
        }
        TRY(take_optional(add, "add", T, I, kFloats, &p.add));
        TRY(take(dx, "dx", T, I, kFloats, &p.out));
        fsdp::ProductRoom room{};
        TRY(take_room(c, p, p.N, &room));
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        return run_product(c, p, room, static_cast<cudaStream_t>(stream), "linear input-gradient launch");
    });
}

int fsdp_linear_grad_weight(fsdp_compute* c, const fsdp_matrix* x, const fsdp_matrix* dy, int weight_layout,
                            const fsdp_matrix* dw, void* dbias, int accumulate, void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (x == nullptr || dy == nullptr || dw == nullptr)
            return fail(FSDP_E_INVALID_ARG, x == nullptr ? "x is null" : dy == nullptr ? "dy is null" : "dw is null");
        const int64_t T = dy->rows, O = dy->cols, I = x->cols;
        TRY(check_linear(T, I, O, weight_layout));
        const bool io = weight_layout == FSDP_WEIGHT_IN_OUT;
        fsdp::Product p{};
        Mat mx, mdy;
        TRY(take(x, "x", T, I, kBf16 | kAct8, &mx));
        TRY(take(dy, "dy", T, O, kBf16, &mdy));
        p.M = io ? I : O;
        p.N = io ? O : I;
        p.K = T;
        p.a = io ? mx : mdy;
        p.b = io ? mdy : mx;
        p.a_trans = p.b_trans = 1;
        TRY(take(dw, "dw", p.M, p.N, kFloats, &p.out));
        if (accumulate) p.add = p.out;
        if (dbias != nullptr) {
            TRY(take_vector(dbias, "dbias", dw->dtype));
        }
        fsdp::ProductRoom room{};
        TRY(take_room(c, p, O, &room));
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        TRY(run_product(c, p, room, st, "linear weight-gradient launch"));
        if (dbias != nullptr) {
            float* sums = reinterpret_cast<float*>(c->workspace() + fsdp::kPartialBytes);
            const cudaError_t e = fsdp::launch_column_sum(T, O, mdy, sums, dbias, dw->dtype,
                                        accumulate != 0, c->sms, st);
            if (e != cudaSuccess) return cuda_fail(e, "bias-gradient launch");
        }
        return FSDP_OK;
    });
}

int fsdp_act8_pack(fsdp_compute* c, const fsdp_matrix* x, const fsdp_matrix* ckpt, void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (x == nullptr) return fail(FSDP_E_INVALID_ARG, "x is null");
        Mat mx, mq;
        TRY(check_shape(x->rows, x->cols, "act8"));
        TRY(take(x, "x", x->rows, x->cols, kFloats, &mx));
        TRY(take(ckpt, "ckpt", x->rows, x->cols, kAct8, &mq));
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e = fsdp::launch_act8_pack(x->rows, x->cols, mx, mq, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "act8 pack launch");
    });
}

int fsdp_act8_unpack(fsdp_compute* c, const fsdp_matrix* ckpt, int activation, const fsdp_matrix* out, void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (ckpt == nullptr) return fail(FSDP_E_INVALID_ARG, "ckpt is null");
        Mat mq, mo;
        TRY(check_shape(ckpt->rows, ckpt->cols, "act8"));
        TRY(take(ckpt, "ckpt", ckpt->rows, ckpt->cols, kAct8, &mq));
        TRY(take(out, "out", ckpt->rows, ckpt->cols, kFloats, &mo));
        TRY(check_activation(activation));
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e =
            fsdp::launch_act8_unpack(ckpt->rows, ckpt->cols, mq, activation, mo, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "act8 unpack launch");
    });
}

}  // extern "C"
