// C entry points of the operators at a training step's ends (declared in
// include/fsdp_unit.h).  Every argument is checked here, before anything is
// enqueued; the launchers in logprobs.cu, residual_norm.cu and adamw_tensors.cu take
// what passed.
#include <cmath>

#include "adamw.hpp"
#include "compute.hpp"
#include "entry.hpp"
#include "fsdp_unit.h"

using namespace fsdp;

namespace {

constexpr int64_t kMostVocab = int64_t(1) << 30;
constexpr int64_t kMostElements = int64_t(1) << 40;

int take_array(const void* p, const char* name, uintptr_t mask) {
    if (p == nullptr) return fail(FSDP_E_INVALID_ARG, std::string(name) + " is null");
    if (reinterpret_cast<uintptr_t>(p) & mask) return fail(FSDP_E_ALIGN, std::string(name) + " is not aligned to its element");
    return FSDP_OK;
}
int take_floats(const void* p, const char* name) { return take_array(p, name, 3); }

int unwanted(const void* p, const char* name, const char* without) {
    return p == nullptr ? FSDP_OK : fail(FSDP_E_INVALID_ARG, std::string(name) + " without " + without);
}

// What the three calls on logits share.
int take_logits(const fsdp_compute* c, const fsdp_matrix* logits, double scale, TokenLogprobs* a) {
    TRY(check_handle(c));
    if (logits == nullptr) return fail(FSDP_E_INVALID_ARG, "logits is null");
    a->rows = logits->rows;
    a->vocab = logits->cols;
    TRY(check_shape(a->rows, a->vocab, "token log probabilities"));
    if (a->vocab > kMostVocab) return fail(FSDP_E_INVALID_ARG, "vocab is at most 2^30");
    TRY(take(logits, "logits", a->rows, a->vocab, kFloats, &a->z));
    a->scale = static_cast<float>(scale);
    if (!(a->scale >= 1e-30f && a->scale <= 1e30f)) return fail(FSDP_E_INVALID_ARG, "scale must be in [1e-30, 1e30]");
    a->status = c->status();
    return FSDP_OK;
}

int take_tokens(const int64_t* tokens, TokenLogprobs* a) {
    if (a->rows > 0) TRY(take_array(tokens, "tokens", 7));
    a->tokens = tokens;
    return FSDP_OK;
}

// The gradients of what a row gives.
int take_weights(const float* dlogprob, const float* dentropy, TokenLogprobs* a) {
    if (a->rows > 0) {
        if (dlogprob == nullptr && dentropy == nullptr) return fail(FSDP_E_INVALID_ARG, "dlogprob and dentropy are null");
        if (dlogprob != nullptr) TRY(take_floats(dlogprob, "dlogprob"));
        if (dentropy != nullptr) TRY(take_floats(dentropy, "dentropy"));
    }
    a->dlogprob = dlogprob;
    a->dentropy = dentropy;
    return FSDP_OK;
}

int run(const fsdp_compute* c, const char* what, cudaError_t (*launch)(const TokenLogprobs&, int, cudaStream_t), const TokenLogprobs& a,
        void* stream) {
    OnDevice dev(c->device);
    if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
    const cudaError_t e = launch(a, c->sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FSDP_OK : cuda_fail(e, what);
}

// The vectors of a residual norm.
int take_params(const void* post, const void* gate, const void* gamma, const void* block, int dtype) {
    if (dtype != FSDP_DTYPE_F32 && dtype != FSDP_DTYPE_BF16)
        return fail(FSDP_E_INVALID_ARG, "param_dtype must be FSDP_DTYPE_F32 or FSDP_DTYPE_BF16");
    if (block == nullptr) {
        TRY(unwanted(post, "post_gamma", "block"));
        TRY(unwanted(gate, "gate", "block"));
    }
    if (post != nullptr) TRY(take_vector(post, "post_gamma", dtype));
    if (gate != nullptr) TRY(take_vector(gate, "gate", dtype));
    if (gamma != nullptr) TRY(take_vector(gamma, "gamma", dtype));
    return FSDP_OK;
}

int check_scale(double residual_scale) {
    if (!std::isfinite(static_cast<float>(residual_scale))) return fail(FSDP_E_INVALID_ARG, "residual_scale must be finite");
    return FSDP_OK;
}

int64_t residual_norm_bytes(int64_t rows, int64_t cols) { return residual_norm_blocks(rows, cols) * 2 * cols * 4; }

int check_state8(int kind, int64_t numel, const uint8_t* codes, const uint8_t* exps) {
    if (kind != FSDP_STATE8_SIGNED && kind != FSDP_STATE8_UNSIGNED) return fail(FSDP_E_INVALID_ARG, "unknown kind of 8-bit moments");
    if (numel < 0 || numel > kMostElements) return fail(FSDP_E_INVALID_ARG, "numel must be in [0, 2^40]");
    if (numel > 0 && (codes == nullptr || exps == nullptr)) return fail(FSDP_E_INVALID_ARG, codes == nullptr ? "codes is null" : "exps is null");
    return FSDP_OK;
}

int check_tensor(const fsdp_adamw_tensor& t, const fsdp_adamw_hp& hp, double bc1, int64_t number) {
    const auto refuse = [&](int code, const char* why) { return fail(code, "tensor " + std::to_string(number) + ": " + why); };
    if (t.numel < 0 || t.numel > kMostElements) return refuse(FSDP_E_INVALID_ARG, "numel must be in [0, 2^40]");
    if (t.grad_dtype != FSDP_DTYPE_F32 && t.grad_dtype != FSDP_DTYPE_BF16) return refuse(FSDP_E_INVALID_ARG, "grad_dtype must be FSDP_DTYPE_F32 or FSDP_DTYPE_BF16");
    if (t.moments != FSDP_MOMENTS_F32 && t.moments != FSDP_MOMENTS_8BIT) return refuse(FSDP_E_INVALID_ARG, "unknown moments");
    if (!(t.lr_scale >= 0) || !(t.decay_scale >= 0) || !std::isfinite(t.lr_scale) || !std::isfinite(t.decay_scale))
        return refuse(FSDP_E_INVALID_ARG, "lr_scale and decay_scale must be finite and >= 0");
    const AdamWScaled own = adamw_scaled(hp, bc1, t.lr_scale, t.decay_scale);
    if (!std::isfinite(own.decay) || !std::isfinite(own.step))
        return refuse(FSDP_E_INVALID_ARG, "the scaled learning rate or weight decay is not finite");
    if (t.numel == 0) return FSDP_OK;
    const bool eight = t.moments == FSDP_MOMENTS_8BIT;
    if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr ||
        (eight && (t.exp_avg_exps == nullptr || t.exp_avg_sq_exps == nullptr)))
        return refuse(FSDP_E_INVALID_ARG, "a pointer is null");
    const auto off = [](const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
    if (off(t.param, 3) || off(t.grad, t.grad_dtype == FSDP_DTYPE_F32 ? 3 : 1) || off(t.copy_bf16, 1) ||
        (!eight && (off(t.exp_avg, 3) || off(t.exp_avg_sq, 3))))
        return refuse(FSDP_E_ALIGN, "a pointer is not aligned to its element");
    return FSDP_OK;
}

}  // namespace

extern "C" {

int fsdp_token_logprobs_forward(fsdp_compute* c, const fsdp_matrix* logits, const int64_t* tokens, double scale, float* logprob,
                                float* entropy, float* stats, int top, int64_t* top_tokens, float* top_logprobs, void* stream) {
    return entry([&]() -> int {
        TokenLogprobs a{};
        TRY(take_logits(c, logits, scale, &a));
        if (top < 0 || top > kMostTop || top > a.vocab) return fail(FSDP_E_INVALID_ARG, "top must be in [0, 32] and at most vocab");
        if (a.rows > 0) {
            if ((tokens == nullptr) != (logprob == nullptr)) return fail(FSDP_E_INVALID_ARG, "tokens and logprob come together");
            if (tokens != nullptr) {
                TRY(take_tokens(tokens, &a));
                TRY(take_floats(logprob, "logprob"));
            }
            if (entropy != nullptr) TRY(take_floats(entropy, "entropy"));
            if (stats != nullptr) TRY(take_floats(stats, "stats"));
            if (top > 0) {
                TRY(take_array(top_tokens, "top_tokens", 7));
                TRY(take_floats(top_logprobs, "top_logprobs"));
            } else if (top_tokens != nullptr || top_logprobs != nullptr) {
                return fail(FSDP_E_INVALID_ARG, "top_tokens and top_logprobs need top > 0");
            }
        }
        a.logprob = logprob;
        a.entropy = entropy;
        a.stats = stats;
        a.top = top;
        a.top_tokens = top_tokens;
        a.top_logprobs = top_logprobs;
        return run(c, "token log probabilities launch", launch_token_logprobs, a, stream);
    });
}

int fsdp_token_logprobs_backward(fsdp_compute* c, const fsdp_matrix* logits, const int64_t* tokens, double scale, const float* stats,
                                 const float* entropy, const float* dlogprob, const float* dentropy, const fsdp_matrix* dlogits,
                                 void* stream) {
    return entry([&]() -> int {
        TokenLogprobs a{};
        TRY(take_logits(c, logits, scale, &a));
        TRY(take(dlogits, "dlogits", a.rows, a.vocab, kFloats, &a.dz));
        TRY(take_weights(dlogprob, dentropy, &a));
        if (dlogprob != nullptr) TRY(take_tokens(tokens, &a));
        if (a.rows > 0) {
            TRY(take_floats(stats, "stats"));
            if (dentropy != nullptr) TRY(take_floats(entropy, "entropy"));
        }
        a.stats = const_cast<float*>(stats);         // read only
        a.entropy = dentropy != nullptr ? const_cast<float*>(entropy) : nullptr;
        return run(c, "logits' gradient launch", launch_token_logprobs_backward, a, stream);
    });
}

int fsdp_token_logprobs_loss(fsdp_compute* c, const fsdp_matrix* logits, const int64_t* tokens, double scale, const float* dlogprob,
                             const float* dentropy, float* logprob, float* entropy, float* stats, const fsdp_matrix* dlogits,
                             void* stream) {
    return entry([&]() -> int {
        TokenLogprobs a{};
        TRY(take_logits(c, logits, scale, &a));
        TRY(take(dlogits, "dlogits", a.rows, a.vocab, kFloats, &a.dz));
        TRY(take_weights(dlogprob, dentropy, &a));
        TRY(take_tokens(tokens, &a));
        if (a.rows > 0) {
            TRY(take_floats(logprob, "logprob"));
            if (entropy != nullptr) TRY(take_floats(entropy, "entropy"));
            if (stats != nullptr) TRY(take_floats(stats, "stats"));
        }
        a.logprob = logprob;
        a.entropy = entropy;
        a.stats = stats;
        return run(c, "token log probabilities launch", launch_token_logprobs, a, stream);
    });
}

int fsdp_residual_norm_workspace_bytes(int64_t rows, int64_t cols, int64_t* bytes) {
    return entry([&]() -> int {
        if (bytes == nullptr) return fail(FSDP_E_INVALID_ARG, "bytes is null");
        TRY(check_shape(rows, cols, "residual norm"));
        *bytes = residual_norm_bytes(rows, cols);
        return FSDP_OK;
    });
}

int fsdp_residual_norm_forward(fsdp_compute* c, const fsdp_matrix* residual, const fsdp_matrix* block, const void* post_gamma,
                               const void* gate, const void* gamma, int param_dtype, double residual_scale, double eps,
                               const fsdp_matrix* out, const fsdp_matrix* y, float* post_rstd, float* rstd, void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (residual == nullptr) return fail(FSDP_E_INVALID_ARG, "residual is null");
        ResidualNorm a{};
        a.rows = residual->rows;
        a.cols = residual->cols;
        TRY(check_shape(a.rows, a.cols, "residual norm"));
        TRY(take(residual, "residual", a.rows, a.cols, kFloats, &a.h));
        TRY(take_optional(block, "block", a.rows, a.cols, kFloats, &a.o));
        TRY(take(out, "out", a.rows, a.cols, kFloats, &a.out));
        TRY(take_optional(y, "y", a.rows, a.cols, kFloats, &a.y));
        TRY(take_params(post_gamma, gate, gamma, block, param_dtype));
        TRY(check_scale(residual_scale));
        if (!(eps >= 0.0) || !std::isfinite(static_cast<float>(eps))) return fail(FSDP_E_INVALID_ARG, "eps must be finite and >= 0");
        if ((gamma == nullptr) != (y == nullptr)) return fail(FSDP_E_INVALID_ARG, "gamma and y come together");
        if (a.rows > 0) {
            if (post_gamma != nullptr) TRY(take_floats(post_rstd, "post_rstd"));
            if (gamma != nullptr) TRY(take_floats(rstd, "rstd"));
        }
        if (post_gamma == nullptr) TRY(unwanted(post_rstd, "post_rstd", "post_gamma"));
        if (gamma == nullptr) TRY(unwanted(rstd, "rstd", "gamma"));
        a.post = post_gamma;
        a.gate = gate;
        a.gamma = gamma;
        a.param_dtype = param_dtype;
        a.alpha = static_cast<float>(residual_scale);
        a.eps = static_cast<float>(eps);
        a.post_rstd = post_rstd;
        a.rstd = rstd;
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e = launch_residual_norm_forward(a, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "residual norm forward launch");
    });
}

int fsdp_residual_norm_backward(fsdp_compute* c, const fsdp_matrix* dy, const fsdp_matrix* dout, const fsdp_matrix* out,
                                const fsdp_matrix* block, const void* post_gamma, const void* gate, const void* gamma, int param_dtype,
                                double residual_scale, const float* post_rstd, const float* rstd, const fsdp_matrix* dresidual,
                                const fsdp_matrix* dblock, void* dgamma, void* dpost_gamma, void* dgate, int grad_dtype, int accumulate,
                                void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (dresidual == nullptr) return fail(FSDP_E_INVALID_ARG, "dresidual is null");
        ResidualNormGrad a{};
        a.rows = dresidual->rows;
        a.cols = dresidual->cols;
        TRY(check_shape(a.rows, a.cols, "residual norm"));
        TRY(take(dresidual, "dresidual", a.rows, a.cols, kFloats, &a.dh));
        if (dy == nullptr && dout == nullptr) return fail(FSDP_E_INVALID_ARG, "dy and dout are null");
        TRY(take_optional(dy, "dy", a.rows, a.cols, kFloats, &a.dy));
        TRY(take_optional(dout, "dout", a.rows, a.cols, kFloats, &a.dout));
        TRY(take_optional(block, "block", a.rows, a.cols, kFloats, &a.o));
        TRY(take_optional(dblock, "dblock", a.rows, a.cols, kFloats, &a.dblock));
        TRY(take_params(post_gamma, gate, gamma, block, param_dtype));
        TRY(check_scale(residual_scale));
        const auto together = [](const void* p, const void* q) { return (p == nullptr) == (q == nullptr); };
        if (!together(gamma, dy)) return fail(FSDP_E_INVALID_ARG, "gamma and dy come together");
        if (!together(block, dblock)) return fail(FSDP_E_INVALID_ARG, "block and dblock come together");
        if (!together(gamma, dgamma) || !together(post_gamma, dpost_gamma) || !together(gate, dgate))
            return fail(FSDP_E_INVALID_ARG, "each of gamma, post_gamma and gate comes with its gradient");
        if (dgamma != nullptr) {
            TRY(take(out, "out", a.rows, a.cols, kFloats, &a.out));   // xh is made of it
            if (a.rows > 0) TRY(take_floats(rstd, "rstd"));
            TRY(take_vector(dgamma, "dgamma", grad_dtype));
        }
        if (dpost_gamma != nullptr) {
            if (a.rows > 0) TRY(take_floats(post_rstd, "post_rstd"));
            TRY(take_vector(dpost_gamma, "dpost_gamma", grad_dtype));
        }
        if (dgate != nullptr) TRY(take_vector(dgate, "dgate", grad_dtype));
        TRY(check_workspace(c, residual_norm_bytes(a.rows, a.cols)));
        a.post = post_gamma;
        a.gate = gate;
        a.gamma = gamma;
        a.param_dtype = param_dtype;
        a.alpha = static_cast<float>(residual_scale);
        a.post_rstd = post_rstd;
        a.rstd = rstd;
        a.dgamma = dgamma;
        a.dpost = dpost_gamma;
        a.dgate = dgate;
        a.grad_dtype = grad_dtype;
        a.accumulate = accumulate != 0;
        a.partials = reinterpret_cast<float*>(c->workspace());
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e = launch_residual_norm_backward(a, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "residual norm backward launch");
    });
}

int fsdp_state8_pack(fsdp_compute* c, int kind, const float* x, int64_t numel, uint8_t* codes, uint8_t* exps, void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        TRY(check_state8(kind, numel, codes, exps));
        if (numel > 0) TRY(take_floats(x, "x"));
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e = launch_state8_pack(kind, x, numel, codes, exps, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "state8 pack launch");
    });
}

int fsdp_state8_unpack(fsdp_compute* c, int kind, const uint8_t* codes, const uint8_t* exps, int64_t numel, void* out, int out_dtype,
                       void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        TRY(check_state8(kind, numel, codes, exps));
        if (out_dtype != FSDP_DTYPE_F32 && out_dtype != FSDP_DTYPE_BF16)
            return fail(FSDP_E_INVALID_ARG, "out_dtype must be FSDP_DTYPE_F32 or FSDP_DTYPE_BF16");
        if (numel > 0) TRY(take_vector(out, "out", out_dtype));
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e = launch_state8_unpack(kind, codes, exps, numel, out, out_dtype, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "state8 unpack launch");
    });
}

int fsdp_adamw_tensors(fsdp_compute* c, const fsdp_adamw_tensor* tensors, int64_t count, const fsdp_adamw_hp* hp, int64_t step,
                       uint64_t seed, const float* grad_scale_dev, const int32_t* skip_dev, void* stream) {
    return entry([&]() -> int {
        TRY(check_handle(c));
        if (count < 0) return fail(FSDP_E_INVALID_ARG, "count must be >= 0");
        if (count > 0 && tensors == nullptr) return fail(FSDP_E_INVALID_ARG, "tensors is null");
        TRY(check_hp(hp));
        if (step < 1) return fail(FSDP_E_INVALID_ARG, "step must be >= 1");
        const double bc1 = adamw_bc1(*hp, step);
        for (int64_t j = 0; j < count; ++j) TRY(check_tensor(tensors[j], *hp, bc1, j));
        if (grad_scale_dev != nullptr) TRY(take_floats(grad_scale_dev, "grad_scale_dev"));
        if (skip_dev != nullptr) TRY(take_array(skip_dev, "skip_dev", 3));
        OnDevice dev(c->device);
        if (!dev.ok()) return fail(FSDP_E_CUDA, "cannot select the handle's device");
        const cudaError_t e = launch_adamw_tensors(tensors, count, *hp, step, seed, grad_scale_dev, skip_dev, c->sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "AdamW launch");
    });
}

}  // extern "C"
