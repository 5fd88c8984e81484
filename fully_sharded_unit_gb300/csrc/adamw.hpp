// AdamW's constants, the checks of its hyper-parameters, and its update of one element,
// as the unit's step and the step over many tensors both have them.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "fsdp_unit.h"

namespace fsdp {

// Records the calling thread's failure reason for fsdp_last_error (api.cu).
int record_error(int code, const std::string& why);

// fp32 constants of one AdamW step, formed on the host.
struct AdamWConsts {
    float decay;   // 1 - lr*wd
    float b1, c1;  // beta1, 1 - beta1
    float b2, c2;  // beta2, 1 - beta2
    float bc2;     // 1 - beta2^t
    float step;    // lr / (1 - beta1^t)
    float eps;
};

inline int check_hp(const fsdp_adamw_hp* hp) {
    if (hp == nullptr) return record_error(FSDP_E_INVALID_ARG, "hp is null");
    auto fin = [](double x) { return std::isfinite(x); };
    if (!fin(hp->lr) || !fin(hp->beta1) || !fin(hp->beta2) || !fin(hp->eps) || !fin(hp->weight_decay))
        return record_error(FSDP_E_INVALID_ARG, "AdamW hyper-parameters must be finite");
    if (hp->lr < 0 || hp->eps < 0 || hp->weight_decay < 0)
        return record_error(FSDP_E_INVALID_ARG, "lr, eps and weight_decay must be >= 0");
    if (!(hp->beta1 >= 0 && hp->beta1 < 1) || !(hp->beta2 >= 0 && hp->beta2 < 1))
        return record_error(FSDP_E_INVALID_ARG, "betas must be in [0, 1)");
    return FSDP_OK;
}

inline double adamw_bc1(const fsdp_adamw_hp& hp, int64_t t) { return 1.0 - std::pow(hp.beta1, static_cast<double>(t)); }

inline AdamWConsts adamw_consts(const fsdp_adamw_hp* hp, int64_t t) {
    const double bc1 = adamw_bc1(*hp, t);
    const double bc2 = 1.0 - std::pow(hp->beta2, static_cast<double>(t));
    AdamWConsts c;
    c.decay = static_cast<float>(1.0 - hp->lr * hp->weight_decay);
    c.b1 = static_cast<float>(hp->beta1);
    c.c1 = static_cast<float>(1.0 - hp->beta1);
    c.b2 = static_cast<float>(hp->beta2);
    c.c2 = static_cast<float>(1.0 - hp->beta2);
    c.bc2 = static_cast<float>(bc2);
    c.step = static_cast<float>(hp->lr / bc1);
    c.eps = static_cast<float>(hp->eps);
    return c;
}

struct AdamWScaled {
    float decay, step;
};
// decay and step of a tensor with scales of its own, as adamw_consts forms them.
// bc1: 1 - beta1^t, the same for all of a call's tensors.
inline AdamWScaled adamw_scaled(const fsdp_adamw_hp& hp, double bc1, double lr_scale, double decay_scale) {
    const double lr = hp.lr * lr_scale;
    return {static_cast<float>(1.0 - lr * (hp.weight_decay * decay_scale)), static_cast<float>(lr / bc1)};
}

#ifdef __CUDACC__
__device__ __forceinline__ void adamw_elem(float& p, float g, float& m, float& v,
                                           const AdamWConsts& c) {
    const float pd = __fmul_rn(p, c.decay);
    m = __fadd_rn(__fmul_rn(c.b1, m), __fmul_rn(c.c1, g));
    v = __fadd_rn(__fmul_rn(c.b2, v), __fmul_rn(c.c2, __fmul_rn(g, g)));
    const float denom = __fadd_rn(__fsqrt_rn(__fdiv_rn(v, c.bc2)), c.eps);
    p = __fsub_rn(pd, __fmul_rn(c.step, __fdiv_rn(m, denom)));
}
#endif

}  // namespace fsdp
