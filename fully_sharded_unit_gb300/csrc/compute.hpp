// Launchers of the block operators (layer norm, linear layer, 8-bit activation
// checkpoints) and of those at a step's ends (log probabilities, residual norm, AdamW over
// tensors).  Every launcher enqueues on `st` only and returns the launch
// status; arguments are checked by the C entry points in compute.cu and compute_step.cu.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "fsdp_unit.h"

namespace fsdp {

// Block counts are planned for this many SMs at most, so that the workspace
// can be told without a device.
constexpr int kSms = 152;

// A matrix as the kernels see it: element (r, c) at p + (r*ld + c) elements.
// ACT8: p is the int8 payload, e the exponent bytes, eld their row stride.
struct Mat {
    void* p;
    uint8_t* e;
    int64_t ld;
    int64_t eld;
    int dtype;   // FSDP_DTYPE_*
};

// Every kernel of the block operators is launched so that its start may overlap
// the end of the kernel before it (programmatic stream serialization): it lets
// the kernel after it start early (starts_early), and touches memory only
// after everything before it in the stream is complete (after_previous).  Such a
// kernel's lifetime covers the end of the kernel that writes its inputs, so its
// loads are ordinary ones: the non-coherent path (__ldg, ld.global.nc, const
// __restrict__ parameters) is for data that nobody writes while the kernel lives,
// and a line it left in an SM's cache may be older than the wait.
template <typename... Params, typename... Args>
cudaError_t launch_early_clusters(void (*kernel)(Params...), dim3 grid, int threads, size_t shared, int cluster, cudaStream_t st,
                                  const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = shared;
    cfg.stream = st;
    cudaLaunchAttribute attrs[2]{};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t shared, cudaStream_t st, const Args&... args) {
    return launch_early_clusters(kernel, grid, threads, shared, 1, st, args...);
}

// The value of f() for the current device, computed once for each device (a
// kernel's attributes belong to a device).  Every call site's f is a type of its
// own; two threads that come first together both compute the same value.
template <typename F>
int once_per_device(F f) {
    static std::atomic<int> values[64] = {};   // value + 1
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= 64) return f();
    int v = values[device].load(std::memory_order_acquire);
    if (v == 0) {
        v = f() + 1;
        values[device].store(v, std::memory_order_release);
    }
    return v - 1;
}

constexpr int kGroup = 32;   // elements that share an exponent in an ACT8 matrix

inline int64_t act8_groups(int64_t cols) { return (cols + kGroup - 1) / kGroup; }

// Rows of m start on boundaries of `to` bytes (16: vector accesses of 8 elements).
inline bool rows_aligned(const Mat& m, uintptr_t to = 16) {
    const uintptr_t esz = m.dtype == 0 ? 4 : m.dtype == 1 ? 2 : 1;
    return ((reinterpret_cast<uintptr_t>(m.p) | static_cast<uintptr_t>(m.ld) * esz) & (to - 1)) == 0;
}

// ---- layer norm (norm.cu) ----
struct NormForward {
    int64_t rows, cols;
    Mat x, y, ckpt;             // ckpt.p null: none
    const void *gamma, *beta;
    int param_dtype;
    float eps;
    float *mean, *rstd;
};
cudaError_t launch_norm_forward(const NormForward& a, int sms, cudaStream_t st);

struct NormBackward {
    int64_t rows, cols;
    Mat dy, x, add, dx;         // add.p null: none
    const void* gamma;
    int param_dtype;
    const float *mean, *rstd;
    void *dgamma, *dbeta;
    int grad_dtype, accumulate;
    float* partials;            // workspace: a row of 2 x cols floats for each of up to min(rows, sms) blocks
};
cudaError_t launch_norm_backward(const NormBackward& a, int sms, cudaStream_t st);

// out[c] (+)= sum over p of partials[p*stride + c], in the order of p.
cudaError_t launch_sum_partials(const float* partials, int64_t count, int64_t stride, int64_t cols, void* out,
                                int out_dtype, int accumulate, cudaStream_t st);

// ---- 8-bit checkpoints (act8.cu) ----
cudaError_t launch_act8_pack(int64_t rows, int64_t cols, const Mat& x, const Mat& q, int sms, cudaStream_t st);
cudaError_t launch_act8_unpack(int64_t rows, int64_t cols, const Mat& q, int activation, const Mat& out, int sms,
                               cudaStream_t st);

// ---- linear layer (linear.cu) ----
// C[m, n] = sum_k A(m, k) B(n, k) followed by, per element,
//   v = c + bias[n];  forward (slope == 0): store v to pre, v = act(v)
//                     slope == 1: v = c * act'(pre[m, n])
//   v += add[m, n];  store v to out.
struct Product {
    int64_t M, N, K;
    Mat a, b;                   // a: M x K (a_trans 0) or K x M (a_trans 1); b: N x K or K x N
    int a_trans, b_trans;
    const void* bias;
    int bias_dtype;
    int act, slope;
    Mat pre, add, out;          // p null: none
};

// What a product takes from the handle.
constexpr int kMaxClusters = 76;                                  // pairs of SMs
constexpr int64_t kPartialBytes = int64_t(kMaxClusters) * 256 * 256 * 4;
struct ProductRoom {
    float* partials;            // kPartialBytes: sums of tiles that several clusters share
    char* copies;               // product_copy_bytes() of both operands
    int32_t* status;            // FSDP_KSTATUS_* bits
    unsigned long long wait_ns; // bound of every wait
    int withhold;               // one-shot test of the give-up path
};
// Clusters of two CTAs that run at once (0: the kernel cannot run here).
int product_clusters(int sms);
// Bytes of the aligned bf16 copy that an operand needs (0: it is read in place).
size_t product_copy_bytes(const Mat& m, int64_t rows, int64_t cols);
cudaError_t launch_product(const Product& p, const ProductRoom& room, int sms, cudaStream_t st);

// Products of at most kFewRows rows (few.cu): bound by reading B, which passes
// once through registers; no workspace, any alignment.
constexpr int kFewRows = 8;
inline bool few_rows(const Product& p) {
    return p.M <= kFewRows && !p.a_trans && p.a.dtype == 1 && p.b.dtype == 1;   // both BF16
}
cudaError_t launch_few_rows(const Product& p, int sms, cudaStream_t st);

// Column sums of dy (rows x cols, bf16) over its rows, through `partials`
// (column_sum_partials() x cols floats).
int64_t column_sum_partials(int64_t rows, int64_t cols, int sms);
cudaError_t launch_column_sum(int64_t rows, int64_t cols, const Mat& dy, float* partials, void* out, int out_dtype,
                              int accumulate, int sms, cudaStream_t st);

// ---- log probabilities of tokens (logprobs.cu) ----
constexpr int kMostTop = 32;   // alternatives of a row
struct TokenLogprobs {
    int64_t rows, vocab;
    Mat z;
    const int64_t* tokens;          // null: none given
    float scale;
    float *logprob, *entropy, *stats;   // null: not wanted (backward: stats and entropy are read)
    int top;
    int64_t* top_tokens;
    float* top_logprobs;
    Mat dz;                         // p null: no gradient
    const float *dlogprob, *dentropy;   // null: zeros
    int32_t* status;                // FSDP_KSTATUS_* bits
};
// Everything but the gradient; with dz, the gradient behind it.
cudaError_t launch_token_logprobs(const TokenLogprobs& a, int sms, cudaStream_t st);
// The gradient alone, from stats (and entropy).
cudaError_t launch_token_logprobs_backward(const TokenLogprobs& a, int sms, cudaStream_t st);

// ---- residual norm (residual_norm.cu) ----
struct ResidualNorm {
    int64_t rows, cols;
    Mat h, o, out, y;               // o.p, y.p null: none
    const void *post, *gate, *gamma;
    int param_dtype;
    float alpha, eps;
    float *post_rstd, *rstd;
};
cudaError_t launch_residual_norm_forward(const ResidualNorm& a, int sms, cudaStream_t st);

struct ResidualNormGrad {
    int64_t rows, cols;
    Mat dy, dout, out, o, dh, dblock;   // dy.p, dout.p, o.p null: none
    const void *post, *gate, *gamma;
    int param_dtype;
    float alpha;
    const float *post_rstd, *rstd;
    void *dgamma, *dpost, *dgate;
    int grad_dtype, accumulate;
    float* partials;                // workspace: a row of 2 x cols floats a block
};
// Blocks that sums over rows are split over, at most (the workspace's rows).
int64_t residual_norm_blocks(int64_t rows, int64_t cols);
cudaError_t launch_residual_norm_backward(const ResidualNormGrad& a, int sms, cudaStream_t st);

// ---- AdamW over many tensors, 8-bit moments (adamw_tensors.cu) ----
cudaError_t launch_state8_pack(int kind, const float* x, int64_t n, uint8_t* codes, uint8_t* exps, int sms, cudaStream_t st);
cudaError_t launch_state8_unpack(int kind, const uint8_t* codes, const uint8_t* exps, int64_t n, void* out, int out_dtype,
                                 int sms, cudaStream_t st);
cudaError_t launch_adamw_tensors(const fsdp_adamw_tensor* tensors, int64_t count, const fsdp_adamw_hp& hp, int64_t step,
                                 uint64_t seed, const float* grad_scale, const int32_t* skip, int sms, cudaStream_t st);

}  // namespace fsdp
