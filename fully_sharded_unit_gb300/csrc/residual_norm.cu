// The norms before and after a block with its gate and residual scale, forward and
// backward.
#include <algorithm>

#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// Sums over the block, for every thread.  `red` is free again after the next barrier.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*red)[32]) {
    const int w = threadIdx.x >> 5, n = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = warp_sum(v[i]);
        if ((threadIdx.x & 31) == 0) red[i][w] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.0f;
        for (int j = 0; j < n; ++j) v[i] += red[i][j];
    }
}

// Eight elements of a row from column c on, those inside the row; 0 past its end, and
// `otherwise` where there is no matrix or vector.
__device__ __forceinline__ void load_any(const void* p, int dtype, int64_t at, int in, float otherwise, float* v) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = otherwise;
    } else {
        load_chunks_any<1>(p, dtype, at, &in, 0, reinterpret_cast<float(*)[8]>(v));
    }
}

// ---- any rows ----
//
// A row to a block, in chunks of eight columns that start anywhere, read again (from L1
// or L2) for each of the passes that a row takes.

__device__ __forceinline__ void residual_chunk(const ResidualNorm& a, int64_t row, int64_t c, int in, float post_rstd, float* s) {
    float h[8], o[8], p[8], g[8];
    load_any(a.h.p, a.h.dtype, row * a.h.ld + c, in, 0.0f, h);
    load_any(a.o.p, a.o.dtype, row * a.o.ld + c, in, 0.0f, o);
    load_any(a.post, a.param_dtype, c, in, 1.0f, p);
    load_any(a.gate, a.param_dtype, c, in, 1.0f, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = fmaf(a.alpha, h[j], o[j] * post_rstd * p[j] * g[j]);
}

__global__ void __launch_bounds__(512) residual_norm_any_kernel(const ResidualNorm a) {
    __shared__ float red[2][1][32];
    starts_early();
    after_previous();
    const float n = static_cast<float>(a.cols);
    const int64_t chunks = (a.cols + 7) / 8;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float post_rstd = 1.0f;
        if (a.post != nullptr) {
            float ss[1] = {0.0f};
            for (int64_t q = threadIdx.x; q < chunks; q += blockDim.x) {
                float o[8];
                load_any(a.o.p, a.o.dtype, row * a.o.ld + q * 8, inside8(q * 8, a.cols), 0.0f, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss[0] = fmaf(o[j], o[j], ss[0]);
            }
            block_sums(ss, red[0]);
            post_rstd = 1.0f / sqrtf(ss[0] / n + a.eps);
            if (threadIdx.x == 0) a.post_rstd[row] = post_rstd;
        }
        float ss[1] = {0.0f};
        for (int64_t first = 0; first < chunks; first += blockDim.x) {   // whole warps store together
            const int64_t c = (first + threadIdx.x) * 8;
            const int in = inside8(c, a.cols);
            float s[8];
            residual_chunk(a, row, c, in, post_rstd, s);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < in) ss[0] = fmaf(s[j], s[j], ss[0]);
            store_chunk_any(a.out.p, a.out.dtype, row * a.out.ld + c, in, s);
        }
        if (a.y.p != nullptr) {
            block_sums(ss, red[1]);
            const float rstd = 1.0f / sqrtf(ss[0] / n + a.eps);
            if (threadIdx.x == 0) a.rstd[row] = rstd;
            for (int64_t first = 0; first < chunks; first += blockDim.x) {
                const int64_t c = (first + threadIdx.x) * 8;
                const int in = inside8(c, a.cols);
                float s[8], g[8];
                residual_chunk(a, row, c, in, post_rstd, s);
                load_any(a.gamma, a.param_dtype, c, in, 1.0f, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = s[j] * rstd * g[j];
                store_chunk_any(a.y.p, a.y.dtype, row * a.y.ld + c, in, s);
            }
        }
        __syncthreads();
    }
}

// A chunk of the backward pass.
struct GradChunk {
    float dy[8], xh[8], g[8], k[8], u[8], t[8];   // k: gate * post_gamma; t: dout so far
};
__device__ __forceinline__ void grad_chunk(const ResidualNormGrad& a, int64_t row, int64_t c, int in, float rstd, float post_rstd,
                                           GradChunk& v) {
    load_any(a.dy.p, a.dy.dtype, row * a.dy.ld + c, in, 0.0f, v.dy);
    load_any(a.dout.p, a.dout.dtype, row * a.dout.ld + c, in, 0.0f, v.t);
    load_any(a.o.p, a.o.dtype, row * a.o.ld + c, in, 0.0f, v.u);
    load_any(a.dy.p != nullptr ? a.out.p : nullptr, a.out.dtype, row * a.out.ld + c, in, 0.0f, v.xh);
    float w[8];
    load_any(a.post, a.param_dtype, c, in, 1.0f, v.k);
    load_any(a.gate, a.param_dtype, c, in, 1.0f, w);
    load_any(a.gamma, a.param_dtype, c, in, 1.0f, v.g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v.k[j] *= w[j];
        v.u[j] *= post_rstd;
        v.xh[j] *= rstd;
        v.g[j] *= v.dy[j];
    }
}

__global__ void __launch_bounds__(512) residual_norm_any_backward_kernel(const ResidualNormGrad a) {
    __shared__ float red[3][32];
    starts_early();
    after_previous();
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    const int64_t chunks = (a.cols + 7) / 8;
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.dy.p != nullptr ? a.rstd[row] : 0.0f, post_rstd = a.post != nullptr ? a.post_rstd[row] : 1.0f;
        // with e = t k and t = dout + rstd (g - xh c1), sum(e u) is linear in c1
        float s[3] = {0.0f, 0.0f, 0.0f};
        for (int64_t q = threadIdx.x; q < chunks; q += blockDim.x) {
            GradChunk v;
            grad_chunk(a, row, q * 8, inside8(q * 8, a.cols), rstd, post_rstd, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float ku = v.k[j] * v.u[j];
                s[0] = fmaf(v.g[j], v.xh[j], s[0]);
                s[1] = fmaf(ku, fmaf(rstd, v.g[j], v.t[j]), s[1]);
                s[2] = fmaf(ku, v.xh[j], s[2]);
            }
        }
        block_sums(s, red);
        const float c1 = s[0] * inv_n, c2 = a.post != nullptr ? (s[1] - rstd * c1 * s[2]) * inv_n : 0.0f;
        const bool fresh = row == blockIdx.x;
        for (int64_t first = 0; first < chunks; first += blockDim.x) {
            const int64_t c = (first + threadIdx.x) * 8;
            const int in = inside8(c, a.cols);
            GradChunk v;
            grad_chunk(a, row, c, in, rstd, post_rstd, v);
            float dh[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = fmaf(rstd, fmaf(-v.xh[j], c1, v.g[j]), v.t[j]);
                dh[j] = a.alpha * t;
                v.dy[j] *= v.xh[j];
                v.t[j] = t * v.u[j];
                v.u[j] = post_rstd * fmaf(-v.u[j], c2, t * v.k[j]);
                if (j < in) {
                    if (a.dgamma != nullptr) part[c + j] = (fresh ? 0.0f : part[c + j]) + v.dy[j];
                    if (a.o.p != nullptr) part[a.cols + c + j] = (fresh ? 0.0f : part[a.cols + c + j]) + v.t[j];
                }
            }
            store_chunk_any(a.dh.p, a.dh.dtype, row * a.dh.ld + c, in, dh);
            if (a.dblock.p != nullptr) store_chunk_any(a.dblock.p, a.dblock.dtype, row * a.dblock.ld + c, in, v.u);
        }
        __syncthreads();
    }
}

// The columns' sums over the blocks, in their order: dgamma from the first half of the
// partial rows, dpost_gamma and dgate from the second.  16 columns across and 16
// slices of the blocks down.
__global__ void __launch_bounds__(256) residual_norm_sums_kernel(const ResidualNormGrad a, int64_t count) {
    __shared__ float part[16][17];
    starts_early();
    after_previous();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 16 + tx;
    const float* p = a.partials + blockIdx.y * a.cols + c;
    float s = 0.0f;
    if (c < a.cols) {
#pragma unroll 10
        for (int64_t i = ty; i < count; i += 16) s += __ldcg(p + i * 2 * a.cols);
    }
    part[ty][tx] = s;
    __syncthreads();
    if (ty != 0 || c >= a.cols) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += part[i][tx];
    const auto put = [&](void* out, const void* by) {
        if (out == nullptr) return;
        float v = by != nullptr ? s * load1(by, a.param_dtype, c) : s;
        if (a.accumulate) v += load1(out, a.grad_dtype, c);
        store1(out, a.grad_dtype, c, v);
    };
    if (blockIdx.y == 0) {
        put(a.dgamma, nullptr);
    } else {
        put(a.dpost, a.gate);
        put(a.dgate, a.post);
    }
}

constexpr int kSms = 152;

}  // namespace

int64_t residual_norm_blocks(int64_t rows, int64_t) { return std::min<int64_t>(rows, 2 * kSms); }

cudaError_t launch_residual_norm_forward(const ResidualNorm& a, int sms, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    return launch_early(residual_norm_any_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t(1) << 30))), 512, 0, st, a);
}

cudaError_t launch_residual_norm_backward(const ResidualNormGrad& a, int sms, cudaStream_t st) {
    const int64_t blocks = residual_norm_blocks(a.rows, a.cols);
    if (a.rows > 0) {
        const cudaError_t e = launch_early(residual_norm_any_backward_kernel, dim3(static_cast<unsigned>(blocks)), 512, 0, st, a);
        if (e != cudaSuccess) return e;
    }
    if (a.dgamma == nullptr && a.dpost == nullptr && a.dgate == nullptr) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>((a.cols + 15) / 16), 2);
    return launch_early(residual_norm_sums_kernel, grid, 256, 0, st, a, blocks);
}

}  // namespace fsdp
