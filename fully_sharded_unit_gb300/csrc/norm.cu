// Layer norm, forward and backward.  Both are bound by DRAM: the forward reads
// a row once into registers (two-pass mean and variance there) and writes y;
// the backward reads dy and x once, keeps each thread's columns of dgamma and
// dbeta in registers over all the rows its block walks, and a second small
// kernel joins the blocks' partial sums in a fixed order.
#include <algorithm>

#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Sum over the block; every thread gets it.  `red` holds 32 floats and is free
// again after the next barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    const int w = threadIdx.x >> 5, n = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s += red[i];
    return s;
}

// One row to a warp (WARP) or to a block; chunk k of a thread holds the V
// columns from (t + k * threads) * V.
template <int V, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024) norm_forward_kernel(NormForward a) {
    __shared__ float red[2][32];
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int threads = WARP ? 32 : blockDim.x;
    const int64_t first = WARP ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t stride = WARP ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x;
    const float n = static_cast<float>(a.cols);
    for (int64_t row = first; row < a.rows; row += stride) {
        float v[NV][V];
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = static_cast<int64_t>(t + k * threads) * V;
            if (c < a.cols) {
                loadv<V>(a.x.p, a.x.dtype, row * a.x.ld + c, v[k]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] = 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) s += v[k][j];
        const float mean = (WARP ? warp_sum(s) : block_sum(s, red[0])) / n;
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (static_cast<int64_t>(t + k * threads) * V < a.cols) {
#pragma unroll
                for (int j = 0; j < V; ++j) ss = fmaf(v[k][j] - mean, v[k][j] - mean, ss);
            }
        }
        const float var = (WARP ? warp_sum(ss) : block_sum(ss, red[1])) / n;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (t == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = static_cast<int64_t>(t + k * threads) * V;
            if (a.ckpt.p != nullptr) {
                const uint32_t byte = act8_group_byte<V>(v[k]);
                if (c < a.ckpt.ld) {
                    act8_writev<V>(static_cast<uint8_t*>(a.ckpt.p) + row * a.ckpt.ld, c, v[k], byte);
                    if ((t & (32 / V - 1)) == 0) a.ckpt.e[row * a.ckpt.eld + (c >> 5)] = static_cast<uint8_t>(byte);
                }
            }
            if (c < a.cols) {
                float g[V], b[V];
                loadv<V>(a.gamma, a.param_dtype, c, g);
                loadv<V>(a.beta, a.param_dtype, c, b);
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] = fmaf((v[k][j] - mean) * rstd, g[j], b[j]);
                storev<V>(a.y.p, a.y.dtype, row * a.y.ld + c, v[k]);
            }
        }
        if (!WARP) __syncthreads();
    }
}

// Rows too long for registers: three passes, the later ones from L2.
__global__ void __launch_bounds__(1024) norm_forward_wide_kernel(NormForward a) {
    __shared__ float red[2][32];
    const float n = static_cast<float>(a.cols);
    const int64_t ceil32 = (a.cols + 31) / 32 * 32;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) s += load1(a.x.p, a.x.dtype, row * a.x.ld + c);
        const float mean = block_sum(s, red[0]) / n;
        float ss = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float d = load1(a.x.p, a.x.dtype, row * a.x.ld + c) - mean;
            ss = fmaf(d, d, ss);
        }
        const float rstd = 1.0f / sqrtf(block_sum(ss, red[1]) / n + a.eps);
        if (threadIdx.x == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        for (int64_t c = threadIdx.x; c < ceil32; c += blockDim.x) {
            const bool on = c < a.cols;
            const float x = on ? load1(a.x.p, a.x.dtype, row * a.x.ld + c) : 0.0f;
            if (a.ckpt.p != nullptr) {   // ceil32 and the block are multiples of 32: whole warps
                const uint32_t byte = act8_group_byte<1>(&x);
                act8_writev<1>(static_cast<uint8_t*>(a.ckpt.p) + row * a.ckpt.ld, c, &x, byte);
                if ((threadIdx.x & 31) == 0) a.ckpt.e[row * a.ckpt.eld + (c >> 5)] = static_cast<uint8_t>(byte);
            }
            if (on)
                store1(a.y.p, a.y.dtype, row * a.y.ld + c,
                       fmaf((x - mean) * rstd, load1(a.gamma, a.param_dtype, c), load1(a.beta, a.param_dtype, c)));
        }
        __syncthreads();
    }
}

template <int V>
__device__ __forceinline__ void load_x(const Mat& x, int64_t row, int64_t c, float* v) {
    if (x.dtype == FSDP_DTYPE_ACT8)
        act8_readv<V>(static_cast<const uint8_t*>(x.p) + row * x.ld, x.e + row * x.eld, c, v);
    else
        loadv<V>(x.p, x.dtype, row * x.ld + c, v);
}

// A block holds G groups of `gt` threads (a multiple of 32); a group walks the
// rows group, group + groups, ...  Thread t of a group owns the columns of
// chunks t + k*gt, k < NV.
template <int V, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(NormBackward a, int gt) {
    extern __shared__ float comb[];          // 2 * cols floats where the block has several groups
    __shared__ float2 red[2][THREADS / 32];
    const int g = threadIdx.x / gt, t = threadIdx.x % gt, G = blockDim.x / gt;
    const int w0 = g * (gt >> 5), nw = gt >> 5;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    float dg[NV][V], db[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) dg[k][j] = db[k][j] = 0.0f;
    int flip = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * G + g; row < a.rows; row += static_cast<int64_t>(gridDim.x) * G) {
        float xh[NV][V], dy[NV][V];
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = static_cast<int64_t>(t + k * gt) * V;
            if (c < a.cols) {
                loadv<V>(a.dy.p, a.dy.dtype, row * a.dy.ld + c, dy[k]);
                load_x<V>(a.x, row, c, xh[k]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dy[k][j] = 0.0f;
                    xh[k][j] = mean;
                }
            }
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = static_cast<int64_t>(t + k * gt) * V;
            float gm[V];
            if (c < a.cols) {
                loadv<V>(a.gamma, a.param_dtype, c, gm);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) gm[j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xh[k][j] = (xh[k][j] - mean) * rstd;
                db[k][j] += dy[k][j];
                dg[k][j] = fmaf(dy[k][j], xh[k][j], dg[k][j]);
                dy[k][j] *= gm[j];
                s1 += dy[k][j];
                s2 = fmaf(dy[k][j], xh[k][j], s2);
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (nw > 1) {
            // two buffers in turn: a thread that writes one again has passed the
            // barrier behind which every thread had read it
            if ((t & 31) == 0) red[flip][threadIdx.x >> 5] = make_float2(s1, s2);
            asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(gt) : "memory");
            s1 = s2 = 0.0f;
            for (int i = 0; i < nw; ++i) {
                const float2 r = red[flip][w0 + i];
                s1 += r.x;
                s2 += r.y;
            }
            flip ^= 1;
        }
        const float c1 = s1 * inv_n, c2 = s2 * inv_n;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = static_cast<int64_t>(t + k * gt) * V;
            if (c < a.cols) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = rstd * (dy[k][j] - c1 - xh[k][j] * c2);
                if (a.add.p != nullptr) {
                    float e[V];
                    loadv<V>(a.add.p, a.add.dtype, row * a.add.ld + c, e);
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] += e[j];
                }
                storev<V>(a.dx.p, a.dx.dtype, row * a.dx.ld + c, o);
            }
        }
    }
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    if (G > 1) {
        for (int i = 0; i < G; ++i) {
            if (g == i) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int64_t c = static_cast<int64_t>(t + k * gt) * V;
                    if (c < a.cols) {
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            float* p = comb + c + j;
                            p[0] = (i ? p[0] : 0.0f) + dg[k][j];
                            p[a.cols] = (i ? p[a.cols] : 0.0f) + db[k][j];
                        }
                    }
                }
            }
            __syncthreads();
        }
        for (int64_t i = threadIdx.x; i < 2 * a.cols; i += blockDim.x) part[i] = comb[i];
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = static_cast<int64_t>(t + k * gt) * V;
            if (c < a.cols) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    part[c + j] = dg[k][j];
                    part[a.cols + c + j] = db[k][j];
                }
            }
        }
    }
}

// Rows too long for registers: dx first (two passes over a row), then the
// column sums from dy and x once more.
__global__ void __launch_bounds__(1024) norm_backward_wide_dx_kernel(NormBackward a) {
    __shared__ float red[2][32];
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float x;
            load_x<1>(a.x, row, c, &x);
            const float gr = load1(a.dy.p, a.dy.dtype, row * a.dy.ld + c) * load1(a.gamma, a.param_dtype, c);
            s1 += gr;
            s2 = fmaf(gr, (x - mean) * rstd, s2);
        }
        const float c1 = block_sum(s1, red[0]) * inv_n, c2 = block_sum(s2, red[1]) * inv_n;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float x;
            load_x<1>(a.x, row, c, &x);
            const float gr = load1(a.dy.p, a.dy.dtype, row * a.dy.ld + c) * load1(a.gamma, a.param_dtype, c);
            float o = rstd * (gr - c1 - (x - mean) * rstd * c2);
            if (a.add.p != nullptr) o += load1(a.add.p, a.add.dtype, row * a.add.ld + c);
            store1(a.dx.p, a.dx.dtype, row * a.dx.ld + c, o);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) norm_backward_wide_sums_kernel(NormBackward a) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= a.cols) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        float x;
        load_x<1>(a.x, row, c, &x);
        const float d = load1(a.dy.p, a.dy.dtype, row * a.dy.ld + c);
        db += d;
        dg = fmaf(d, (x - a.mean[row]) * a.rstd[row], dg);
    }
    float* part = a.partials + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
    part[c] = dg;
    part[a.cols + c] = db;
}

// out0 from partials[p*stride + c], out1 (blockIdx.y == 1) from columns
// further on by `second`: 32 columns and 32 slices of p to a block, the slices
// joined in order.
__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* partials, int64_t count, int64_t stride,
                                                            int64_t second, int64_t cols, void* out0, void* out1,
                                                            int dtype, int accumulate) {
    __shared__ float part[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + tx;
    void* out = blockIdx.y ? out1 : out0;
    const float* p = partials + (blockIdx.y ? second : 0) + c;
    float s = 0.0f;
    if (c < cols)
        for (int64_t i = ty; i < count; i += 32) s += p[i * stride];
    part[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < cols) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += part[i][tx];
        if (accumulate) s += load1(out, dtype, c);
        store1(out, dtype, c, s);
    }
}

cudaError_t sum_partials(const float* partials, int64_t count, int64_t stride, int64_t second, int64_t cols,
                         void* out0, void* out1, int dtype, int accumulate, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((cols + 31) / 32), out1 != nullptr ? 2 : 1);
    sum_partials_kernel<<<grid, 1024, 0, st>>>(partials, count, stride, second, cols, out0, out1, dtype, accumulate);
    return cudaGetLastError();
}

int round32(int64_t n) { return static_cast<int>((n + 31) / 32 * 32); }

template <int V, int NV>
cudaError_t run_forward(const NormForward& a, int64_t chunks, cudaStream_t st) {
    const int64_t cap = int64_t(1) << 30;
    if (chunks <= 32 * NV) {
        norm_forward_kernel<V, NV, true><<<static_cast<unsigned>(std::min((a.rows + 3) / 4, cap)), 128, 0, st>>>(a);
    } else {
        norm_forward_kernel<V, NV, false><<<static_cast<unsigned>(std::min(a.rows, cap)),
                                            round32((chunks + NV - 1) / NV), 0, st>>>(a);
    }
    return cudaGetLastError();
}

// The backward's split: vector chunks or single columns, threads to a row,
// rows to a block.
struct BackwardPlan {
    int V, NV, gt, groups;   // NV 0: rows too long for registers
    int64_t blocks;
};

BackwardPlan backward_plan(int64_t rows, int64_t cols, bool vec, int sms) {
    BackwardPlan p{};
    p.V = vec ? 8 : 1;
    const int64_t chunks = (cols + p.V - 1) / p.V;
    if (vec) p.NV = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : chunks <= 1536 ? 3 : 0;
    else p.NV = chunks <= 4096 ? 8 : chunks <= 12288 ? 24 : 0;
    if (p.NV == 0) {
        p.blocks = std::max<int64_t>(1, std::min<int64_t>(rows, 16));
        return p;
    }
    p.gt = round32((chunks + p.NV - 1) / p.NV);
    const int most = p.NV == 1 || p.NV == 8 ? 1024 : 512;
    // a named barrier to a group: 15 at most
    p.groups = std::max(1, std::min(std::min(most / p.gt, 15), static_cast<int>(std::min<int64_t>(rows, 15))));
    p.blocks = std::max<int64_t>(1, std::min<int64_t>((rows + p.groups - 1) / p.groups, sms));
    return p;
}

}  // namespace

cudaError_t launch_norm_forward(const NormForward& a, int sms, cudaStream_t st) {
    (void)sms;
    if (a.rows == 0) return cudaSuccess;
    const bool vec = rows_aligned(a.x) && rows_aligned(a.y) && a.cols % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.gamma) | reinterpret_cast<uintptr_t>(a.beta)) & 15u) == 0;
    if (vec) {
        const int64_t chunks = a.cols / 8;
        if (chunks <= 512) return run_forward<8, 2>(a, chunks, st);
        if (chunks <= 4096) return run_forward<8, 4>(a, chunks, st);
    } else {
        if (a.cols <= 4096) return run_forward<1, 8>(a, a.cols, st);
        if (a.cols <= 16384) return run_forward<1, 16>(a, a.cols, st);
    }
    norm_forward_wide_kernel<<<static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t(1) << 30)), 1024, 0, st>>>(a);
    return cudaGetLastError();
}

int64_t norm_partials(int64_t rows, int64_t cols, int sms) {
    return std::max(backward_plan(rows, cols, true, sms).blocks, backward_plan(rows, cols, false, sms).blocks);
}

cudaError_t launch_norm_backward(const NormBackward& a, int sms, cudaStream_t st) {
    const bool vec = rows_aligned(a.dy) && rows_aligned(a.x) && rows_aligned(a.dx) &&
                     (a.add.p == nullptr || rows_aligned(a.add)) && a.cols % 8 == 0 &&
                     (reinterpret_cast<uintptr_t>(a.gamma) & 15u) == 0;
    const BackwardPlan p = backward_plan(a.rows, a.cols, vec, sms);
    cudaError_t e = cudaSuccess;
    int64_t count = p.blocks;
    if (a.rows == 0) {
        count = 0;
    } else if (p.NV == 0) {
        norm_backward_wide_dx_kernel<<<static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t(1) << 30)), 1024, 0, st>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const dim3 grid(static_cast<unsigned>((a.cols + 255) / 256), static_cast<unsigned>(p.blocks));
        norm_backward_wide_sums_kernel<<<grid, 256, 0, st>>>(a);
        e = cudaGetLastError();
    } else {
        const int threads = p.gt * p.groups;
        const size_t smem = p.groups > 1 ? static_cast<size_t>(2 * a.cols) * sizeof(float) : 0;
        auto go = [&](auto kernel) {
            if (smem > 40 * 1024)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (e == cudaSuccess) {
                kernel<<<static_cast<unsigned>(p.blocks), threads, smem, st>>>(a, p.gt);
                e = cudaGetLastError();
            }
        };
        if (p.V == 8) {
            if (p.NV == 1) go(norm_backward_kernel<8, 1, 1024>);
            else if (p.NV == 2) go(norm_backward_kernel<8, 2, 512>);
            else go(norm_backward_kernel<8, 3, 512>);
        } else {
            if (p.NV == 8) go(norm_backward_kernel<1, 8, 1024>);
            else go(norm_backward_kernel<1, 24, 512>);
        }
    }
    if (e != cudaSuccess) return e;
    return sum_partials(a.partials, count, 2 * a.cols, a.cols, a.cols, a.dgamma, a.dbeta, a.grad_dtype, a.accumulate, st);
}

cudaError_t launch_sum_partials(const float* partials, int64_t count, int64_t stride, int64_t cols, void* out,
                                int out_dtype, int accumulate, cudaStream_t st) {
    return sum_partials(partials, count, stride, 0, cols, out, nullptr, out_dtype, accumulate, st);
}

}  // namespace fsdp
