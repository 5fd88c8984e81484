// The linear layer's products, and the column sums of its bias's gradient.
#include <algorithm>

#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {
namespace {

__device__ __forceinline__ float load_mat(const Mat& m, int64_t r, int64_t c) {
    if (m.dtype == FSDP_DTYPE_ACT8) {
        float v;
        act8_readv<1>(static_cast<const uint8_t*>(m.p) + r * m.ld, m.e + r * m.eld, c, &v);
        return v;
    }
    return load1(m.p, m.dtype, r * m.ld + c);
}

// A 64 x 64 tile to a block, 4 x 4 products to a thread, fp32 multiply-adds.
__global__ void __launch_bounds__(256) product_kernel(Product p) {
    __shared__ float sa[16][65], sb[16][65], sz[64][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * 64; m0 < p.M; m0 += static_cast<int64_t>(gridDim.y) * 64) {
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
            for (int i = threadIdx.x; i < 1024; i += 256) {
                const int ka = p.a_trans ? i >> 6 : i & 15, ma = p.a_trans ? i & 63 : i >> 4;
                const int kb = p.b_trans ? i >> 6 : i & 15, nb = p.b_trans ? i & 63 : i >> 4;
                const int64_t m = m0 + ma, n = n0 + nb;
                float va = 0.0f, vb = 0.0f;
                if (m < p.M && k0 + ka < p.K) va = p.a_trans ? load_mat(p.a, k0 + ka, m) : load_mat(p.a, m, k0 + ka);
                if (n < p.N && k0 + kb < p.K) vb = p.b_trans ? load_mat(p.b, k0 + kb, n) : load_mat(p.b, n, k0 + kb);
                sa[ka][ma] = va;
                sb[kb][nb] = vb;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                float x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = sa[k][ty + 16 * i];
                    y[i] = sb[k][tx + 16 * i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sz[ty + 16 * i][tx + 16 * j] = acc[i][j];
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int r = threadIdx.x >> 5; r < 64; r += 8) {
            const int64_t m = m0 + r;
            if (m >= p.M) break;   // the same for the whole warp
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t n = n0 + h * 32 + lane;
                const bool on = n < p.N;
                float v = on ? sz[r][h * 32 + lane] : 0.0f;
                if (p.bias != nullptr && on) v += load1(p.bias, p.bias_dtype, n);
                if (!p.slope) {
                    if (p.pre.p != nullptr) {
                        if (p.pre.dtype == FSDP_DTYPE_ACT8) {
                            const uint32_t byte = act8_group_byte<1>(&v);
                            if (n < p.pre.ld) {
                                act8_writev<1>(static_cast<uint8_t*>(p.pre.p) + m * p.pre.ld, n, &v, byte);
                                if (lane == 0) p.pre.e[m * p.pre.eld + (n >> 5)] = static_cast<uint8_t>(byte);
                            }
                        } else if (on) {
                            store1(p.pre.p, p.pre.dtype, m * p.pre.ld + n, v);
                        }
                    }
                    v = activate(v, p.act);
                } else if (on) {
                    v *= act_slope(load_mat(p.pre, m, n), p.act);
                }
                if (on) {
                    if (p.add.p != nullptr) v += load1(p.add.p, p.add.dtype, m * p.add.ld + n);
                    store1(p.out.p, p.out.dtype, m * p.out.ld + n, v);
                }
            }
        }
        __syncthreads();
    }
}

// 256 columns and one slice of the rows to a block.
__global__ void __launch_bounds__(256) column_sum_kernel(int64_t rows, int64_t cols, Mat dy, float* partials) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= cols) return;
    float s = 0.0f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) s += load1(dy.p, dy.dtype, r * dy.ld + c);
    partials[static_cast<int64_t>(blockIdx.y) * cols + c] = s;
}

}  // namespace

cudaError_t launch_product(const Product& p, int sms, cudaStream_t st) {
    (void)sms;
    if (p.M == 0 || p.N == 0) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>((p.N + 63) / 64), static_cast<unsigned>(std::min<int64_t>((p.M + 63) / 64, 65535)));
    product_kernel<<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

int64_t column_sum_partials(int64_t rows, int64_t cols, int sms) {
    const int64_t blocks = (cols + 255) / 256;
    return std::max<int64_t>(1, std::min<int64_t>(rows, std::min<int64_t>(256, (4 * sms + blocks - 1) / blocks)));
}

cudaError_t launch_column_sum(int64_t rows, int64_t cols, const Mat& dy, float* partials, void* out, int out_dtype,
                              int accumulate, int sms, cudaStream_t st) {
    int64_t count = 0;
    if (rows > 0) {
        count = column_sum_partials(rows, cols, sms);
        const dim3 grid(static_cast<unsigned>((cols + 255) / 256), static_cast<unsigned>(count));
        column_sum_kernel<<<grid, 256, 0, st>>>(rows, cols, dy, partials);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return launch_sum_partials(partials, count, cols, cols, out, out_dtype, accumulate, st);
}

}  // namespace fsdp
