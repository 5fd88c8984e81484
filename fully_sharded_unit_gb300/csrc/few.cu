// Products of a few rows: y = x W for one to eight tokens, and the same for an
// input gradient.  W is read once; no tile of the tensor cores could be filled.
// One token, 1280 -> 5120: 10.3 us alone and cold, where 13 MB of W from DRAM take
// 1.9 and a launch two more: two dependent steps of loads bound it, the second a
// quarter full.  7.0 a call in a stream of them that finds W in L2, which the
// launching host bounds; by the tensor cores, 64 tokens take 7.5.
//
// A block computes 32 columns (a checkpoint's group), a cluster of up to 8
// blocks splits k where the columns alone would leave SMs idle, and the first
// block of the cluster adds the others' sums from their shared memory, in order.
#include <cooperative_groups.h>

#include <algorithm>

#include "block_device.cuh"
#include "compute.hpp"
#include "epilogue.cuh"

namespace cg = cooperative_groups;

namespace fsdp {
namespace {

// One row by columns keeps more of W in flight with 16 warps; by rows, 8 warps
// of 4 columns make up a block's 32.
__host__ __device__ constexpr int few_threads(int T, bool by_columns) { return T == 1 && by_columns ? 512 : 256; }

__device__ __forceinline__ float bf(uint16_t w) { return __uint_as_float(static_cast<uint32_t>(w) << 16); }

// The first `left` (0 or fewer: none) of eight elements, the others 0.
__device__ __forceinline__ uint4 load_end(const uint16_t* src, int64_t left) {
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; i < 8; ++i)
        if (i < left) w[i >> 1] |= static_cast<uint32_t>(src[i]) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// W contiguous along the columns (p.b_trans): V columns and 8 rows of W to a
// thread at a time.
template <int V, int T>
__device__ __forceinline__ void sums_by_columns(const Product& p, int64_t n0, int64_t k0, int64_t k1, float (*part)[T][33]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kAcross = 32 / V;                     // lanes across the 32 columns
    constexpr int kDown = 32 / kAcross;                 // row groups in a warp
    const int64_t n = n0 + (lane % kAcross) * V;
    const uint16_t* W = static_cast<const uint16_t*>(p.b.p);
    const uint16_t* X = static_cast<const uint16_t*>(p.a.p);
    float acc[T][V];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[t][j] = 0.0f;
    for (int64_t k = k0 + (warp * kDown + lane / kAcross) * 8; k < k1; k += (blockDim.x >> 5) * kDown * 8) {
        uint4 w8[8];
        uint16_t w1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (V == 8)
                w8[i] = k + i < k1 && n < p.N ? *reinterpret_cast<const uint4*>(W + (k + i) * p.b.ld + n) : make_uint4(0, 0, 0, 0);
            else
                w1[i] = k + i < k1 && n < p.N ? W[(k + i) * p.b.ld + n] : uint16_t(0);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float x[8];
            if (t < p.M && V == 8 && k + 8 <= k1) {
                unpack8(*reinterpret_cast<const uint4*>(X + t * p.a.ld + k), x);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = t < p.M && k + i < k1 ? bf(X[t * p.a.ld + k + i]) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (V == 8) {
                    float w[8];
                    unpack8(w8[i], w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[t][j] = fmaf(x[i], w[j], acc[t][j]);
                } else {
                    acc[t][0] = fmaf(x[i], bf(w1[i]), acc[t][0]);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float s = acc[t][j];
#pragma unroll
            for (int d = kAcross; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (lane < kAcross) part[warp][t][lane * V + j] = s;
        }
}

// W contiguous along k: 4 columns to a warp, V values of k to a lane at a time.
template <int V, int T>
__device__ __forceinline__ void sums_by_rows(const Product& p, int64_t n0, int64_t k0, int64_t k1, float (*part)[T][33]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t* W = static_cast<const uint16_t*>(p.b.p);
    const uint16_t* X = static_cast<const uint16_t*>(p.a.p);
    float acc[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = 0.0f;
    if constexpr (V == 8) {
        // two steps of k at a time: eight loads of W in flight to a lane
        for (int64_t k = k0 + lane * 8; k < k1; k += 512) {
            uint4 w[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t n = n0 + warp * 4 + j, kk = k + u * 256;
                    w[u][j] = n < p.N && kk + 8 <= k1 ? *reinterpret_cast<const uint4*>(W + n * p.b.ld + kk)
                                                      : load_end(W + n * p.b.ld + kk, n < p.N ? k1 - kk : 0);
                }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const int64_t kk = k + u * 256;
                    const uint16_t* src = X + t * p.a.ld + kk;
                    float x[8];
                    unpack8(t < p.M && kk + 8 <= k1 ? *reinterpret_cast<const uint4*>(src)
                                                    : load_end(src, t < p.M ? k1 - kk : 0), x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v[8];
                        unpack8(w[u][j], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[t][j] = fmaf(x[i], v[i], acc[t][j]);
                    }
                }
        }
    } else {
#pragma unroll 4
        for (int64_t k = k0 + lane; k < k1; k += 32) {
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + warp * 4 + j;
                w[j] = n < p.N ? bf(W[n * p.b.ld + k]) : 0.0f;
            }
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const float x = t < p.M ? bf(X[t * p.a.ld + k]) : 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[t][j] = fmaf(x, w[j], acc[t][j]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float s = acc[t][j];
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (lane == 0) part[0][t][warp * 4 + j] = s;
        }
}

template <int V, int T, bool BY_COLUMNS>
__global__ void __launch_bounds__(few_threads(T, BY_COLUMNS)) few_rows_kernel(const __grid_constant__ Product p) {
    constexpr int kWarps = few_threads(T, BY_COLUMNS) / 32;
    __shared__ float part[kWarps][T][33];
    __shared__ float total[T][33];
    starts_early();
    after_previous();
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int64_t n0 = static_cast<int64_t>(blockIdx.x / parts) * 32;
    const int64_t chunks = (p.K + 7) / 8;   // the cut of k falls on multiples of 8
    const int64_t k0 = chunks * rank / parts * 8;
    const int64_t k1 = min(p.K, chunks * (rank + 1) / parts * 8);
    if constexpr (BY_COLUMNS) sums_by_columns<V, T>(p, n0, k0, k1, part);
    else sums_by_rows<V, T>(p, n0, k0, k1, part);
    __syncthreads();
    for (int i = threadIdx.x; i < T * 32; i += kWarps * 32) {
        const int t = i >> 5, c = i & 31;
        float s = part[0][t][c];
        if constexpr (BY_COLUMNS) {
#pragma unroll
            for (int w = 1; w < kWarps; ++w) s += part[w][t][c];
        }
        total[t][c] = s;
    }
    if (parts > 1) cluster.sync();
    else __syncthreads();
    if (rank == 0 && threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int64_t n = n0 + lane;
        float v[T];
#pragma unroll
        for (int t = 0; t < T; ++t) v[t] = total[t][lane];
        for (int r = 1; r < parts; ++r) {
            const float(*theirs)[33] = reinterpret_cast<const float(*)[33]>(cluster.map_shared_rank(&total[0][0], r));
#pragma unroll
            for (int t = 0; t < T; ++t) v[t] += theirs[t][lane];
        }
        const float bias = p.bias != nullptr && n < p.N ? load1(p.bias, p.bias_dtype, n) : 0.0f;
        if (p.slope) finish_column<T, true>(p, 0, static_cast<int>(p.M), n, bias, v, lane);
        else finish_column<T, false>(p, 0, static_cast<int>(p.M), n, bias, v, lane);
    }
    if (parts > 1) cluster.sync();   // the sums stay until the first block has read them
}

template <int V, int T>
cudaError_t run(const Product& p, cudaLaunchConfig_t& cfg) {
    cfg.blockDim = dim3(few_threads(T, p.b_trans != 0));
    return p.b_trans ? cudaLaunchKernelEx(&cfg, few_rows_kernel<V, T, true>, p)
                     : cudaLaunchKernelEx(&cfg, few_rows_kernel<V, T, false>, p);
}

}  // namespace

cudaError_t launch_few_rows(const Product& p, int sms, cudaStream_t st) {
    const int64_t blocks = (p.N + 31) / 32;
    // parts of k, of at least 256 each, until every SM has a block
    int parts = 1;
    while (parts < 8 && blocks * parts < sms && p.K >= 512 * parts) parts *= 2;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(parts);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * parts));
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = parts > 1 ? 2 : 1;
    const bool vec = rows_aligned(p.a) && rows_aligned(p.b) && (!p.b_trans || p.N % 8 == 0);
    if (p.M == 1) return vec ? run<8, 1>(p, cfg) : run<1, 1>(p, cfg);
    if (p.M <= 4) return vec ? run<8, 4>(p, cfg) : run<1, 4>(p, cfg);
    return vec ? run<8, 8>(p, cfg) : run<1, 8>(p, cfg);
}

}  // namespace fsdp
