// 8-bit activation checkpoints: pack (quantise) and unpack.  Streaming passes,
// bound by DRAM: pack reads 2 or 4 bytes and writes 33/32 byte an element,
// unpack the reverse.
#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {
namespace {

// Work is cut into items of 32*V consecutive columns of one row, one item to a
// warp at a time.  A warp walks items w, w + W, w + 2W, ... and keeps its row
// and segment by adding (W / segs, W % segs), so no division runs in the loop.
struct Items {
    int64_t count;      // rows * segs
    int64_t segs;       // items in a row
    int64_t step_row;   // W / segs
    int64_t step_seg;   // W % segs
};

template <int V, int U>
__global__ void __launch_bounds__(256) act8_pack_kernel(int64_t cols, Mat x, Mat q, Items it) {
    const int lane = threadIdx.x & 31;
    const int64_t W = static_cast<int64_t>(gridDim.x) * 8;
    int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    int64_t row = i / it.segs, seg = i % it.segs;
    while (i < it.count) {
        float v[U][V];
        int64_t rows[U], c[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rows[u] = row;
            c[u] = (seg * 32 + lane) * V;
            on[u] = i < it.count;
            // cols is a multiple of 8 where V = 8
            if (on[u] && c[u] < cols) {
                loadv<V>(x.p, x.dtype, row * x.ld + c[u], v[u]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v[u][j] = 0.0f;
            }
            i += W;
            row += it.step_row;
            seg += it.step_seg;
            if (seg >= it.segs) { seg -= it.segs; ++row; }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t byte = act8_group_byte<V>(v[u]);
            if (on[u] && c[u] < q.ld) {
                act8_writev<V>(static_cast<uint8_t*>(q.p) + rows[u] * q.ld, c[u], v[u], byte);
                if ((lane & (32 / V - 1)) == 0) q.e[rows[u] * q.eld + (c[u] >> 5)] = static_cast<uint8_t>(byte);
            }
        }
    }
}

template <int V, int U>
__global__ void __launch_bounds__(256) act8_unpack_kernel(int64_t cols, Mat q, int act, Mat out, Items it) {
    const int lane = threadIdx.x & 31;
    const int64_t W = static_cast<int64_t>(gridDim.x) * 8;
    int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    int64_t row = i / it.segs, seg = i % it.segs;
    while (i < it.count) {
        float v[U][V];
        int64_t rows[U], c[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rows[u] = row;
            c[u] = (seg * 32 + lane) * V;
            on[u] = i < it.count && c[u] < cols;
            if (on[u])
                act8_readv<V>(static_cast<const uint8_t*>(q.p) + row * q.ld, q.e + row * q.eld, c[u], v[u]);
            i += W;
            row += it.step_row;
            seg += it.step_seg;
            if (seg >= it.segs) { seg -= it.segs; ++row; }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!on[u]) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) v[u][j] = activate(v[u][j], act);
            storev<V>(out.p, out.dtype, rows[u] * out.ld + c[u], v[u]);
        }
    }
}

Items plan_items(int64_t rows, int64_t cols, int per_warp, int sms, int U, int* blocks) {
    Items it;
    it.segs = (cols + per_warp - 1) / per_warp;
    it.count = rows * it.segs;
    const int64_t want = (it.count + 8 * U - 1) / (8 * U);
    const int64_t most = static_cast<int64_t>(sms) * 8;
    *blocks = static_cast<int>(want < most ? want : most);
    const int64_t W = static_cast<int64_t>(*blocks) * 8;
    it.step_row = W / it.segs;
    it.step_seg = W % it.segs;
    return it;
}

}  // namespace

cudaError_t launch_act8_pack(int64_t rows, int64_t cols, const Mat& x, const Mat& q, int sms, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    int blocks = 0;
    if (rows_aligned(x) && cols % 8 == 0) {
        const Items it = plan_items(rows, cols, 256, sms, 4, &blocks);
        act8_pack_kernel<8, 4><<<blocks, 256, 0, st>>>(cols, x, q, it);
    } else {
        const Items it = plan_items(rows, cols, 32, sms, 8, &blocks);
        act8_pack_kernel<1, 8><<<blocks, 256, 0, st>>>(cols, x, q, it);
    }
    return cudaGetLastError();
}

cudaError_t launch_act8_unpack(int64_t rows, int64_t cols, const Mat& q, int activation, const Mat& out, int sms,
                               cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    int blocks = 0;
    if (rows_aligned(out) && cols % 8 == 0) {
        const Items it = plan_items(rows, cols, 256, sms, 4, &blocks);
        act8_unpack_kernel<8, 4><<<blocks, 256, 0, st>>>(cols, q, activation, out, it);
    } else {
        const Items it = plan_items(rows, cols, 32, sms, 8, &blocks);
        act8_unpack_kernel<1, 8><<<blocks, 256, 0, st>>>(cols, q, activation, out, it);
    }
    return cudaGetLastError();
}

}  // namespace fsdp
