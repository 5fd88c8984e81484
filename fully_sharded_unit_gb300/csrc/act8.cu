// 8-bit activation checkpoints: pack (quantise) and unpack.  Streaming passes,
// bound by DRAM: pack reads 2 or 4 bytes and writes 33/32 byte an element,
// unpack the reverse.
#include <algorithm>

#include "block_device.cuh"
#include "compute.hpp"
#include "epilogue.cuh"

namespace fsdp {
namespace {

// A whole group to a lane: 32 elements hide each other's latency, the largest
// magnitude needs no exchange between lanes, and loads, payload and exponents
// are whole sectors.  The payload's rows and the exponents' are contiguous
// (their strides are the format's), so a group's place in them is its index.
// 8192 x 5120: pack 24.5 us (5.2 TB/s), unpack with GELU 28 (4.5; the special
// functions take half of it); 4096 x 12288: unpack 27 (5.7).
template <bool WIDE, bool PACK>
__global__ void __launch_bounds__(256) act8_groups_kernel(int64_t cols, Mat q, int act, Mat x, int64_t count, uint32_t groups) {
    starts_early();
    after_previous();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; g < count; g += stride) {
        // a 32-bit division where the index allows it
        const int64_t row = g <= 0xffffffffll ? static_cast<uint32_t>(g) / groups : g / groups;
        const int64_t n = (g - row * groups) * kGroup;
        const int left = static_cast<int>(min(static_cast<int64_t>(kGroup), cols - n));
        float v[32];
        if (PACK) {
            load_row32<WIDE>(x, row, n, left, v);
            q.e[g] = static_cast<uint8_t>(store_row32<WIDE>(q, row, n, left, v));
        } else {
            load_row32<WIDE>(q, row, n, left, v);
            activate_n<32>(v, act);
            store_row32<WIDE>(x, row, n, left, v);
        }
    }
}

// Rows that start anywhere: a group to a warp, an element to a lane, U groups
// in flight.  Bound by loads and stores of two bytes a lane: pack of 4096 x 1281,
// 27 us (an aligned 4096 x 1280 takes 6.4).
template <bool PACK>
__global__ void __launch_bounds__(256) act8_elements_kernel(int64_t cols, Mat q, int act, Mat x, int64_t count, uint32_t groups) {
    starts_early();
    after_previous();
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t g0 = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); g0 < count; g0 += stride * U) {
        float v[U];
        int64_t row[U], n[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * stride;
            row[u] = g <= 0xffffffffll ? static_cast<uint32_t>(g) / groups : g / groups;
            n[u] = (g - row[u] * groups) * kGroup + lane;
            on[u] = g < count && n[u] < cols;
            v[u] = 0.0f;
        }
        if (PACK && x.dtype == FSDP_DTYPE_F32) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (on[u]) v[u] = static_cast<const float*>(x.p)[row[u] * x.ld + n[u]];
        } else if (PACK) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (on[u]) v[u] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(x.p)[row[u] * x.ld + n[u]]) << 16);
        } else {
            int w[U];
            uint32_t byte[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                w[u] = on[u] ? static_cast<const int8_t*>(q.p)[row[u] * q.ld + n[u]] : 0;
                byte[u] = on[u] ? q.e[row[u] * q.eld + (n[u] >> 5)] : 127u;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = static_cast<float>(w[u]) * act8_step(byte[u]);
        }
        if (PACK) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t top = act8_group_top<1>(&v[u]);
                if (g0 + u * stride < count) {
                    act8_writev<1>(static_cast<uint8_t*>(q.p) + row[u] * q.ld, n[u], &v[u], top);
                    if (lane == 0) q.e[row[u] * q.eld + (n[u] >> 5)] = static_cast<uint8_t>(act8_byte(top));
                }
            }
        } else {
            activate_n<U>(v, act);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (on[u]) store1(x.p, x.dtype, row[u] * x.ld + n[u], v[u]);
        }
    }
}

template <bool PACK>
cudaError_t launch(int64_t rows, int64_t cols, const Mat& q, int act, const Mat& x, int sms, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    const int64_t groups = act8_groups(cols), count = rows * groups;
    if (groups > 0xffffffffll) return cudaErrorInvalidValue;
    const auto blocks = [&](int64_t per_block) {
        return static_cast<unsigned>(std::min((count + per_block - 1) / per_block, static_cast<int64_t>(sms) * 24));
    };
    const uint32_t gr = static_cast<uint32_t>(groups);
    if (rows_aligned(x) && cols % 8 == 0) {
        const bool wide = rows_aligned(x, 32) && rows_aligned(q, 32) && cols % 16 == 0;
        return launch_early(wide ? act8_groups_kernel<true, PACK> : act8_groups_kernel<false, PACK>, dim3(blocks(256)), 256, 0, st,
                            cols, q, act, x, count, gr);
    }
    return launch_early(act8_elements_kernel<PACK>, dim3(blocks(32)), 256, 0, st, cols, q, act, x, count, gr);
}

}  // namespace

cudaError_t launch_act8_pack(int64_t rows, int64_t cols, const Mat& x, const Mat& q, int sms, cudaStream_t st) {
    return launch<true>(rows, cols, q, 0, x, sms, st);
}

cudaError_t launch_act8_unpack(int64_t rows, int64_t cols, const Mat& q, int activation, const Mat& out, int sms,
                               cudaStream_t st) {
    return launch<false>(rows, cols, q, activation, out, sms, st);
}

}  // namespace fsdp
