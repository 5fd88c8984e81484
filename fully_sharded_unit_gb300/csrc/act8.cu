// 8-bit activation checkpoints: pack (quantise) and unpack.  Streaming passes:
// pack reads 2 or 4 bytes and writes 33/32 byte an element, unpack the reverse.
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
// functions take half of it); 4096 x 12288: unpack 27 (5.7).  DRAM is half busy, by
// ncu, with 31 % of the warps that an SM can hold: what is in flight bounds them.
// ANY: x's rows start anywhere and are read and stored as the 16-byte words that
// hold them (4096 x 1281: pack 11 us, unpack 11; an element to a lane took 27).
template <bool WIDE, bool ANY, bool PACK>
__global__ void __launch_bounds__(256) act8_groups_kernel(int64_t cols, Mat q, int act, Mat x, int64_t count, uint32_t groups) {
    starts_early();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    // whole warps where lanes store together
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; g - (ANY ? lane : 0) < count; g += stride) {
        // a 32-bit division where the index allows it
        const int64_t row = g <= 0xffffffffll ? static_cast<uint32_t>(g) / groups : g / groups;
        const int64_t n = (g - row * groups) * kGroup;
        const int left = g < count ? static_cast<int>(min(static_cast<int64_t>(kGroup), cols - n)) : 0;
        float v[32];
        if constexpr (PACK) {
            if (ANY && left == 0) continue;
            if (ANY) load_row32_any(x, row, n, left, v);
            else load_row32<WIDE>(x, row, n, left, v);
            q.e[g] = static_cast<uint8_t>(store_row32<WIDE>(q, row, n, left, v));
        } else {
            if (!ANY || left > 0) load_row32<WIDE>(q, row, n, left, v);
            activate_n<32>(v, act);
            if constexpr (ANY) store_row32_any(x, row, n, left, lane > 0 && n > 0 && left > 0, v);
            else store_row32<WIDE>(x, row, n, left, v);
        }
    }
}

template <bool PACK>
cudaError_t launch(int64_t rows, int64_t cols, const Mat& q, int act, const Mat& x, int sms, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    const int64_t groups = act8_groups(cols), count = rows * groups;
    if (groups > 0xffffffffll) return cudaErrorInvalidValue;
    const unsigned blocks = static_cast<unsigned>(std::min((count + 255) / 256, static_cast<int64_t>(sms) * 24));
    const bool aligned = rows_aligned(x) && cols % 8 == 0;
    const bool wide = aligned && rows_aligned(x, 32) && rows_aligned(q, 32) && cols % 16 == 0;
    const auto kernel = wide ? act8_groups_kernel<true, false, PACK>
                             : aligned ? act8_groups_kernel<false, false, PACK> : act8_groups_kernel<false, true, PACK>;
    return launch_early(kernel, dim3(blocks), 256, 0, st, cols, q, act, x, count, static_cast<uint32_t>(groups));
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
