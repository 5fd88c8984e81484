// The linear layer's epilogue (see Product in compute.hpp): bias, kept
// pre-activation, activation or its slope, added matrix, store.
#pragma once

#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {

// 32 consecutive columns of one row, from column n (a multiple of 32); `left`
// of them are inside the matrix (a multiple of 8, of 16 where WIDE).
template <bool WIDE>
__device__ __forceinline__ void load_row32(const Mat& x, int64_t m, int64_t n, int left, float* v) {
    if (x.dtype == FSDP_DTYPE_F32) {
        const float* src = static_cast<const float*>(x.p) + m * x.ld + n;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s * 8 < left) {
                if (WIDE) {
                    uint32_t w[8];
                    load32b(src + s * 8, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[s * 8 + j] = __uint_as_float(w[j]);
                } else {
                    load8(src, FSDP_DTYPE_F32, s * 8, v + s * 8);
                }
            }
        }
    } else if (x.dtype == FSDP_DTYPE_BF16) {
        const uint16_t* src = static_cast<const uint16_t*>(x.p) + m * x.ld + n;
        if (WIDE) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s * 16 < left) {
                    uint32_t w[8];
                    load32b(src + s * 16, w);
                    unpack8(make_uint4(w[0], w[1], w[2], w[3]), v + s * 16);
                    unpack8(make_uint4(w[4], w[5], w[6], w[7]), v + s * 16 + 8);
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (s * 8 < left) load8(src, FSDP_DTYPE_BF16, s * 8, v + s * 8);
        }
    } else {   // a whole group: the pads are there
        const uint8_t* src = static_cast<const uint8_t*>(x.p) + m * x.ld + n;
        const float step = act8_step(x.e[m * x.eld + (n >> 5)]);
        uint32_t w[8];
        if (WIDE) {
            load32b(src, w);
        } else {
            const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) act8_read4(w[s], step, v + s * 4);
    }
}

// Returns the exponent byte of an ACT8 group, which is left to the caller.
template <bool WIDE>
__device__ __forceinline__ uint32_t store_row32(const Mat& x, int64_t m, int64_t n, int left, const float* v) {
    if (x.dtype == FSDP_DTYPE_F32) {
        float* dst = static_cast<float*>(x.p) + m * x.ld + n;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s * 8 < left) {
                if (WIDE) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[s * 8 + j]);
                    store32b(dst + s * 8, w);
                } else {
                    store8(dst, FSDP_DTYPE_F32, s * 8, v + s * 8);
                }
            }
        }
    } else if (x.dtype == FSDP_DTYPE_BF16) {
        uint16_t* dst = static_cast<uint16_t*>(x.p) + m * x.ld + n;
        if (WIDE) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s * 16 < left) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = to_bf16x2(v[s * 16 + 2 * j], v[s * 16 + 2 * j + 1]);
                    store32b(dst + s * 16, w);
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (s * 8 < left) store8(dst, FSDP_DTYPE_BF16, s * 8, v + s * 8);
        }
    } else {   // a checkpoint's group, in one lane
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) most = j < left ? larger(most, v[j]) : most;
        const uint32_t top = __float_as_uint(most);
        uint32_t w[8];
        act8_quant_n<32>(v, top, act8_scale(act8_byte(top)), w);
        if (left < 32) {   // the pad of a short group is zeros
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s * 4 >= left) w[s] = 0u;
        }
        uint8_t* dst = static_cast<uint8_t*>(x.p) + m * x.ld + n;
        if (WIDE) {
            store32b(dst, w);
        } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return act8_byte(top);
    }
    return 0;
}

// The epilogue of 32 columns of one row: everything a lane needs is in its own
// registers (a checkpoint's group too), so 32 independent elements hide each
// other's latency, and every access is a whole 32-byte sector.  `bias` is the
// lane's column's; `byte` takes the exponent byte of a checkpoint's group, which
// the caller stores.  All lanes of the warp come here; `on` if the lane's row
// exists.
template <bool WIDE, bool SLOPE>
__device__ __forceinline__ void finish_row(const Product& p, int64_t m, int64_t n, bool on, float bias, float* v,
                                           uint32_t* byte) {
    const int left = static_cast<int>(min(static_cast<int64_t>(32), p.N - n));
    if (p.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, bias, j);
    }
    if (!on) return;
    if (SLOPE) {
        float z[32];
        load_row32<WIDE>(p.pre, m, n, left, z);
        slope_n<32>(v, z, p.act);
    } else {
        if (p.pre.p != nullptr) *byte = store_row32<WIDE>(p.pre, m, n, left, v);
        activate_n<32>(v, p.act);
    }
    if (p.add.p != nullptr) {
        float e[32];
        load_row32<WIDE>(p.add, m, n, left, e);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += e[j];
    }
    store_row32<WIDE>(p.out, m, n, left, v);
}

// The epilogue where a lane holds one column n of R consecutive rows from m
// (`count` of them inside the matrix): matrices whose rows start anywhere, and
// tiles whose rows are C's columns.  n - lane is a multiple of 32.
template <int R, bool SLOPE>
__device__ __forceinline__ void finish_column(const Product& p, int64_t m, int count, int64_t n, float bias, float* v, int lane) {
    const bool in = n < p.N;
    const auto on = [&](int i) { return in && i < count; };
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] += bias;
    float e[R];
    if (p.add.p != nullptr) load_strided<R>(p.add.p, p.add.dtype, m * p.add.ld + n, p.add.ld, on, e);
    if (SLOPE) {
        float z[R];
        if (p.pre.dtype == FSDP_DTYPE_ACT8) {
            const int8_t* q = static_cast<const int8_t*>(p.pre.p) + m * p.pre.ld + n;
            const uint8_t* x = p.pre.e + m * p.pre.eld + (n >> 5);
            int w[R];
            uint32_t byte[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                w[i] = on(i) ? q[i * p.pre.ld] : 0;
                byte[i] = on(i) ? x[i * p.pre.eld] : 127u;
            }
#pragma unroll
            for (int i = 0; i < R; ++i) z[i] = static_cast<float>(w[i]) * act8_step(byte[i]);
        } else {
            load_strided<R>(p.pre.p, p.pre.dtype, m * p.pre.ld + n, p.pre.ld, on, z);
        }
        slope_n<R>(v, z, p.act);
    } else {
        if (p.pre.p != nullptr) {
            if (p.pre.dtype == FSDP_DTYPE_ACT8) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float x = in ? v[i] : 0.0f;
                    const uint32_t top = act8_group_top<1>(&x);
                    if (i < count && n < p.pre.ld) {
                        act8_writev<1>(static_cast<uint8_t*>(p.pre.p) + (m + i) * p.pre.ld, n, &x, top);
                        if (lane == 0) p.pre.e[(m + i) * p.pre.eld + (n >> 5)] = static_cast<uint8_t>(act8_byte(top));
                    }
                }
            } else {
                store_strided<R>(p.pre.p, p.pre.dtype, m * p.pre.ld + n, p.pre.ld, on, v);
            }
        }
        activate_n<R>(v, p.act);
    }
    if (p.add.p != nullptr) {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] += e[i];
    }
    store_strided<R>(p.out.p, p.out.dtype, m * p.out.ld + n, p.out.ld, on, v);
}

}  // namespace fsdp
