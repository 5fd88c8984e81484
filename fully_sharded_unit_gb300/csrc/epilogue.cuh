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
            for (int s = 0; s < 8; ++s) w[s] = s * 4 >= left ? 0u : s * 4 + 4 <= left ? w[s] : w[s] & ((1u << 8 * (left - s * 4)) - 1u);
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

// The same from a row that starts anywhere (BF16 or F32).  An element at a time,
// 32 loads of 64 bytes a warp, it took twice the time of the whole product.
__device__ __forceinline__ void load_row32_any(const Mat& x, int64_t m, int64_t n, int left, float* v) {
    if (x.dtype == FSDP_DTYPE_ACT8) {
        load_row32<false>(x, m, n, left, v);   // aligned by its format
    } else if (x.dtype == FSDP_DTYPE_F32) {
        uint32_t w[36];
        load_window<9>(reinterpret_cast<uintptr_t>(static_cast<const float*>(x.p) + m * x.ld + n), left * 4, w);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]);
    } else {
        uint32_t w[20];
        load_window<5>(reinterpret_cast<uintptr_t>(static_cast<const uint16_t*>(x.p) + m * x.ld + n), left * 2, w);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            v[2 * j] = bf16_lo(w[j]);
            v[2 * j + 1] = bf16_hi(w[j]);
        }
    }
}

// The reverse (see store_window); all lanes take part.
__device__ __forceinline__ void store_row32_any(const Mat& x, int64_t m, int64_t n, int left, bool joined, const float* v) {
    if (x.dtype == FSDP_DTYPE_F32) {
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j]);
        store_window<8>(reinterpret_cast<uintptr_t>(static_cast<float*>(x.p) + m * x.ld + n), left * 4, joined, w);
    } else {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = to_bf16x2(v[2 * j], v[2 * j + 1]);
        store_window<4>(reinterpret_cast<uintptr_t>(static_cast<uint16_t*>(x.p) + m * x.ld + n), left * 2, joined, w);
    }
}

// A 32 x 32 chunk whose rows lie one to a lane, stored to rows that start
// anywhere: turned in shared memory (buf: 4 KiB, 16-byte slot s of row r at
// s ^ (r & 7): no bank conflicts either way), so that a store is a piece of one
// row.  `count` rows from m, the lane's column n.
__device__ __forceinline__ void store_rows_any(const Mat& x, int64_t m, int count, int64_t n, int64_t cols, const float* v,
                                               float4* buf, int lane) {
    float t[32];
#pragma unroll
    for (int s = 0; s < 8; ++s)
        buf[lane * 8 + (s ^ (lane & 7))] = make_float4(v[4 * s], v[4 * s + 1], v[4 * s + 2], v[4 * s + 3]);
    __syncwarp();
    const float* f = reinterpret_cast<const float*>(buf);
#pragma unroll
    for (int r = 0; r < 32; ++r) t[r] = f[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)];
    __syncwarp();
    store_strided<32>(x.p, x.dtype, m * x.ld + n, x.ld, [&](int i) { return n < cols && i < count; }, t);
}

// The epilogue of a chunk whose matrices' rows start anywhere: as finish_row, a
// row to a lane; only the stores go by columns.  All lanes take part.
template <bool SLOPE>
__device__ __forceinline__ void finish_rows_any(const Product& p, int64_t m0, int64_t n, int lane, float bias, float* v,
                                                float4* buf) {
    const int left = static_cast<int>(min(static_cast<int64_t>(32), p.N - n));
    const int count = static_cast<int>(min(static_cast<int64_t>(32), p.M - m0));
    const int64_t m = m0 + lane;
    const bool on = lane < count;
    if (p.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, bias, j);
    }
    if (SLOPE) {
        float z[32];
        if (on) {
            load_row32_any(p.pre, m, n, left, z);
            slope_n<32>(v, z, p.act);
        }
    } else {
        if (p.pre.p != nullptr) {
            if (p.pre.dtype == FSDP_DTYPE_ACT8) {
                if (on) p.pre.e[m * p.pre.eld + (n >> 5)] = static_cast<uint8_t>(store_row32<false>(p.pre, m, n, left, v));
            } else {
                store_rows_any(p.pre, m0, count, n + lane, p.N, v, buf, lane);
            }
        }
        activate_n<32>(v, p.act);
    }
    if (p.add.p != nullptr && on) {
        float e[32];
        load_row32_any(p.add, m, n, left, e);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += e[j];
    }
    store_rows_any(p.out, m0, count, n + lane, p.N, v, buf, lane);
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
// (`count` of them inside the matrix): tiles whose rows are C's columns, and the
// products of few rows.  n - lane is a multiple of 32.
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
