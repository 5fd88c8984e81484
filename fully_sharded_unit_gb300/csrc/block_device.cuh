// Device helpers shared by the block operators: element types, the ACT8
// format and the activations.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "fsdp_unit.h"

namespace fsdp {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats rounded to nearest even, `a` in the low half.
__device__ __forceinline__ uint32_t to_bf16x2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
    return dtype == FSDP_DTYPE_F32 ? static_cast<const float*>(p)[i]
                                   : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void store1(void* p, int dtype, int64_t i, float v) {
    if (dtype == FSDP_DTYPE_F32) static_cast<float*>(p)[i] = v;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void unpack8(uint4 w, float* v) {
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

// Eight elements from a 16-byte boundary.
__device__ __forceinline__ void load8(const void* p, int dtype, int64_t i, float* v) {
    if (dtype == FSDP_DTYPE_F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i), v);
    }
}

__device__ __forceinline__ void store8(void* p, int dtype, int64_t i, const float* v) {
    if (dtype == FSDP_DTYPE_F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
            make_uint4(to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]), to_bf16x2(v[4], v[5]), to_bf16x2(v[6], v[7]));
    }
}

// V elements: 8 from a 16-byte boundary, or 1 from anywhere.
template <int V>
__device__ __forceinline__ void loadv(const void* p, int dtype, int64_t i, float* v) {
    if constexpr (V == 8) load8(p, dtype, i, v);
    else v[0] = load1(p, dtype, i);
}
template <int V>
__device__ __forceinline__ void storev(void* p, int dtype, int64_t i, const float* v) {
    if constexpr (V == 8) store8(p, dtype, i, v);
    else store1(p, dtype, i, v[0]);
}

// ---- ACT8 ----

// The magnitude bits of a float compare like the magnitudes; an infinity or a
// NaN compares above every finite value.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The exponent byte of a group from its largest magnitude's bits: the biased
// exponent itself, at least 7 (so that 2^(6-E) and 2^(E-6) are normal floats).
__device__ __forceinline__ uint32_t act8_byte(uint32_t top) {
    return max(top >> 23, 7u);   // 255 where the group is not finite
}

// 2^(6-E) as a float; 0 for a group that is not finite (its q are then 0 or
// NaN-derived and never read).
__device__ __forceinline__ float act8_scale(uint32_t byte) { return __uint_as_float(byte == 255u ? 0u : (260u - byte) << 23); }

// 2^(E-6); NaN for byte 255.
__device__ __forceinline__ float act8_step(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fc00000u : (max(byte, 7u) - 6u) << 23);
}

// x * 2^(6-E) rounded to nearest even and clamped to +-127, as the low byte of
// the result.  The product is exact (a power of two), so adding 1.5 * 2^23 in
// the same fma rounds it once, at the integers.
__device__ __forceinline__ uint32_t act8_quant(float x, float scale) {
    const float magic = 12582912.0f;
    const float t = fminf(fmaxf(fmaf(x, scale, magic), magic - 127.0f), magic + 127.0f);
    return __float_as_uint(t);
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

__device__ __forceinline__ uint2 act8_quant8(const float* v, float scale) {
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = act8_quant(v[j], scale);
    return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
}

// Four int8 values of a word times `step`: the byte plus 128 goes into the
// mantissa of 2^23, so one subtraction gives the integer exactly.
__device__ __forceinline__ void act8_read4(uint32_t w, float step, float* v) {
    w ^= 0x80808080u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + j)) - 8388736.0f) * step;
}

// V elements of an ACT8 row: payload q, exponent bytes e, column c.
template <int V>
__device__ __forceinline__ void act8_readv(const uint8_t* q, const uint8_t* e, int64_t c, float* v) {
    const float step = act8_step(e[c >> 5]);
    if constexpr (V == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(q + c);
        act8_read4(w.x, step, v);
        act8_read4(w.y, step, v + 4);
    } else {
        v[0] = static_cast<float>(reinterpret_cast<const int8_t*>(q)[c]) * step;
    }
}

// Quantise V consecutive elements per lane; the 32/V lanes that hold a group
// are consecutive and all take part (elements past the row's end are 0).
// Returns the group's exponent byte.
template <int V>
__device__ __forceinline__ uint32_t act8_group_byte(const float* v) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) top = max(top, mag_bits(v[j]));
#pragma unroll
    for (int d = 1; d < 32 / V; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    return act8_byte(top);
}

template <int V>
__device__ __forceinline__ void act8_writev(uint8_t* q, int64_t c, const float* v, uint32_t byte) {
    const float scale = act8_scale(byte);
    if constexpr (V == 8) {
        const uint2 w = act8_quant8(v, scale);
        *reinterpret_cast<uint2*>(q + c) = byte == 255u ? make_uint2(0, 0) : w;
    } else {
        q[c] = byte == 255u ? 0 : static_cast<uint8_t>(act8_quant(v[0], scale));
    }
}

// ---- activations ----

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float kGeluK2 = 1.5957691216057308f;    // 2 sqrt(2/pi)
constexpr float kGeluC = 0.044715f;

// z/2 (1 + tanh(u)) = z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3):
// no cancellation for negative z, and exp's overflow gives the limit 0.
__device__ __forceinline__ float gelu_tanh(float z) {
    const float u2 = z * fmaf(kGeluK2 * kGeluC * z, z, kGeluK2);
    return __fdividef(z, 1.0f + __expf(-u2));
}

// s + z s (1 - s) (2u)', s = 1 / (1 + exp(-2u)).  Past +-30 the slope is 1 or
// 0 exactly; the clamp keeps z^2 finite.
__device__ __forceinline__ float gelu_tanh_slope(float z) {
    z = min_nan(max_nan(z, -30.0f), 30.0f);
    const float zz = z * z;
    const float u2 = z * fmaf(kGeluK2 * kGeluC, zz, kGeluK2);
    const float s = __fdividef(1.0f, 1.0f + __expf(-u2));
    return fmaf(z * fmaf(3.0f * kGeluK2 * kGeluC, zz, kGeluK2), s - s * s, s);
}

__device__ __forceinline__ float gelu_erf(float z) { return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f)); }

__device__ __forceinline__ float gelu_erf_slope(float z) {
    z = min_nan(max_nan(z, -30.0f), 30.0f);
    return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), 0.5f * (1.0f + erff(z * 0.70710678118654752f)));
}

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case FSDP_ACTIVATION_RELU: return max_nan(z, 0.0f);
        case FSDP_ACTIVATION_GELU_TANH: return gelu_tanh(z);
        case FSDP_ACTIVATION_GELU_ERF: return gelu_erf(z);
        default: return z;
    }
}

__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
        case FSDP_ACTIVATION_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case FSDP_ACTIVATION_GELU_TANH: return gelu_tanh_slope(z);
        case FSDP_ACTIVATION_GELU_ERF: return gelu_erf_slope(z);
        default: return 1.0f;
    }
}

}  // namespace fsdp
