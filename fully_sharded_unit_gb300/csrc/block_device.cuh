// Device helpers shared by the block operators: element types, the ACT8
// format and the activations.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "fsdp_unit.h"

namespace fsdp {

// See launch_early in compute.hpp.
__device__ __forceinline__ void starts_early() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// N elements `stride` apart, or 0 where on(i) is false.  The type is looked at
// once, outside the loop: with a branch in it, each load would wait for the one
// before.
template <int N, typename On>
__device__ __forceinline__ void load_strided(const void* p, int dtype, int64_t i, int64_t stride, On on, float* v) {
    if (dtype == FSDP_DTYPE_F32) {
        const float* s = static_cast<const float*>(p) + i;
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = on(j) ? s[j * stride] : 0.0f;
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(p) + i;
        uint32_t w[N];
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = on(j) ? s[j * stride] : 0u;
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = __uint_as_float(w[j] << 16);
    }
}

template <int N, typename On>
__device__ __forceinline__ void store_strided(void* p, int dtype, int64_t i, int64_t stride, On on, const float* v) {
    if (dtype == FSDP_DTYPE_F32) {
        float* s = static_cast<float*>(p) + i;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (on(j)) s[j * stride] = v[j];
    } else {
        __nv_bfloat16* s = static_cast<__nv_bfloat16*>(p) + i;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (on(j)) s[j * stride] = __float2bfloat16_rn(v[j]);
    }
}

// Chunks of eight, `stride` elements apart, from 16-byte boundaries.
template <int N, typename On>
__device__ __forceinline__ void load_chunks(const void* p, int dtype, int64_t i, int64_t stride, On on, float (*v)[8]) {
    if (dtype == FSDP_DTYPE_F32) {
        const float* s = static_cast<const float*>(p) + i;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float4 a = make_float4(0, 0, 0, 0), b = a;
            if (on(j)) {
                a = reinterpret_cast<const float4*>(s + j * stride)[0];
                b = reinterpret_cast<const float4*>(s + j * stride)[1];
            }
            v[j][0] = a.x; v[j][1] = a.y; v[j][2] = a.z; v[j][3] = a.w;
            v[j][4] = b.x; v[j][5] = b.y; v[j][6] = b.z; v[j][7] = b.w;
        }
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(p) + i;
        uint4 w[N];
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = on(j) ? *reinterpret_cast<const uint4*>(s + j * stride) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < N; ++j) unpack8(w[j], v[j]);
    }
}

// ---- rows that start anywhere ----

// `bytes` bytes from an address that is aligned to its elements only, as words: the
// 16-byte words that hold them (each read only if it holds one), moved together by
// the address's offset.  What lies past `bytes` in w is not defined.
template <int WORDS>
__device__ __forceinline__ void load_window(uintptr_t from, int bytes, uint32_t* w) {
    const uintptr_t word = from & ~uintptr_t(15);
    const int end = bytes > 0 ? static_cast<int>(from & 15) + bytes : 0;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (16 * i < end) a = *reinterpret_cast<const uint4*>(word + 16 * i);
        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
    }
    if (from & 8) {
#pragma unroll
        for (int i = 0; i + 2 < 4 * WORDS; ++i) w[i] = w[i + 2];
    }
    if (from & 4) {
#pragma unroll
        for (int i = 0; i + 1 < 4 * WORDS; ++i) w[i] = w[i + 1];
    }
    if (from & 2) {
#pragma unroll
        for (int i = 0; i + 1 < 4 * WORDS; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
}

// The reverse: `bytes` (at most 16 N) of the words in v to an address that is
// aligned to its elements only, in whole 16-byte words where the address allows
// it.  `joined`: the lane before stores the 16 N bytes that end where this lane's
// begin, so that this lane's first word takes their end along.  What is left at
// the ends of such a run goes two bytes at a time.  All lanes take part.
template <int N>
__device__ __forceinline__ void store_window(uintptr_t to, int bytes, bool joined, const uint32_t* v) {
    const bool next = __shfl_down_sync(0xffffffffu, static_cast<int>(joined), 1) != 0 && (threadIdx.x & 31) != 31;
    uint32_t w[4 * N + 8];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, v[4 * N - 4 + i], 1);
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) w[4 + i] = v[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * N + 4 + i] = 0;
    // w holds the bytes from to - 16 on: brought to those from the word below `to`
    const uint32_t shift = 16 - static_cast<uint32_t>(to & 15);
    if (shift & 16) {
#pragma unroll
        for (int i = 0; i < 4 * N + 4; ++i) w[i] = w[i + 4];
    }
    if (shift & 8) {
#pragma unroll
        for (int i = 0; i < 4 * N + 4; ++i) w[i] = w[i + 2];
    }
    if (shift & 4) {
#pragma unroll
        for (int i = 0; i < 4 * N + 4; ++i) w[i] = w[i + 1];
    }
    if (shift & 2) {
#pragma unroll
        for (int i = 0; i < 4 * N + 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    uint8_t* const base = reinterpret_cast<uint8_t*>(to & ~uintptr_t(15));
    const int skip = static_cast<int>(to & 15), end = skip + bytes, first = joined ? 0 : skip;
#pragma unroll
    for (int i = 0; i <= N; ++i) {
        if (16 * i >= first && 16 * i + 16 <= end) {
            reinterpret_cast<uint4*>(base)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if (16 * i < end && bytes > 0 && !(next && 16 * i + 16 > end)) {
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (16 * i + 2 * h >= first && 16 * i + 2 * h < end)
                    reinterpret_cast<uint16_t*>(base)[8 * i + h] = static_cast<uint16_t>(w[4 * i + h / 2] >> (16 * (h & 1)));
        }
    }
}

// How many of the eight columns from c on are inside a row of `cols`.
__device__ __forceinline__ int inside8(int64_t c, int64_t cols) {
    return static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(8), cols - c)));
}

// Chunks of eight columns `stride` elements apart, n[k] of them inside the row
// (see inside8); the others are 0.
template <int N>
__device__ __forceinline__ void load_chunks_any(const void* p, int dtype, int64_t i, const int* n, int64_t stride, float (*v)[8]) {
    if (dtype == FSDP_DTYPE_F32) {
        uint32_t w[N][12];
#pragma unroll
        for (int k = 0; k < N; ++k)
            load_window<3>(reinterpret_cast<uintptr_t>(static_cast<const float*>(p) + i + k * stride), n[k] * 4, w[k]);
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = j < n[k] ? __uint_as_float(w[k][j]) : 0.0f;
    } else {
        uint32_t w[N][8];
#pragma unroll
        for (int k = 0; k < N; ++k)
            load_window<2>(reinterpret_cast<uintptr_t>(static_cast<const uint16_t*>(p) + i + k * stride), n[k] * 2, w[k]);
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = j < n[k] ? (j & 1 ? bf16_hi(w[k][j / 2]) : bf16_lo(w[k][j / 2])) : 0.0f;
    }
}

// The reverse, one chunk; the lane before holds the chunk before.  All lanes take part.
__device__ __forceinline__ void store_chunk_any(void* p, int dtype, int64_t i, int n, const float* v) {
    const bool joined = n > 0 && (threadIdx.x & 31) != 0;
    if (dtype == FSDP_DTYPE_F32) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[j]);
        store_window<2>(reinterpret_cast<uintptr_t>(static_cast<float*>(p) + i), n * 4, joined, w);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = to_bf16x2(v[2 * j], v[2 * j + 1]);
        store_window<1>(reinterpret_cast<uintptr_t>(static_cast<uint16_t*>(p) + i), n * 2, joined, w);
    }
}

// ---- pairs of floats in one 64-bit register (one instruction for both) ----

using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(f32x2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {   // 2^x, relative error about 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {   // 1/x to an ulp; 1/inf = 0
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 32 bytes from a 32-byte boundary.
__device__ __forceinline__ void load32b(const void* p, uint32_t* w) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void store32b(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// ---- clusters of blocks ----

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}

// The same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// A barrier of the cluster for what the first warp has stored in the other blocks' shared memory.
// The other warps do not wait for their own stores to global memory to be complete.  Warps arrive whole:
// lanes of one that arrived in different branches would wait for one another.
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    if (threadIdx.x < 32) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    else asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ---- ACT8 ----

// Larger magnitude of the two, as a non-negative float; NaN if either is.  Its
// bits order like the magnitudes, an infinity's and a NaN's above all others.
__device__ __forceinline__ float larger(float top, float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(x)));
    return r;
}

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

// x * 2^(6-E) rounded to nearest even (and clamped to +-127), as the low byte
// of the result.  The product is exact (a power of two), so adding 1.5 * 2^23
// in the same fma rounds it once, at the integers.
constexpr float kMagic = 12582912.0f;
__device__ __forceinline__ uint32_t act8_quant(float x, float scale) {
    return __float_as_uint(fminf(fmaxf(fmaf(x, scale, kMagic), kMagic - 127.0f), kMagic + 127.0f));
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// N/4 words of N values whose largest magnitude has the bits `top`.  Only a
// group whose largest value rounds to 128 steps needs the clamp (one in a few
// hundred), so the others leave its two instructions an element out.
template <int N>
__device__ __forceinline__ void act8_quant_n(const float* v, uint32_t top, float scale, uint32_t* w) {
    if (__uint_as_float(top) * scale < 127.5f) {
        const f32x2 s = pair(scale, scale), m = pair(kMagic, kMagic);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            float a, b, c, d;
            unpair(fma2(pair(v[4 * i], v[4 * i + 1]), s, m), a, b);
            unpair(fma2(pair(v[4 * i + 2], v[4 * i + 3]), s, m), c, d);
            w[i] = pack4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
        }
    } else {   // also a group that is not finite: its scale is 0 and its words become 0
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = scale == 0.0f ? 0u
                                 : pack4(act8_quant(v[4 * i], scale), act8_quant(v[4 * i + 1], scale),
                                         act8_quant(v[4 * i + 2], scale), act8_quant(v[4 * i + 3], scale));
    }
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

// The bits of the largest magnitude of a group whose V consecutive elements lie
// in each of 32/V consecutive lanes, which all take part (elements past the
// row's end are 0).
template <int V>
__device__ __forceinline__ uint32_t act8_group_top(const float* v) {
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) most = larger(most, v[j]);
    uint32_t top = __float_as_uint(most);
    if constexpr (V == 1) {
        top = __reduce_max_sync(0xffffffffu, top);
    } else {
#pragma unroll
        for (int d = 1; d < 32 / V; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    return top;
}

// V elements into the payload, at column c of the row at q.
template <int V>
__device__ __forceinline__ void act8_writev(uint8_t* q, int64_t c, const float* v, uint32_t top) {
    const float scale = act8_scale(act8_byte(top));
    if constexpr (V == 8) {
        uint32_t w[2];
        act8_quant_n<8>(v, top, scale, w);
        *reinterpret_cast<uint2*>(q + c) = make_uint2(w[0], w[1]);
    } else {
        q[c] = scale == 0.0f ? 0 : static_cast<uint8_t>(act8_quant(v[0], scale));
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
constexpr float kLog2e = 1.4426950408889634f;

// z/2 (1 + tanh(u)) = z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3):
// no cancellation for negative z, and exp's overflow gives the limit 0.  Two
// elements at a time: five packed instructions and four on the special-function
// units, which bound it (16 lanes a cycle an SM).  Rounding: with s = 1 / (1 + e) an
// error d of e's exponent moves s by s (1 - s) d, at most d/4; exp2's own (2^-22) and
// that of its argument (2^-24 of it) give 2^-23, the reciprocal's ulp 2^-23 and the
// last product 2^-24: below 2^-21 |z| together, also where the result is F32.
__device__ __forceinline__ void gelu_tanh2(float& z0, float& z1) {
    const f32x2 z = pair(z0, z1);
    const f32x2 t = fma2(mul2(z, z), pair(-kLog2e * kGeluK2 * kGeluC, -kLog2e * kGeluK2 * kGeluC),
                         pair(-kLog2e * kGeluK2, -kLog2e * kGeluK2));
    float a, b;
    unpair(mul2(z, t), a, b);
    unpair(add2(pair(exp2_fast(a), exp2_fast(b)), pair(1.0f, 1.0f)), a, b);
    unpair(mul2(z, pair(rcp_fast(a), rcp_fast(b))), z0, z1);
}

// s + z (s - s^2) (2u)', s = 1 / (1 + exp(-2u)).  Where s is an ulp (2^-24) off 1,
// at |z| up to 5.2, s - s^2 is off by as much and its factor is up to 38: an error
// of up to 2^-18 there, as in any fp32 form that has s or tanh.  z^2 is held at 900 so that it
// stays finite: past |z| = 30, s is 0 or 1 exactly.
__device__ __forceinline__ void gelu_tanh_slope2(float z0, float z1, float& d0, float& d1) {
    const f32x2 z = pair(z0, z1);
    float a, b;
    unpair(mul2(z, z), a, b);
    const f32x2 zz = pair(min_nan(a, 900.0f), min_nan(b, 900.0f));
    const f32x2 t = fma2(zz, pair(-kLog2e * kGeluK2 * kGeluC, -kLog2e * kGeluK2 * kGeluC),
                         pair(-kLog2e * kGeluK2, -kLog2e * kGeluK2));
    unpair(mul2(z, t), a, b);
    unpair(add2(pair(exp2_fast(a), exp2_fast(b)), pair(1.0f, 1.0f)), a, b);
    const f32x2 s = pair(rcp_fast(a), rcp_fast(b));
    const f32x2 rise = fma2(zz, pair(3.0f * kGeluK2 * kGeluC, 3.0f * kGeluK2 * kGeluC), pair(kGeluK2, kGeluK2));
    const f32x2 fall = fma2(mul2(s, pair(-1.0f, -1.0f)), s, s);
    unpair(fma2(mul2(z, rise), fall, s), d0, d1);
}

__device__ __forceinline__ float gelu_tanh(float z) {
    float other = 0.0f;
    gelu_tanh2(z, other);
    return z;
}

__device__ __forceinline__ float gelu_tanh_slope(float z) {
    float d, other;
    gelu_tanh_slope2(z, 0.0f, d, other);
    return d;
}

__device__ __forceinline__ float gelu_erf(float z) { return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f)); }

// __expf: its error, 2^-22 and 2^-23 |z^2/2| of the result, is below 2^-22 of the slope's size.
__device__ __forceinline__ float gelu_erf_slope(float z) {
    z = min_nan(max_nan(z, -30.0f), 30.0f);
    return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), 0.5f * (1.0f + erff(z * 0.70710678118654752f)));
}

// N elements in place; the kind is looked at once.
template <int N>
__device__ __forceinline__ void activate_n(float* v, int act) {
    if (act == FSDP_ACTIVATION_GELU_TANH) {
        if constexpr (N % 2 == 0) {
#pragma unroll
            for (int j = 0; j < N; j += 2) gelu_tanh2(v[j], v[j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = gelu_tanh(v[j]);
        }
    } else if (act == FSDP_ACTIVATION_GELU_ERF) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = gelu_erf(v[j]);
    } else if (act == FSDP_ACTIVATION_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = max_nan(v[j], 0.0f);
    }
}

// v *= slope(z), N elements.
template <int N>
__device__ __forceinline__ void slope_n(float* v, const float* z, int act) {
    if (act == FSDP_ACTIVATION_GELU_TANH) {
        if constexpr (N % 2 != 0) v[N - 1] *= gelu_tanh_slope(z[N - 1]);
#pragma unroll
        for (int j = 0; j + 1 < N; j += 2) {
            float a, b;
            gelu_tanh_slope2(z[j], z[j + 1], a, b);
            v[j] *= a;
            v[j + 1] *= b;
        }
    } else if (act == FSDP_ACTIVATION_GELU_ERF) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] *= gelu_erf_slope(z[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = z[j] > 0.0f ? v[j] : v[j] * 0.0f;
    }
}

}  // namespace fsdp
