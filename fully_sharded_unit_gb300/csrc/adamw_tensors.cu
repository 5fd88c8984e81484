// AdamW over many tensors in one launch, with moments in 32 or 8 bits, and 8-bit moments
// from and to floats.
#include <algorithm>
#include <cmath>

#include "adamw.hpp"
#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---- 8-bit moments ----
//
// With the group's exponent byte B, |x| 2^(127-B) is below 2.  Scaled down once more, by a
// power of two that puts the smallest exponent of the 8 bits at fp32's subnormal
// numbers, the code is the upper bits of that float: cutting its 20 low bits off
// (after adding what rounds them) gives codes of normal and subnormal small floats
// alike, and the reverse reads them.

template <bool SIGNED>
constexpr float kDown = SIGNED ? 0x1p-112f : 0x1p-96f;
template <bool SIGNED>
constexpr float kUp = SIGNED ? 0x1p112f : 0x1p96f;
constexpr uint32_t kNearest = 0x100000u;   // `random` for rounding to nearest even

// The exponent byte from the bits of the group's largest magnitude: the exponent, one more
// where the mantissa is above 1.875, so that rounding up does not leave the codes.
__device__ __forceinline__ uint32_t state8_byte(uint32_t top) {
    return top >= 0x7f800000u ? 255u : min(max((top + 0xfffffu) >> 23, 1u), 253u);
}

template <bool SIGNED>
__device__ __forceinline__ uint32_t state8_code(float x, uint32_t byte, uint32_t random) {
    if (byte == 255u) return 0;
    const float away = __uint_as_float((254u - byte) << 23);   // 2^(127-B)
    const float y = (SIGNED ? fabsf(x) : fmaxf(x, 0.0f)) * away;
    uint32_t b, r = random;
    if (random == kNearest) {   // cut off, and what that lost moves a half up: one rounding in all
        const float cut = __fmul_rz(y, kDown<SIGNED>);
        b = __float_as_uint(cut);
        r = 0x7ffffu + (((b >> 20) & 1u) | (cut * kUp<SIGNED> != y ? 1u : 0u));
    } else {
        b = __float_as_uint(y * kDown<SIGNED>);
    }
    uint32_t code = min((b + r) >> 20, SIGNED ? 0x7fu : 0xffu);
    if (SIGNED) return code != 0 ? code | ((__float_as_uint(x) >> 24) & 0x80u) : 0u;
    return x > 0.0f ? max(code, 1u) : 0u;
}

// What is added below a code, of its 32 random bits: 16 of 20.
template <bool SIGNED>
__device__ __forceinline__ uint32_t below(uint32_t r) { return (SIGNED ? r << 4 : r >> 12) & 0xffff0u; }

// The code where value and random bits add up to a code exactly (one in 2^20): as the plain form in
// 64 bits has it (perf/more_operators.py), |x| pow(2, 127-B) in codes' steps and r / 2^16 cut off.  Where CUDA's pow is
// an ulp low (2^11 is) that leaves the sum below the code, which with 16 random bits is as near in the mean.  The
// sum in whole numbers is that code, and takes 2.30 ms for 708 M elements instead of 2.51, but 545 codes of 236 M then differ
// from the plain form's, and 460 of the next step's parameters by up to 4 % of their root mean square.  Not worth
// registers in the kernels.
template <bool SIGNED>
__device__ __noinline__ uint32_t state8_code64(float x, uint32_t byte, uint32_t added) {
    const int low = SIGNED ? -14 : -30;
    const double y = static_cast<double>(SIGNED ? fabsf(x) : fmaxf(x, 0.0f)) * pow(2.0, 127.0 - static_cast<double>(byte));
    int e = 0;
    frexp(y, &e);
    e = y > 0.0 ? max(e - 1, low) : low;
    const double k = floor(y * pow(2.0, static_cast<double>(3 - e)) + static_cast<double>(added) * 0x1p-20);
    const uint32_t code = min(static_cast<uint32_t>(static_cast<int>(k) + ((e - low) << 3)), SIGNED ? 0x7fu : 0xffu);
    if (SIGNED) return code != 0 ? code | ((__float_as_uint(x) >> 24) & 0x80u) : 0u;
    return x > 0.0f ? max(code, 1u) : 0u;
}

// state8_code for random bits.
template <bool SIGNED>
__device__ __forceinline__ uint32_t state8_random_code(float x, uint32_t byte, uint32_t r) {
    if (byte == 255u) return 0;
    const float away = __uint_as_float((254u - byte) << 23);
    const uint32_t added = below<SIGNED>(r);
    const uint32_t sum = __float_as_uint((SIGNED ? fabsf(x) : fmaxf(x, 0.0f)) * away * kDown<SIGNED>) + added;
    return (sum & 0xfffffu) == 0 ? state8_code64<SIGNED>(x, byte, added) : state8_code<SIGNED>(x, byte, added);
}

// 2^(B-127); NaN for byte 255, 0 for byte 0.
__device__ __forceinline__ float state8_unit(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

template <bool SIGNED>
__device__ __forceinline__ float state8_value(uint32_t code, float unit) {
    const float f = __uint_as_float((SIGNED ? code & 0x7fu : code) << 20) * kUp<SIGNED> * unit;
    return SIGNED && (code & 0x80u) ? -f : f;
}

// Eight codes of one group.  Up to an exponent byte of kPlain the two scalings of a value are one
// multiplication by a normal or subnormal power of two, and no code needs its limit; larger
// groups (magnitudes from 2^15) take the steps one by one.
constexpr uint32_t kPlain = 142;

template <bool SIGNED>
__device__ __forceinline__ void state8_values(uint2 w, uint32_t byte, float* v) {
    if (byte <= kPlain) {
        const float by = byte == 0 ? 0.0f : __uint_as_float((byte + (SIGNED ? 112u : 96u)) << 23);
        const f32x2 by2 = pair(by, by);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            uint32_t b[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // the code as the float's top byte, then where it belongs
                const uint32_t top = __byte_perm(j < 4 ? w.x : w.y, 0, (((j + h) & 3) << 12) | 0x0444);
                b[h] = SIGNED ? static_cast<uint32_t>(static_cast<int32_t>(top) >> 4) & 0x87ffffffu : top >> 4;
            }
            unpair(mul2(pair(__uint_as_float(b[0]), __uint_as_float(b[1])), by2), v[j], v[j + 1]);
        }
    } else {
        const float unit = state8_unit(byte);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = state8_value<SIGNED>(((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 0xffu, unit);
    }
}

// Four words' top bytes.
__device__ __forceinline__ uint32_t top_bytes(const uint32_t* t) {
    return __byte_perm(__byte_perm(t[0], t[1], 0x0073), __byte_perm(t[2], t[3], 0x0073), 0x5410);
}

// Eight codes one by one, out of the way of the kernels' registers.
struct Eight {
    float x[8];
    uint32_t random[8];
};
template <bool SIGNED>
__device__ __noinline__ uint2 state8_codes_slow(Eight e, uint32_t byte) {
    uint32_t w[2] = {0, 0};
#pragma unroll 1
    for (int j = 0; j < 8; ++j) w[j >> 2] |= state8_random_code<SIGNED>(e.x[j], byte, e.random[j]) << (8 * (j & 3));
    return make_uint2(w[0], w[1]);
}

// `random`: the elements' 32 bits.
template <bool SIGNED>
__device__ __forceinline__ uint2 state8_codes(const float* x, uint32_t byte, const uint32_t* random) {
    uint32_t w[2] = {0, 0};
    if (byte <= kPlain) {
        // 2^(15-B) or 2^(31-B): 2^-127 at the least, a subnormal number
        const int e = (SIGNED ? 142 : 158) - static_cast<int>(byte);
        const float by = __uint_as_float(e > 0 ? static_cast<uint32_t>(e) << 23 : 0x400000u);
        const f32x2 by2 = pair(by, by);
        uint32_t least = 0xffffffu;   // of what is below the codes: 0 for a sum that is a code exactly
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t t[4];
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const int i = 4 * q + j;
                float a, b;
                unpair(mul2(pair(x[i], x[i + 1]), by2), a, b);
                const uint32_t mask = SIGNED ? 0x7fffffffu : 0xffffffffu;
                t[j] = (__float_as_uint(a) & mask) + below<SIGNED>(random[i]);
                t[j + 1] = (__float_as_uint(b) & mask) + below<SIGNED>(random[i + 1]);
                least = min(least, min(t[j] & 0xfffffu, t[j + 1] & 0xfffffu));
                if (!SIGNED) {   // an element that is not 0 is at least the first code
                    t[j] = max(t[j], x[i] > 0.0f ? 0x100000u : 0u);
                    t[j + 1] = max(t[j + 1], x[i + 1] > 0.0f ? 0x100000u : 0u);
                }
                t[j] <<= 4;
                t[j + 1] <<= 4;
            }
            w[q] = top_bytes(t);
            if (SIGNED) {   // the sign, of codes that are not 0
                uint32_t b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(x[4 * q + j]);
                w[q] |= top_bytes(b) & (w[q] + 0x7f7f7f7fu) & 0x80808080u;
            }
        }
        if (least != 0) return make_uint2(w[0], w[1]);
    }
    Eight e;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        e.x[j] = x[j];
        e.random[j] = random[j];
    }
    return state8_codes_slow<SIGNED>(e, byte);
}

__device__ __forceinline__ float magnitude(float x, bool is_signed) { return is_signed ? x : max_nan(x, 0.0f); }

// A group to a warp, an element to a lane: 100 M elements 246 us, 2.0 TB/s.  (A checkpoint's read, not a step's.)
template <bool SIGNED>
__global__ void __launch_bounds__(256) state8_pack_kernel(const float* x, int64_t n, uint8_t* codes, uint8_t* exps) {
    starts_early();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t g = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); g * 32 < n; g += stride) {
        const int64_t i = g * 32 + lane;
        const float v = i < n ? x[i] : 0.0f;
        const uint32_t byte = state8_byte(__reduce_max_sync(kAll, __float_as_uint(larger(0.0f, magnitude(v, SIGNED)))));
        if (i < n) codes[i] = static_cast<uint8_t>(state8_code<SIGNED>(v, byte, kNearest));
        if (lane == 0) exps[g] = static_cast<uint8_t>(byte);
    }
}

// 708 M elements to BF16: 343 us, 6.3 TB/s.
template <bool SIGNED>
__global__ void __launch_bounds__(256) state8_unpack_kernel(const uint8_t* codes, const uint8_t* exps, int64_t n, void* out, int dtype,
                                                            bool vector) {
    starts_early();
    after_previous();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256, first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t eights = vector ? n / 8 : 0;
    for (int64_t q = first; q < eights; q += stride) {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + q * 8);
        float v[8];
        state8_values<SIGNED>(w, exps[q >> 2], v);
        store8(out, dtype, q * 8, v);
    }
    for (int64_t i = eights * 8 + first; i < n; i += stride) store1(out, dtype, i, state8_value<SIGNED>(codes[i], state8_unit(exps[i >> 5])));
}

// ---- AdamW ----

struct Tensor {
    float* p;
    const void* g;
    void* m;
    void* v;
    uint8_t* me;
    uint8_t* ve;
    uint16_t* copy;
    int64_t n;
    float decay, step;
    uint32_t key;
    uint32_t first;      // tile
    int grad_dtype;
    int vector;
};

// Elements of a tile, which a block takes at a time: few for little work, so that it spreads (its latency
// is that of a thread's passes over the tile), many for a lot, so that finding a tile's tensor counts little.
constexpr int kLeastTile = 256, kMostTile32 = 2048, kMostTile8 = 16384;
constexpr int kFew = 16, kTensors = 256;   // tensors of one launch, in the kernel's parameters

template <int MOST>
struct Tensors {
    AdamWConsts c;               // decay and step: the tensor's
    const float* grad_scale;
    const int32_t* skip;
    uint32_t count, tiles;
    int tile;                    // elements of one
    Tensor t[MOST];
};

// i's part of what is hashed; of i + j, j < 8 with i a multiple of 8, it is that ^ j.
__device__ __forceinline__ uint32_t random_input(int64_t i, uint32_t key) {
    return static_cast<uint32_t>(i) ^ key ^ static_cast<uint32_t>(i >> 32) * 0x85157AF5u;
}
__device__ __forceinline__ uint32_t random_bits(uint32_t x) {
    x ^= x >> 16;
    x *= 0xD36F86A9u;
    x ^= x >> 15;
    x *= 0xC242E759u;
    return x ^ (x >> 16);
}

// adamw_elem for two elements beside one another: the same operations, each rounded by itself, the
// products in one instruction for both.  The sums are scalar: the compiler joins an add2 with
// the mul2 before it into one rounding.
__device__ __forceinline__ void adamw_pair(float* p, const float* g, float* m, float* v, const AdamWConsts& c) {
    const f32x2 g2 = pair(g[0], g[1]);
    float pd[2], om[2], gm[2], ov[2], gv[2], q[2];
    unpair(mul2(pair(p[0], p[1]), pair(c.decay, c.decay)), pd[0], pd[1]);
    unpair(mul2(pair(m[0], m[1]), pair(c.b1, c.b1)), om[0], om[1]);
    unpair(mul2(g2, pair(c.c1, c.c1)), gm[0], gm[1]);
    unpair(mul2(pair(v[0], v[1]), pair(c.b2, c.b2)), ov[0], ov[1]);
    unpair(mul2(mul2(g2, g2), pair(c.c2, c.c2)), gv[0], gv[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        m[j] = __fadd_rn(om[j], gm[j]);
        v[j] = __fadd_rn(ov[j], gv[j]);
        q[j] = __fdiv_rn(m[j], __fadd_rn(__fsqrt_rn(__fdiv_rn(v[j], c.bc2)), c.eps));
    }
    unpair(mul2(pair(q[0], q[1]), pair(c.step, c.step)), q[0], q[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) p[j] = __fsub_rn(pd[j], q[j]);
}

// The last tensor whose first tile is at or before `tile`.
template <int MOST>
__device__ __forceinline__ uint32_t tensor_of(const Tensors<MOST>& a, uint32_t tile) {
    uint32_t lo = 0, hi = a.count;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (a.t[mid].first <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Eight elements of a tensor whose pointers allow vector accesses; the four threads
// beside one another that have a group of 32 take part together (`n` of a thread's elements are
// the tensor's, and may be none).
template <bool EIGHT>
__device__ __forceinline__ void step8(const Tensor& t, const AdamWConsts& c, bool scaled, float scale, int64_t i, int n) {
    float p[8], g[8], m[8], v[8];
    uint2 cm = make_uint2(0, 0), cv = cm;
    uint32_t em = 0, ev = 0;
    if (n == 8) {
        load8(t.p, FSDP_DTYPE_F32, i, p);
        load8(t.g, t.grad_dtype, i, g);
        if (EIGHT) {
            cm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i);
            cv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i);
        } else {
            load8(t.m, FSDP_DTYPE_F32, i, m);
            load8(t.v, FSDP_DTYPE_F32, i, v);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool on = j < n;
            p[j] = on ? t.p[i + j] : 0.0f;
            g[j] = on ? load1(t.g, t.grad_dtype, i + j) : 0.0f;
            if (EIGHT) {
                uint32_t& wm = j < 4 ? cm.x : cm.y;
                uint32_t& wv = j < 4 ? cv.x : cv.y;
                wm |= on ? static_cast<uint32_t>(static_cast<const uint8_t*>(t.m)[i + j]) << (8 * (j & 3)) : 0u;
                wv |= on ? static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[i + j]) << (8 * (j & 3)) : 0u;
            } else {
                m[j] = on ? static_cast<const float*>(t.m)[i + j] : 0.0f;
                v[j] = on ? static_cast<const float*>(t.v)[i + j] : 0.0f;
            }
        }
    }
    if (EIGHT) {
        if (n > 0) {
            em = t.me[i >> 5];
            ev = t.ve[i >> 5];
        }
        state8_values<true>(cm, em, m);
        state8_values<false>(cv, ev, v);
    }
    if (scaled) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(g[j], scale);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) adamw_pair(p + j, g + j, m + j, v + j, c);
    if (n == 8) {
        store8(t.p, FSDP_DTYPE_F32, i, p);
        if (t.copy != nullptr) store8(t.copy, FSDP_DTYPE_BF16, i, p);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= n) continue;
            t.p[i + j] = p[j];
            if (t.copy != nullptr) store1(t.copy, FSDP_DTYPE_BF16, i + j, p[j]);
        }
    }
    if (EIGHT) {
        if (n < 8) {   // what is not the tensor's stays out of the groups' largest
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= n) m[j] = v[j] = 0.0f;
        }
        float mt = 0.0f, vt = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            mt = larger(mt, m[j]);
            vt = larger(vt, v[j]);
        }
        uint32_t mb = __float_as_uint(mt), vb = __float_as_uint(vt);
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            mb = max(mb, __shfl_xor_sync(kAll, mb, d));
            vb = max(vb, __shfl_xor_sync(kAll, vb, d));
        }
        mb = state8_byte(mb);
        vb = state8_byte(vb);
        const uint32_t input = random_input(i, t.key);
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = random_bits(input ^ j);
        cm = state8_codes<true>(m, mb, r);
        cv = state8_codes<false>(v, vb, r);
        if (n > 0 && (i & 31) == 0) {
            t.me[i >> 5] = static_cast<uint8_t>(mb);
            t.ve[i >> 5] = static_cast<uint8_t>(vb);
        }
    }
    if (n == 8) {
        if (EIGHT) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i) = cm;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i) = cv;
        } else {
            store8(t.m, FSDP_DTYPE_F32, i, m);
            store8(t.v, FSDP_DTYPE_F32, i, v);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= n) continue;
            if (EIGHT) {
                static_cast<uint8_t*>(t.m)[i + j] = static_cast<uint8_t>((j < 4 ? cm.x : cm.y) >> (8 * (j & 3)));
                static_cast<uint8_t*>(t.v)[i + j] = static_cast<uint8_t>((j < 4 ? cv.x : cv.y) >> (8 * (j & 3)));
            } else {
                static_cast<float*>(t.m)[i + j] = m[j];
                static_cast<float*>(t.v)[i + j] = v[j];
            }
        }
    }
}

// The same for tensors that begin anywhere: a group of 32 to a warp, an element to a lane.
template <bool EIGHT>
__device__ __forceinline__ void step1(const Tensor& t, const AdamWConsts& c, bool scaled, float scale, int64_t i, bool on) {
    float p = on ? t.p[i] : 0.0f, g = on ? load1(t.g, t.grad_dtype, i) : 0.0f, m = 0.0f, v = 0.0f;
    if (scaled) g = __fmul_rn(g, scale);
    if (on) {
        if (EIGHT) {
            m = state8_value<true>(static_cast<uint8_t*>(t.m)[i], state8_unit(t.me[i >> 5]));
            v = state8_value<false>(static_cast<uint8_t*>(t.v)[i], state8_unit(t.ve[i >> 5]));
        } else {
            m = static_cast<float*>(t.m)[i];
            v = static_cast<float*>(t.v)[i];
        }
    }
    adamw_elem(p, g, m, v, c);
    if (on) {
        t.p[i] = p;
        if (t.copy != nullptr) store1(t.copy, FSDP_DTYPE_BF16, i, p);
    }
    if (EIGHT) {
        const uint32_t r = random_bits(random_input(i, t.key));
        const uint32_t mb = state8_byte(__reduce_max_sync(kAll, on ? __float_as_uint(larger(0.0f, m)) : 0u));
        const uint32_t vb = state8_byte(__reduce_max_sync(kAll, on ? __float_as_uint(larger(0.0f, v)) : 0u));
        if (on) {
            static_cast<uint8_t*>(t.m)[i] = static_cast<uint8_t>(state8_random_code<true>(m, mb, r));
            static_cast<uint8_t*>(t.v)[i] = static_cast<uint8_t>(state8_random_code<false>(v, vb, r));
        }
        if ((i & 31) == 0) {
            t.me[i >> 5] = static_cast<uint8_t>(mb);
            t.ve[i >> 5] = static_cast<uint8_t>(vb);
        }
    } else if (on) {
        static_cast<float*>(t.m)[i] = m;
        static_cast<float*>(t.v)[i] = v;
    }
}

// EIGHT: moments in 8 bits.  A block takes tiles in turn.  236 M elements, 32 bits, with BF16 copies: 1.16 ms,
// 6.1 TB/s.  708 M, 8 bits, BF16 gradients and copies: 2.50 ms, 4.6 TB/s, bound by issue (3.0 of 4 a
// cycle): 103 instructions an element, a third of them the two divisions and the root, rounded as IEEE has
// them.  Fp32 moments owe that to the unit's bits; 8-bit ones share the code.  (Four blocks an SM: with three or
// five, and 80 or 48 registers, 0.3 ms more.)  Tensors that begin anywhere, an element to a lane: 100 M elements
// 0.71 ms against 0.49, and in 8 bits 1.19 against 0.36.
template <bool EIGHT, int MOST>
__global__ void __launch_bounds__(256, 4) adamw_tensors_kernel(const __grid_constant__ Tensors<MOST> a) {
    starts_early();
    after_previous();
    if (a.skip != nullptr && *a.skip != 0) return;
    const bool scaled = a.grad_scale != nullptr;
    const float scale = scaled ? *a.grad_scale : 1.0f;
    for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const Tensor& t = a.t[tensor_of(a, tile)];
        AdamWConsts c = a.c;
        c.decay = t.decay;
        c.step = t.step;
        const int64_t begin = static_cast<int64_t>(tile - t.first) * a.tile, end = min(begin + a.tile, t.n);
        if (t.vector) {   // whole warps: a group's threads take part together
            for (int64_t at = begin + (threadIdx.x & ~31) * 8; at < end; at += 256 * 8) {
                const int64_t i = at + (threadIdx.x & 31) * 8;
                const int n = inside8(i, end);
                step8<EIGHT>(t, c, scaled, scale, i, n);
            }
        } else {
            for (int64_t at = begin + (threadIdx.x & ~31); at < end; at += 256) {
                const int64_t i = at + (threadIdx.x & 31);
                step1<EIGHT>(t, c, scaled, scale, i, i < end);
            }
        }
    }
}

// Whether step8 may have the tensor.
bool vector_accesses(const fsdp_adamw_tensor& t) {
    const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    const uintptr_t moments = at(t.exp_avg) | at(t.exp_avg_sq);
    return ((at(t.param) | at(t.grad) | at(t.copy_bf16)) & 15) == 0 && (moments & (t.moments == FSDP_MOMENTS_8BIT ? 7 : 15)) == 0;
}

unsigned blocks_for(int64_t items, int64_t each, int64_t most) { return static_cast<unsigned>(std::min((items + each - 1) / each, most)); }

}  // namespace

cudaError_t launch_state8_pack(int kind, const float* x, int64_t n, uint8_t* codes, uint8_t* exps, int sms, cudaStream_t st) {
    if (n == 0) return cudaSuccess;
    return launch_early(kind == FSDP_STATE8_SIGNED ? state8_pack_kernel<true> : state8_pack_kernel<false>, dim3(blocks_for(n, 256, sms * 32)),
                        256, 0, st, x, n, codes, exps);
}

cudaError_t launch_state8_unpack(int kind, const uint8_t* codes, const uint8_t* exps, int64_t n, void* out, int out_dtype,
                                 int sms, cudaStream_t st) {
    if (n == 0) return cudaSuccess;
    const bool vector = (reinterpret_cast<uintptr_t>(codes) & 7) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    return launch_early(kind == FSDP_STATE8_SIGNED ? state8_unpack_kernel<true> : state8_unpack_kernel<false>,
                        dim3(blocks_for(n, vector ? 2048 : 256, sms * 16)), 256, 0, st, codes, exps, n, out, out_dtype, vector);
}

namespace {

template <int MOST>
cudaError_t launch_tensors(const fsdp_adamw_tensor* tensors, int64_t count, const fsdp_adamw_hp& hp, int64_t step, uint64_t seed,
                           const float* grad_scale, const int32_t* skip, int sms, cudaStream_t st) {
    Tensors<MOST> a;
    a.c = adamw_consts(&hp, step);
    const double bc1 = adamw_bc1(hp, step);
    a.grad_scale = grad_scale;
    a.skip = skip;
    for (const int moments : {FSDP_MOMENTS_F32, FSDP_MOMENTS_8BIT}) {   // a kernel for each kind
        const bool eight = moments == FSDP_MOMENTS_8BIT;
        int64_t total = 0;
        for (int64_t j = 0; j < count; ++j) total += tensors[j].moments == moments ? tensors[j].numel : 0;
        a.tile = static_cast<int>(std::min<int64_t>(eight ? kMostTile8 : kMostTile32,
                                                    std::max<int64_t>(1, total / (static_cast<int64_t>(sms) * 8 * kLeastTile)) * kLeastTile));
        for (int64_t j = 0; j < count;) {
            a.count = a.tiles = 0;
            for (; j < count && a.count < MOST; ++j) {
                const fsdp_adamw_tensor& s = tensors[j];
                if (s.numel == 0 || s.moments != moments) continue;
                const int64_t tiles = (s.numel + a.tile - 1) / a.tile;
                if (a.tiles + tiles > 0x7fffffff) break;   // 2^40 elements are at most 2^29 tiles of the largest size
                const AdamWScaled own = adamw_scaled(hp, bc1, s.lr_scale, s.decay_scale);
                const uint64_t key = seed * 0x9E3779B97F4A7C15ull + (static_cast<uint64_t>(j) + 1) * 0xD1B54A32D192ED03ull;
                a.t[a.count++] = Tensor{s.param, s.grad, s.exp_avg, s.exp_avg_sq, s.exp_avg_exps, s.exp_avg_sq_exps, s.copy_bf16, s.numel,
                                        own.decay, own.step, static_cast<uint32_t>(key >> 32), a.tiles, s.grad_dtype, vector_accesses(s)};
                a.tiles += static_cast<uint32_t>(tiles);
            }
            if (a.count == 0) continue;
            const cudaError_t e = launch_early(eight ? adamw_tensors_kernel<true, MOST> : adamw_tensors_kernel<false, MOST>,
                                               dim3(std::min<uint32_t>(a.tiles, static_cast<uint32_t>(sms) * 8)), 256, 0, st, a);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_adamw_tensors(const fsdp_adamw_tensor* tensors, int64_t count, const fsdp_adamw_hp& hp, int64_t step,
                                 uint64_t seed, const float* grad_scale, const int32_t* skip, int sms, cudaStream_t st) {
    // a few tensors: kilobytes of parameters instead of tens of them for a launch to carry
    return count <= kFew ? launch_tensors<kFew>(tensors, count, hp, step, seed, grad_scale, skip, sms, st)
                         : launch_tensors<kTensors>(tensors, count, hp, step, seed, grad_scale, skip, sms, st);
}

}  // namespace fsdp
