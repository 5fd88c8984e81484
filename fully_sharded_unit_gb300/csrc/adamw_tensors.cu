// AdamW over many tensors in one launch, with moments in 32 or 8 bits, and 8-bit moments
// from and to floats.
#include <algorithm>

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
    const uint32_t b = __float_as_uint(SIGNED ? fabsf(x) * away * kDown<SIGNED> : fmaxf(x, 0.0f) * away * kDown<SIGNED>);
    const uint32_t r = random == kNearest ? 0x7ffffu + ((b >> 20) & 1u) : random;
    uint32_t code = min((b + r) >> 20, SIGNED ? 0x7fu : 0xffu);
    if (SIGNED) return code != 0 ? code | ((__float_as_uint(x) >> 24) & 0x80u) : 0u;
    return x > 0.0f ? max(code, 1u) : 0u;
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

__device__ __forceinline__ float magnitude(float x, bool is_signed) { return is_signed ? x : max_nan(x, 0.0f); }

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

template <bool SIGNED>
__global__ void __launch_bounds__(256) state8_unpack_kernel(const uint8_t* codes, const uint8_t* exps, int64_t n, void* out, int dtype) {
    starts_early();
    after_previous();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += stride)
        store1(out, dtype, i, state8_value<SIGNED>(codes[i], state8_unit(exps[i >> 5])));
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
    int moments8;
};

constexpr int kTile = 2048;      // elements of a tile
constexpr int kTensors = 256;    // of one launch, in the kernel's parameters

struct Tensors {
    AdamWConsts c;               // decay and step: the tensor's
    const float* grad_scale;
    const int32_t* skip;
    uint32_t count, tiles;
    Tensor t[kTensors];
};

__device__ __forceinline__ uint32_t random_bits(int64_t i, uint32_t key) {
    uint32_t x = static_cast<uint32_t>(i) ^ key ^ static_cast<uint32_t>(i >> 32) * 0x85157AF5u;
    x ^= x >> 16;
    x *= 0xD36F86A9u;
    x ^= x >> 15;
    x *= 0xC242E759u;
    return x ^ (x >> 16);
}

// A group of 32 elements to a warp.
__global__ void __launch_bounds__(256) adamw_tensors_kernel(const __grid_constant__ Tensors a) {
    starts_early();
    after_previous();
    if (a.skip != nullptr && *a.skip != 0) return;
    const float scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
    const int lane = threadIdx.x & 31;
    for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        uint32_t lo = 0, hi = a.count;   // the last tensor whose first tile is at or before this one
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) / 2;
            if (a.t[mid].first <= tile) lo = mid;
            else hi = mid;
        }
        const Tensor& t = a.t[lo];
        AdamWConsts c = a.c;
        c.decay = t.decay;
        c.step = t.step;
        const int64_t begin = static_cast<int64_t>(tile - t.first) * kTile, end = min(begin + kTile, t.n);
        for (int64_t at = begin + (threadIdx.x & ~31); at < end; at += 256) {
            const int64_t i = at + lane;
            const bool on = i < end;
            float p = on ? t.p[i] : 0.0f, g = on ? load1(t.g, t.grad_dtype, i) : 0.0f, m = 0.0f, v = 0.0f;
            if (a.grad_scale != nullptr) g = __fmul_rn(g, scale);
            if (t.moments8) {
                if (on) {
                    m = state8_value<true>(static_cast<uint8_t*>(t.m)[i], state8_unit(t.me[i >> 5]));
                    v = state8_value<false>(static_cast<uint8_t*>(t.v)[i], state8_unit(t.ve[i >> 5]));
                }
            } else if (on) {
                m = static_cast<float*>(t.m)[i];
                v = static_cast<float*>(t.v)[i];
            }
            adamw_elem(p, g, m, v, c);
            if (on) {
                t.p[i] = p;
                if (t.copy != nullptr) reinterpret_cast<__nv_bfloat16*>(t.copy)[i] = __float2bfloat16_rn(p);
            }
            if (t.moments8) {
                const uint32_t r = random_bits(i, t.key);
                const uint32_t mb = state8_byte(__reduce_max_sync(kAll, on ? __float_as_uint(larger(0.0f, m)) : 0u));
                const uint32_t vb = state8_byte(__reduce_max_sync(kAll, on ? __float_as_uint(larger(0.0f, v)) : 0u));
                if (on) {
                    static_cast<uint8_t*>(t.m)[i] = static_cast<uint8_t>(state8_code<true>(m, mb, (r & 0xffffu) << 4));
                    static_cast<uint8_t*>(t.v)[i] = static_cast<uint8_t>(state8_code<false>(v, vb, (r >> 16) << 4));
                }
                if (lane == 0) {
                    t.me[i >> 5] = static_cast<uint8_t>(mb);
                    t.ve[i >> 5] = static_cast<uint8_t>(vb);
                }
            } else if (on) {
                static_cast<float*>(t.m)[i] = m;
                static_cast<float*>(t.v)[i] = v;
            }
        }
    }
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
    return launch_early(kind == FSDP_STATE8_SIGNED ? state8_unpack_kernel<true> : state8_unpack_kernel<false>,
                        dim3(blocks_for(n, 256, sms * 32)), 256, 0, st, codes, exps, n, out, out_dtype);
}

cudaError_t launch_adamw_tensors(const fsdp_adamw_tensor* tensors, int64_t count, const fsdp_adamw_hp& hp, int64_t step,
                                 uint64_t seed, const float* grad_scale, const int32_t* skip, int sms, cudaStream_t st) {
    Tensors a;
    a.c = adamw_consts(&hp, step);
    a.grad_scale = grad_scale;
    a.skip = skip;
    for (int64_t j = 0; j < count;) {
        a.count = a.tiles = 0;
        for (; j < count && a.count < kTensors; ++j) {
            const fsdp_adamw_tensor& s = tensors[j];
            if (s.numel == 0) continue;
            const int64_t tiles = (s.numel + kTile - 1) / kTile;
            if (a.tiles + tiles > 0x7fffffff) break;   // a tensor has at most 2^29 tiles
            fsdp_adamw_hp own = hp;
            own.lr *= s.lr_scale;
            own.weight_decay *= s.decay_scale;
            const AdamWConsts c = adamw_consts(&own, step);
            const uint64_t key = seed * 0x9E3779B97F4A7C15ull + (static_cast<uint64_t>(j) + 1) * 0xD1B54A32D192ED03ull;
            a.t[a.count++] = Tensor{s.param, s.grad, s.exp_avg, s.exp_avg_sq, s.exp_avg_exps, s.exp_avg_sq_exps, s.copy_bf16, s.numel,
                                    c.decay, c.step, static_cast<uint32_t>(key >> 32), a.tiles, s.grad_dtype, s.moments == FSDP_MOMENTS_8BIT};
            a.tiles += static_cast<uint32_t>(tiles);
        }
        if (a.count == 0) continue;
        const cudaError_t e = launch_early(adamw_tensors_kernel, dim3(std::min<uint32_t>(a.tiles, static_cast<uint32_t>(sms) * 8)), 256, 0, st, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace fsdp
