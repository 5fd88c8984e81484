// Layer norm, forward and backward.  Both stream their matrices once: the forward
// reads a row into registers (two-pass mean and variance there) and writes y;
// the backward reads dy and x once, keeps each thread's columns of dgamma and
// dbeta in registers over all the rows its block walks, and a second small
// kernel joins the blocks' partial sums in a fixed order.
#include <algorithm>

#include "block_device.cuh"
#include "compute.hpp"
#include "rows.cuh"

namespace fsdp {
namespace {

// Sum over the block; every thread gets it.  `red` holds 32 floats and is free
// again after the next barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    const int w = threadIdx.x >> 5, n = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s += red[i];
    return s;
}

// One row to a warp (WARP) or to a block; chunk k of a thread holds the eight
// columns from (t + k * threads) * 8.  For rows that are too few to walk, or (ANY)
// that start anywhere: one row of 1280 takes the latency of a launch, a load and
// two sums; 4096 rows of 1281 columns, 21 us (1.0 TB/s; an element to a lane, 27),
// of 5121, 66 (1.3; 88), which the instructions that move the words bound with
// the rows in flight.
template <int NV, bool WARP, bool ANY>
__global__ void __launch_bounds__(WARP ? 128 : 1024) norm_forward_kernel(NormForward a) {
    __shared__ float red[2][32];
    starts_early();
    after_previous();
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int threads = WARP ? 32 : blockDim.x;
    const int64_t first = WARP ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t stride = WARP ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x;
    const float n = static_cast<float>(a.cols);
    float g[NV][8], b[NV][8];
    int in[NV];   // of a chunk's columns
#pragma unroll
    for (int k = 0; k < NV; ++k) in[k] = inside8(static_cast<int64_t>(t + k * threads) * 8, a.cols);
    if constexpr (ANY) {   // the blocks walk rows
        load_chunks_any<NV>(a.gamma, a.param_dtype, t * 8, in, threads * 8, g);
        load_chunks_any<NV>(a.beta, a.param_dtype, t * 8, in, threads * 8, b);
    }
    for (int64_t row = first; row < a.rows; row += stride) {
        float v[NV][8];
        float s = 0.0f;
        const auto on = [&](int k) { return static_cast<int64_t>(t + k * threads) * 8 < a.cols; };
        if constexpr (ANY) load_chunks_any<NV>(a.x.p, a.x.dtype, row * a.x.ld + t * 8, in, threads * 8, v);
        else load_chunks<NV>(a.x.p, a.x.dtype, row * a.x.ld + t * 8, threads * 8, on, v);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[k][j];
        const float mean = (WARP ? warp_sum(s) : block_sum(s, red[0])) / n;
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = (ANY ? j : 0) < in[k] ? v[k][j] - mean : 0.0f;
                ss = fmaf(d, d, ss);
            }
        }
        const float var = (WARP ? warp_sum(ss) : block_sum(ss, red[1])) / n;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (t == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = static_cast<int64_t>(t + k * threads) * 8;
            if (a.ckpt.p != nullptr) {
                const uint32_t top = act8_group_top<8>(v[k]);
                if (c < a.ckpt.ld) {
                    act8_writev<8>(static_cast<uint8_t*>(a.ckpt.p) + row * a.ckpt.ld, c, v[k], top);
                    if ((t & 3) == 0) a.ckpt.e[row * a.ckpt.eld + (c >> 5)] = static_cast<uint8_t>(act8_byte(top));
                }
            }
            if constexpr (ANY) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][j] = fmaf((v[k][j] - mean) * rstd, g[k][j], b[k][j]);
                store_chunk_any(a.y.p, a.y.dtype, row * a.y.ld + c, in[k], v[k]);
            } else if (c < a.cols) {
                load8(a.gamma, a.param_dtype, c, g[0]);
                load8(a.beta, a.param_dtype, c, b[0]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][j] = fmaf((v[k][j] - mean) * rstd, g[0][j], b[0][j]);
                store8(a.y.p, a.y.dtype, row * a.y.ld + c, v[k]);
            }
        }
        if (!WARP) __syncthreads();
    }
}

// Rows too long for registers: three passes, the later ones from L2, which
// bounds it with one element to a load (4096 x 49152: 597 us, 1.3 TB/s).
__global__ void __launch_bounds__(1024) norm_forward_wide_kernel(NormForward a) {
    __shared__ float red[2][32];
    starts_early();
    after_previous();
    const float n = static_cast<float>(a.cols);
    const int64_t ceil32 = (a.cols + 31) / 32 * 32;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) s += load1(a.x.p, a.x.dtype, row * a.x.ld + c);
        const float mean = block_sum(s, red[0]) / n;
        float ss = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float d = load1(a.x.p, a.x.dtype, row * a.x.ld + c) - mean;
            ss = fmaf(d, d, ss);
        }
        const float rstd = 1.0f / sqrtf(block_sum(ss, red[1]) / n + a.eps);
        if (threadIdx.x == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        for (int64_t c = threadIdx.x; c < ceil32; c += blockDim.x) {
            const bool on = c < a.cols;
            const float x = on ? load1(a.x.p, a.x.dtype, row * a.x.ld + c) : 0.0f;
            if (a.ckpt.p != nullptr) {   // ceil32 and the block are multiples of 32: whole warps
                const uint32_t top = act8_group_top<1>(&x);
                act8_writev<1>(static_cast<uint8_t*>(a.ckpt.p) + row * a.ckpt.ld, c, &x, top);
                if ((threadIdx.x & 31) == 0) a.ckpt.e[row * a.ckpt.eld + (c >> 5)] = static_cast<uint8_t>(act8_byte(top));
            }
            if (on)
                store1(a.y.p, a.y.dtype, row * a.y.ld + c,
                       fmaf((x - mean) * rstd, load1(a.gamma, a.param_dtype, c), load1(a.beta, a.param_dtype, c)));
        }
        __syncthreads();
    }
}

template <int V>
__device__ __forceinline__ void load_x(const Mat& x, int64_t row, int64_t c, float* v) {
    if (x.dtype == FSDP_DTYPE_ACT8)
        act8_readv<V>(static_cast<const uint8_t*>(x.p) + row * x.ld, x.e + row * x.eld, c, v);
    else
        loadv<V>(x.p, x.dtype, row * x.ld + c, v);
}

// ---- rows staged through shared memory ----
//
// A block walks rows with a fixed stride; the rows ahead are copied into a ring
// of shared memory with cp.async.  Every thread copies exactly the chunks (8
// columns) that it will read itself, so no barrier and no wait on another
// thread is needed: only its own cp.async groups.
//
// A row belongs to a group of GT threads; thread t owns chunks t + k*GT, k < NV,
// and a block holds several groups.  NV and GT are constants, so that the
// addresses of a row's chunks differ by constants, and only the last chunk can
// lie past the row's end.  FAST: every matrix and vector is BF16 (x may be
// ACT8); otherwise types are looked at with every chunk (with types that are not
// constants the forward took 67 us where it takes 48).  The arithmetic runs on
// pairs of columns.

constexpr int kRing = 4;   // rows in the ring, at most

// Bytes of eight elements.
__host__ __device__ __forceinline__ int chunk_bytes(int dtype) {
    return dtype == FSDP_DTYPE_F32 ? 32 : dtype == FSDP_DTYPE_BF16 ? 16 : 8;
}

// One matrix's rows as a thread sees them: its first chunk's address in global
// memory for row 0, and its slots.  Slot (place, k) of a group starts at
// (place * NV + k) * GT chunks; an F32 chunk is two halves GT * 16 bytes apart
// (16-byte accesses of neighbouring threads are neighbours).
template <int NV, int GT, bool FAST, bool INT8 = false>
struct Rows {
    const uint8_t* first;
    int64_t pitch;          // bytes between rows
    uint8_t* slots;
    int cb;                 // chunk_bytes
    int place;              // bytes between places

    __device__ Rows(const Mat& m, uint8_t* at, int group, int groups, int t) {
        cb = INT8 ? 8 : FAST ? 16 : chunk_bytes(m.dtype);
        place = groups * NV * GT * cb;
        slots = at + group * NV * GT * cb + t * (INT8 ? 8 : 16);
        first = static_cast<const uint8_t*>(m.p) + t * cb;
        pitch = m.ld * (cb >> 3);
    }
    __device__ void copy(int64_t row, int s, bool end) const {
        const uint8_t* src = first + row * pitch;
        const uint32_t dst = shared_at(slots + s * place);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k + 1 < NV || end) {
                if (INT8) {
                    copy8(dst + k * GT * 8, src + k * GT * 8);
                } else if (FAST || cb == 16) {
                    copy16(dst + k * GT * 16, src + k * GT * 16);
                } else {
                    copy16(dst + k * GT * 32, src + k * GT * 32);
                    copy16(dst + k * GT * 32 + GT * 16, src + k * GT * 32 + 16);
                }
            }
        }
    }
    __device__ void read(int s, int k, f32x2* v) const {
        const uint8_t* p = slots + s * place;
        if (FAST || cb == 16) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + k * GT * 16);
            v[0] = pair(bf16_lo(w.x), bf16_hi(w.x));
            v[1] = pair(bf16_lo(w.y), bf16_hi(w.y));
            v[2] = pair(bf16_lo(w.z), bf16_hi(w.z));
            v[3] = pair(bf16_lo(w.w), bf16_hi(w.w));
        } else {
            const float4 a = *reinterpret_cast<const float4*>(p + k * GT * 32);
            const float4 b = *reinterpret_cast<const float4*>(p + k * GT * 32 + GT * 16);
            v[0] = pair(a.x, a.y);
            v[1] = pair(a.z, a.w);
            v[2] = pair(b.x, b.y);
            v[3] = pair(b.z, b.w);
        }
    }
    // The int8 values of an ACT8 chunk, as floats.
    __device__ void read_ints(int s, int k, f32x2* v) const {
        const uint2 w = *reinterpret_cast<const uint2*>(slots + s * place + k * GT * 8);
        const f32x2 off = pair(-8388736.0f, -8388736.0f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t x = (h ? w.y : w.x) ^ 0x80808080u;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                v[2 * h + j] = add2(pair(__uint_as_float(__byte_perm(x, 0x4b000000u, 0x7440 + 2 * j)),
                                         __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7441 + 2 * j))), off);
        }
    }
};

// Where a thread's chunks of an output row go.
template <int GT, bool FAST>
struct Out {
    uint8_t* first;
    int64_t pitch;
    int dtype;
    __device__ Out(const Mat& m, int t) {
        dtype = m.dtype;
        first = static_cast<uint8_t*>(m.p) + t * chunk_bytes(m.dtype);
        pitch = m.ld * (chunk_bytes(m.dtype) >> 3);
    }
    __device__ void store(uint8_t* row, int k, const f32x2* v) const {
        float o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpair(v[j], o[2 * j], o[2 * j + 1]);
        if (FAST) store8(row + k * GT * 16, FSDP_DTYPE_BF16, 0, o);
        else store8(row + k * GT * chunk_bytes(dtype), dtype, 0, o);
    }
};

// gamma or beta as a matrix of one row (all groups own the same columns and
// share its slots).  Read from L1 or L2 with every row instead, they doubled
// the time: the ring leaves L1 no room for them.
__device__ __forceinline__ Mat vector_row(const void* p, int dtype) { return Mat{const_cast<void*>(p), nullptr, 0, 0, dtype}; }

// Sums over a group of NW warps, for all of its threads.  Each warp leaves its
// own; `red` is one of two buffers used in turn: a thread that writes one again
// has passed the barrier behind which every thread had read it.
template <int NW>
__device__ __forceinline__ float group_sum(float a, float* red, int group) {
    a = warp_sum(a);
    if constexpr (NW == 1) return a;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(NW * 32) : "memory");
    a = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; i += 4) {
        const float4 r = *reinterpret_cast<const float4*>(red + group * NW + i);
        a += NW == 2 ? r.x + r.y : (r.x + r.y) + (r.z + r.w);
    }
    return a;
}

template <int NW>
__device__ __forceinline__ float2 group_sum2(float a, float b, float2* red, int group) {
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (NW == 1) return make_float2(a, b);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(NW * 32) : "memory");
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; i += 2) {
        const float4 r = *reinterpret_cast<const float4*>(red + group * NW + i);
        a += r.x + r.z;
        b += r.y + r.w;
    }
    return make_float2(a, b);
}

// Mean and variance in two passes over registers, as the definition has them.
// 4096 x 12288 with an 8-bit checkpoint: 48 us for 253 MB, 5.3 TB/s where a copy
// has 6.8.  A row's latency at one block of 512 threads an SM bounds it (DRAM is
// 49 % busy, L2 30 %, a quarter of the warps that an SM can hold).
template <int NV, int GT, int THREADS, bool FAST>
__global__ void __launch_bounds__(THREADS) norm_forward_ring_kernel(const __grid_constant__ NormForward a, int places) {
    extern __shared__ __align__(16) uint8_t ring_bytes[];
    __shared__ __align__(16) float red[2][32];
    starts_early();
    after_previous();
    const int g = threadIdx.x / GT, t = threadIdx.x % GT, G = blockDim.x / GT;
    const bool end = (t + (NV - 1) * GT) * 8 < a.cols;
    const Rows<NV, GT, FAST> gammas(vector_row(a.gamma, a.param_dtype), ring_bytes, 0, 1, t);
    const Rows<NV, GT, FAST> betas(vector_row(a.beta, a.param_dtype), ring_bytes + gammas.place, 0, 1, t);
    const Rows<NV, GT, FAST> xs(a.x, ring_bytes + 2 * gammas.place, g, G, t);
    const Out<GT, FAST> ys(a.y, t);
    if (g == 0) {
        gammas.copy(0, 0, end);
        betas.copy(0, 0, end);
        copies_end();
        copies_wait(0);
    }
    __syncthreads();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * G, first = static_cast<int64_t>(blockIdx.x) * G + g;
    const float n = static_cast<float>(a.cols);
    for (int s = 0; s + 1 < places; ++s) {
        if (first + s * stride < a.rows) xs.copy(first + s * stride, s, end);
        copies_end();
    }
    int place = 0;
    for (int64_t row = first; row < a.rows; row += stride) {
        const int64_t ahead = row + (places - 1) * stride;
        if (ahead < a.rows) xs.copy(ahead, place == 0 ? places - 1 : place - 1, end);
        copies_end();
        copies_wait(places - 1);
        f32x2 v[NV][4];
        f32x2 s = pair(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k + 1 < NV || end) {
                xs.read(place, k, v[k]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[k][j] = pair(0.0f, 0.0f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s = add2(s, v[k][j]);
        }
        place = place + 1 == places ? 0 : place + 1;
        const float mean = group_sum<GT / 32>(both(s), red[0], g) / n;
        const f32x2 less = pair(-mean, -mean);
        f32x2 ss = pair(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k + 1 < NV || end) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2 d = add2(v[k][j], less);
                    ss = fma2(d, d, ss);
                }
            }
        }
        const float rstd = 1.0f / sqrtf(group_sum<GT / 32>(both(ss), red[1], g) / n + a.eps);
        if (t == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        if (a.ckpt.p != nullptr) {
            uint8_t* q = static_cast<uint8_t*>(a.ckpt.p) + row * a.ckpt.ld;
            uint8_t* e = a.ckpt.e + row * a.ckpt.eld;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) unpair(v[k][j], x[2 * j], x[2 * j + 1]);
                const uint32_t top = act8_group_top<8>(x);
                const int c = (t + k * GT) * 8;
                if (k + 1 < NV || c < a.ckpt.ld) {   // the pads of a short last group are zeros
                    act8_writev<8>(q, c, x, top);
                    if ((t & 3) == 0) e[c >> 5] = static_cast<uint8_t>(act8_byte(top));
                }
            }
        }
        const f32x2 r2 = pair(rstd, rstd);
        uint8_t* y = ys.first + row * ys.pitch;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k + 1 < NV || end) {
                f32x2 gm[4], bt[4];
                gammas.read(0, k, gm);
                betas.read(0, k, bt);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[k][j] = fma2(mul2(add2(v[k][j], less), r2), gm[j], bt[j]);
                ys.store(y, k, v[k]);
            }
        }
    }
}

// KEPT: x is an ACT8 checkpoint.  AGAIN: a row's x-hat and dy gamma are computed
// from shared memory once more for dx, not held in registers, which leaves those
// to more columns' sums.  What bounds it below 4096 columns or so is the latency
// of a row, from its sums to its last store, and the rows in flight on an SM:
// the blocks hold as many groups as the registers and the ring allow.  Measured,
// with an added branch, from BF16 and from 8 bits (bytes over time): 4096 x 12288
// 74 us (5.4 TB/s) and 70 (5.0); 8192 x 6144 75 (5.3) and 74 (4.7); 8192 x 4096
// 58 (4.6) and 54 (4.4), by one group of 512 threads a block 94 and 78; 8192 x
// 1280 27 (3.1) and 27 (2.7).
template <int NV, int GT, int THREADS, bool FAST, bool KEPT, bool AGAIN>
__global__ void __launch_bounds__(THREADS) norm_backward_ring_kernel(const __grid_constant__ NormBackward a, int places) {
    extern __shared__ __align__(16) uint8_t ring_bytes[];
    __shared__ __align__(16) float2 red[2][32];
    starts_early();
    after_previous();
    const int g = threadIdx.x / GT, t = threadIdx.x % GT, G = blockDim.x / GT;
    const bool end = (t + (NV - 1) * GT) * 8 < a.cols;
    uint8_t* at = ring_bytes;
    const Rows<NV, GT, FAST> gammas(vector_row(a.gamma, a.param_dtype), at, 0, 1, t);
    at += gammas.place;
    const Rows<NV, GT, FAST> dys(a.dy, at, g, G, t);
    at += places * dys.place;
    const Rows<NV, GT, FAST, KEPT> xs(a.x, at, g, G, t);
    at += places * xs.place;
    const Rows<NV, GT, FAST> adds(a.add, at, g, G, t);   // read only if there is one
    const Out<GT, FAST> dxs(a.dx, t);
    const bool added = a.add.p != nullptr;
    if (g == 0) {
        gammas.copy(0, 0, end);
        copies_end();
        copies_wait(0);
    }
    __syncthreads();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * G, first = static_cast<int64_t>(blockIdx.x) * G + g;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    // What a warp needs of a row besides comes with it in one copy instruction, 32
    // words to a warp and place: the aligned words that hold the exponents of its
    // chunks (8 bytes of each chunk's, in three words), mean and rstd.  (A row
    // ahead in registers, the exponents came too late: 96 us against 70 at 4096 x
    // 12288; a copy instruction for each of a thread's, 90.)
    at += added ? places * adds.place : 0;
    const int lane = threadIdx.x & 31;
    uint32_t* const words = reinterpret_cast<uint32_t*>(at) + (threadIdx.x & ~31);
    const uintptr_t exps = reinterpret_cast<uintptr_t>(a.x.e) + ((t & ~31) >> 2);   // of the warp's first chunk
    const auto issue = [&](int64_t row, int s) {
        if (row < a.rows) {
            bool on = lane >= 30;
            uintptr_t from = reinterpret_cast<uintptr_t>((lane == 30 ? a.mean : a.rstd) + row);
            if (KEPT && lane < 3 * NV) {
                const uintptr_t start = row * a.x.eld;
                from = ((exps + start + lane / 3 * (GT / 4)) & ~uintptr_t(3)) + lane % 3 * 4;
                on = from < reinterpret_cast<uintptr_t>(a.x.e) + start + a.x.eld;
            }
            if (on) copy4(shared_at(words + s * blockDim.x + lane), from);
            dys.copy(row, s, end);
            xs.copy(row, s, end);
            if (added) adds.copy(row, s, end);
        }
        copies_end();
    };
    for (int s = 0; s + 1 < places; ++s) issue(first + s * stride, s);
    f32x2 dg[NV][4], db[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[k][j] = db[k][j] = pair(0.0f, 0.0f);
    int place = 0, flip = 0;
    for (int64_t row = first; row < a.rows; row += stride) {
        issue(row + (places - 1) * stride, place == 0 ? places - 1 : place - 1);
        copies_wait(places - 1);
        constexpr int kHeld = AGAIN ? 1 : NV;
        f32x2 xh[kHeld][4], gr[kHeld][4];
        f32x2 s1 = pair(0.0f, 0.0f), s2 = pair(0.0f, 0.0f);
        __syncwarp();   // the words are other lanes' copies
        const uint32_t* w = words + place * blockDim.x;
        const float mean = __uint_as_float(w[30]), r = __uint_as_float(w[31]);
        const f32x2 less = pair(-mean, -mean), r2 = pair(r, r);
        const uint8_t* byte = reinterpret_cast<const uint8_t*>(w) + ((exps + row * a.x.eld) & 3u) + (lane >> 2);
        // x-hat = (x - mean) rstd, and dy gamma.  The difference comes first and is
        // rounded once (a checkpoint's value, its integer times a power of two, is exact):
        // x rstd - (mean rstd) would be off by the rounding of mean rstd, which is
        // thousands of x-hat's own where the mean is thousands of deviations.
        const auto expand = [&](int k, f32x2* x, f32x2* dy, f32x2* g4) {
            f32x2 gm[4];
            gammas.read(0, k, gm);
            dys.read(place, k, dy);
            f32x2 step2 = 0;
            if (KEPT) {
                xs.read_ints(place, k, x);
                const float step = act8_step(byte[k * 12]);
                step2 = pair(step, step);
            } else {
                xs.read(place, k, x);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = mul2(KEPT ? fma2(x[j], step2, less) : add2(x[j], less), r2);
                g4[j] = mul2(dy[j], gm[j]);
            }
        };
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k + 1 < NV || end) {
                const int h = AGAIN ? 0 : k;
                f32x2 dy[4];
                expand(k, xh[h], dy, gr[h]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    db[k][j] = add2(db[k][j], dy[j]);
                    dg[k][j] = fma2(dy[j], xh[h][j], dg[k][j]);
                    s1 = add2(s1, gr[h][j]);
                    s2 = fma2(gr[h][j], xh[h][j], s2);
                }
            }
        }
        const float2 sum = group_sum2<GT / 32>(both(s1), both(s2), red[flip], g);
        flip ^= 1;
        // dx = dy gamma rstd - xh c2 - c1 [+ add]
        const float c1 = -sum.x * inv_n * r, c2 = -sum.y * inv_n * r;
        const f32x2 m1 = pair(c1, c1), m2 = pair(c2, c2);
        uint8_t* dx = dxs.first + row * dxs.pitch;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k + 1 < NV || end) {
                const int h = AGAIN ? 0 : k;
                f32x2 o[4];
                if (AGAIN) expand(k, xh[h], o, gr[h]);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = fma2(r2, gr[h][j], fma2(xh[h][j], m2, m1));
                if (added) {
                    f32x2 e[4];
                    adds.read(place, k, e);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = add2(o[j], e[j]);
                }
                dxs.store(dx, k, o);
            }
        }
        place = place + 1 == places ? 0 : place + 1;
        __syncwarp();   // a place's words are read before they are copied anew
    }
    // the groups' column sums meet in shared memory: element j of chunk i at
    // j * kSlots + i (no bank conflicts writing, nor reading the columns in order)
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    constexpr int kSlots = NV * GT + 4;
    float* comb = reinterpret_cast<float*>(ring_bytes);
    copies_wait(0);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float* to = comb + (g * 16 + 2 * j) * kSlots + t + k * GT;
            unpair(dg[k][j], to[0], to[kSlots]);
            unpair(db[k][j], to[8 * kSlots], to[9 * kSlots]);
        }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o)
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float* from = comb + (o * 8 + (c & 7)) * kSlots + (c >> 3);
            float s = from[0];
            for (int h = 1; h < G; ++h) s += from[h * 16 * kSlots];
            part[o * a.cols + c] = s;
        }
}

// ---- other rows ----

__device__ __forceinline__ float2 group_sum2(float a, float b, float2* red, int group, int gt) {
    a = warp_sum(a);
    b = warp_sum(b);
    const int nw = gt >> 5;
    if (nw == 1) return make_float2(a, b);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gt) : "memory");
    a = b = 0.0f;
    for (int i = 0; i < nw; ++i) {
        a += red[group * nw + i].x;
        b += red[group * nw + i].y;
    }
    return make_float2(a, b);
}

// Rows that start anywhere: chunks of eight columns straight from global memory,
// as words that hold them.  Bound by a row's latency and the registers, which
// allow few rows on an SM (with two chunks to a thread they do not suffice: 460
// bytes a thread are spilled): 4096 x 1281 with an added branch 36 us (1.2 TB/s; an
// element to a lane, 60), 4096 x 5121 109 (1.5; 361).
template <int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(NormBackward a, int gt) {
    extern __shared__ __align__(16) uint8_t ring_bytes[];
    __shared__ float2 red[2][THREADS / 32];
    starts_early();
    after_previous();
    const int g = threadIdx.x / gt, t = threadIdx.x % gt, G = blockDim.x / gt;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    int in[NV];   // of a chunk's columns
#pragma unroll
    for (int k = 0; k < NV; ++k) in[k] = inside8((t + k * gt) * 8, a.cols);
    float dg[NV][8], db[NV][8], gm[NV][8];
    load_chunks_any<NV>(a.gamma, a.param_dtype, t * 8, in, gt * 8, gm);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[k][j] = db[k][j] = 0.0f;
    int flip = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * G + g; row < a.rows; row += static_cast<int64_t>(gridDim.x) * G) {
        float xh[NV][8], dy[NV][8];
        const float mean = a.mean[row], rstd = a.rstd[row];
        load_chunks_any<NV>(a.dy.p, a.dy.dtype, row * a.dy.ld + t * 8, in, gt * 8, dy);
        if (a.x.dtype == FSDP_DTYPE_ACT8) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (t + k * gt) * 8;
                if (c < a.cols) {
                    act8_readv<8>(static_cast<const uint8_t*>(a.x.p) + row * a.x.ld, a.x.e + row * a.x.eld, c, xh[k]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) xh[k][j] = 0.0f;
                }
            }
        } else {
            load_chunks_any<NV>(a.x.p, a.x.dtype, row * a.x.ld + t * 8, in, gt * 8, xh);
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // past the row's end dy and gamma are 0, and x-hat is held at 0
                xh[k][j] = j < in[k] ? (xh[k][j] - mean) * rstd : 0.0f;
                db[k][j] += dy[k][j];
                dg[k][j] = fmaf(dy[k][j], xh[k][j], dg[k][j]);
                dy[k][j] *= gm[k][j];
                s1 += dy[k][j];
                s2 = fmaf(dy[k][j], xh[k][j], s2);
            }
        const float2 sum = group_sum2(s1, s2, red[flip], g, gt);
        flip ^= 1;
        const float c1 = sum.x * inv_n, c2 = sum.y * inv_n;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) dy[k][j] = rstd * (dy[k][j] - c1 - xh[k][j] * c2);
        if (a.add.p != nullptr) {
            load_chunks_any<NV>(a.add.p, a.add.dtype, row * a.add.ld + t * 8, in, gt * 8, xh);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) dy[k][j] += xh[k][j];
            // add may be dx itself: the chunks' neighbours, of which the words above hold
            // a part, are stored after every lane has read them
            __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (t + k * gt) * 8;
            store_chunk_any(a.dx.p, a.dx.dtype, row * a.dx.ld + c, in[k], dy[k]);
        }
    }
    // the groups' column sums meet in shared memory: element j of chunk i at j * slots + i
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    const int slots = NV * gt + 4;
    float* comb = reinterpret_cast<float*>(ring_bytes);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            comb[(g * 16 + j) * slots + t + k * gt] = dg[k][j];
            comb[(g * 16 + 8 + j) * slots + t + k * gt] = db[k][j];
        }
    __syncthreads();
    for (int o = 0; o < 2; ++o)
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float* from = comb + (o * 8 + (c & 7)) * slots + (c >> 3);
            float s = from[0];
            for (int h = 1; h < G; ++h) s += from[h * 16 * slots];
            part[o * a.cols + c] = s;
        }
}

// Rows too long for registers: dx first (two passes over a row), then the
// column sums from dy and x once more.  Bound by loads of one element (4096 x
// 24576 with an added branch: 1009 us).
__global__ void __launch_bounds__(1024) norm_backward_wide_dx_kernel(NormBackward a) {
    __shared__ float red[2][32];
    starts_early();
    after_previous();
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float x;
            load_x<1>(a.x, row, c, &x);
            const float gr = load1(a.dy.p, a.dy.dtype, row * a.dy.ld + c) * load1(a.gamma, a.param_dtype, c);
            s1 += gr;
            s2 = fmaf(gr, (x - mean) * rstd, s2);
        }
        const float c1 = block_sum(s1, red[0]) * inv_n, c2 = block_sum(s2, red[1]) * inv_n;
        for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float x;
            load_x<1>(a.x, row, c, &x);
            const float gr = load1(a.dy.p, a.dy.dtype, row * a.dy.ld + c) * load1(a.gamma, a.param_dtype, c);
            float o = rstd * (gr - c1 - (x - mean) * rstd * c2);
            if (a.add.p != nullptr) o += load1(a.add.p, a.add.dtype, row * a.add.ld + c);
            store1(a.dx.p, a.dx.dtype, row * a.dx.ld + c, o);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) norm_backward_wide_sums_kernel(NormBackward a) {
    starts_early();
    after_previous();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= a.cols) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        float x;
        load_x<1>(a.x, row, c, &x);
        const float d = load1(a.dy.p, a.dy.dtype, row * a.dy.ld + c);
        db += d;
        dg = fmaf(d, (x - a.mean[row]) * a.rstd[row], dg);
    }
    float* part = a.partials + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
    part[c] = dg;
    part[a.cols + c] = db;
}

// out0 from partials[p*stride + c], out1 (blockIdx.y == 1) from `second` floats
// further on: 16 threads of V columns across and 16 slices of p down to a
// block, the slices joined in order.  Bound by latency (152 rows of 2 x 12288:
// 8.6 us, 152 of 2 x 1280: 3): ten loads of a thread are in flight.
template <int V>
__global__ void __launch_bounds__(256) sum_partials_kernel(const float* partials, int64_t count, int64_t stride, int64_t second,
                                                           int64_t cols, void* out0, void* out1, int dtype, int accumulate) {
    __shared__ float part[16][16 * V];
    starts_early();
    after_previous();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 16 + tx) * V;
    const float* p = partials + (blockIdx.y ? second : 0) + c;
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.0f;
    if (c < cols) {
#pragma unroll 10
        for (int64_t i = ty; i < count; i += 16) {
            if constexpr (V == 4) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(p + i * stride));
                s[0] += f.x; s[1] += f.y; s[2] += f.z; s[3] += f.w;
            } else {
                s[0] += __ldcg(p + i * stride);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) part[ty][tx * V + j] = s[j];
    __syncthreads();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 * V + threadIdx.x;
    if (threadIdx.x < 16 * V && col < cols) {
        void* out = blockIdx.y ? out1 : out0;
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += part[i][threadIdx.x];
        if (accumulate) t += load1(out, dtype, col);
        store1(out, dtype, col, t);
    }
}

cudaError_t sum_partials(const float* partials, int64_t count, int64_t stride, int64_t second, int64_t cols,
                         void* out0, void* out1, int dtype, int accumulate, cudaStream_t st) {
    const bool vec = cols % 4 == 0;   // the workspace is aligned
    const dim3 grid(static_cast<unsigned>(vec ? (cols + 63) / 64 : (cols + 15) / 16), out1 != nullptr ? 2 : 1);
    return launch_early(vec ? sum_partials_kernel<4> : sum_partials_kernel<1>, grid, 256, 0, st, partials, count, stride, second,
                        cols, out0, out1, dtype, accumulate);
}

int round32(int64_t n) { return static_cast<int>((n + 31) / 32 * 32); }

// A row to a warp where its lanes hold it whole, or to a block.  ANY: as many
// blocks as run at once, which walk the rows.
template <bool ANY>
cudaError_t run_forward(const NormForward& a, int64_t chunks, int sms, cudaStream_t st) {
    const auto blocks = [&](int64_t rows, int threads) {
        return dim3(static_cast<unsigned>(std::min(rows, ANY ? static_cast<int64_t>(sms) * (1024 / threads) : int64_t(1) << 30)));
    };
    if (chunks <= 32) return launch_early(norm_forward_kernel<1, true, ANY>, blocks((a.rows + 3) / 4, 128), 128, 0, st, a);
    // two chunks to a thread leave room for more rows on an SM (4096 x 4097: 50 us,
    // with one 76; 4096 x 3585: 48 against 52 at 512)
    constexpr int kShort = ANY ? 256 : 512, kMost = ANY ? 2 : 4;
    const int threads = round32(chunks <= kShort ? chunks : (chunks + kMost - 1) / kMost);
    if (chunks <= kShort) return launch_early(norm_forward_kernel<1, false, ANY>, blocks(a.rows, threads), threads, 0, st, a);
    return launch_early(norm_forward_kernel<kMost, false, ANY>, blocks(a.rows, threads), threads, 0, st, a);
}

// How a row is split: threads to it, chunks (or columns) to a thread, rows to a
// block.
struct Split {
    int NV = 0, gt = 0, groups = 0;   // NV 0: rows too long for registers
    int threads() const { return gt * groups; }
};

// The constants' combination that covers the row's chunks with the fewest
// slots; of equals, the one with fewer threads, whose sums cost less.
Split split_row(int64_t rows, int64_t chunks, const int (*options)[2], int count, int block_threads) {
    Split p;
    for (int i = 0; i < count; ++i) {
        const int nv = options[i][0], gt = options[i][1];
        if (nv * gt < chunks || (nv - 1) * gt >= chunks) continue;
        if (p.NV != 0 && nv * gt >= p.NV * p.gt) continue;
        p.NV = nv;
        p.gt = gt;
    }
    if (p.NV != 0)   // a named barrier to a group: 15 at most
        p.groups = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(block_threads / p.gt, 15), rows)));
    return p;
}
constexpr int kForward[][2] = {{1, 32}, {2, 32}, {3, 32}, {4, 32}, {5, 32}, {6, 32}, {2, 128}, {3, 128}, {4, 128}, {5, 128}, {6, 128}, {4, 256}, {5, 256}, {6, 256}, {4, 512}};
constexpr int kBackward[][2] = {{1, 32}, {2, 32}, {3, 32}, {4, 32}, {5, 32}, {2, 128}, {3, 128}, {4, 128}, {3, 256}, {2, 512}, {3, 512}, {4, 512}, {5, 512}};

int64_t walkers(const Split& p, int64_t rows, int64_t most) {
    return std::max<int64_t>(1, std::min((rows + p.groups - 1) / p.groups, most));
}

constexpr int kWideSlices = 64;   // row slices of the column sums where rows are too long

bool backward_aligned(const NormBackward& a) {
    return rows_aligned(a.dy) && rows_aligned(a.x) && rows_aligned(a.dx) && (a.add.p == nullptr || rows_aligned(a.add)) &&
           a.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(a.gamma) & 15u) == 0;
}

// Bytes of eight columns in the ring.
int backward_chunk(const NormBackward& a) {
    return chunk_bytes(a.dy.dtype) + chunk_bytes(a.x.dtype) + (a.add.p != nullptr ? chunk_bytes(a.add.dtype) : 0);
}

Split backward_split(const NormBackward& a, bool vec) {
    const int64_t rows = a.rows, cols = a.cols;
    if (vec) {
        Split p = split_row(rows, cols / 8, kBackward, 13, 512);
        if (p.gt == 32 && p.NV > 3) p.groups = std::min(p.groups, 8);   // 256 threads, which may have twice the registers
        if (p.NV != 0) {
            // two places in the ring for every group, or one for one
            const int row = p.NV * p.gt * backward_chunk(a) + p.gt * 4, room = kSharedMost - p.NV * p.gt * chunk_bytes(a.param_dtype);
            if (row > room) p.NV = 0;
            else p.groups = std::max(1, std::min(p.groups, room / (2 * row)));
        }
        return p;
    }
    Split p;
    const int64_t chunks = (cols + 7) / 8;
    if (chunks <= 1536) {
        p.NV = chunks <= 768 ? 1 : 2;
        p.gt = round32((chunks + p.NV - 1) / p.NV);
        p.groups = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(768 / p.gt, 15), rows)));
    }
    return p;
}

int64_t backward_blocks(const Split& p, int64_t rows, int sms) {
    if (p.NV == 0) return std::max<int64_t>(1, std::min<int64_t>(rows, kWideSlices));
    return walkers(p, rows, sms);
}

}  // namespace

cudaError_t launch_norm_forward(const NormForward& a, int sms, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const bool vec = rows_aligned(a.x) && rows_aligned(a.y) && a.cols % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.gamma) | reinterpret_cast<uintptr_t>(a.beta)) & 15u) == 0;
    if (vec) {
        const Split p = split_row(a.rows, a.cols / 8, kForward, 15, 512);
        const int keep = p.NV * p.gt * 2 * chunk_bytes(a.param_dtype), row_bytes = p.threads() * p.NV * chunk_bytes(a.x.dtype);
        const int places = p.NV == 0 ? 0 : std::min(kRing, (kSharedMost - keep) / row_bytes);
        // rows enough for every group to walk two
        if (places > 0 && a.rows >= 2 * static_cast<int64_t>(sms) * p.groups) {
            const unsigned blocks = static_cast<unsigned>(walkers(p, a.rows, sms));
            const int bytes = keep + places * row_bytes;
            const bool fast = a.x.dtype == FSDP_DTYPE_BF16 && a.y.dtype == FSDP_DTYPE_BF16 && a.param_dtype == FSDP_DTYPE_BF16;
#define RING(nv, gt_)                                                                                             \
    if (p.NV == nv && p.gt == gt_)                                                                                \
        return fast ? launch_shared<norm_forward_ring_kernel<nv, gt_, 512, true>>(blocks, p.threads(), bytes, st, a, places) \
                    : launch_shared<norm_forward_ring_kernel<nv, gt_, 512, false>>(blocks, p.threads(), bytes, st, a, places);
            RING(1, 32) RING(2, 32) RING(3, 32) RING(4, 32) RING(5, 32) RING(6, 32)
            RING(2, 128) RING(3, 128) RING(4, 128) RING(5, 128) RING(6, 128)
            RING(4, 256) RING(5, 256) RING(6, 256) RING(4, 512)
#undef RING
        }
        if (a.cols <= 4096 * 8) return run_forward<false>(a, a.cols / 8, sms, st);
    } else if (a.cols <= 2048 * 8) {
        return run_forward<true>(a, (a.cols + 7) / 8, sms, st);
    }
    return launch_early(norm_forward_wide_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t(1) << 30))), 1024, 0, st, a);
}

cudaError_t launch_norm_backward(const NormBackward& a, int sms, cudaStream_t st) {
    const bool vec = backward_aligned(a);
    const Split p = backward_split(a, vec);
    cudaError_t e = cudaSuccess;
    int64_t count = backward_blocks(p, a.rows, sms);
    const unsigned blocks = static_cast<unsigned>(count);
    if (a.rows == 0) {
        count = 0;
    } else if (p.NV == 0) {
        e = launch_early(norm_backward_wide_dx_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t(1) << 30))), 1024, 0, st, a);
        if (e != cudaSuccess) return e;
        const dim3 grid(static_cast<unsigned>((a.cols + 255) / 256), blocks);
        e = launch_early(norm_backward_wide_sums_kernel, grid, 256, 0, st, a);
    } else if (vec) {
        const int row_bytes = p.threads() * (p.NV * backward_chunk(a) + 4);
        const int keep = p.NV * p.gt * chunk_bytes(a.param_dtype);
        const int places = std::max(1, std::min(kRing, (kSharedMost - keep) / row_bytes));
        const int comb = p.groups * 16 * (p.NV * p.gt + 4) * 4;
        const int bytes = std::max(keep + places * row_bytes, comb);
        const bool kept = a.x.dtype == FSDP_DTYPE_ACT8;
        const bool fast = a.dy.dtype == FSDP_DTYPE_BF16 && a.dx.dtype == FSDP_DTYPE_BF16 && a.param_dtype == FSDP_DTYPE_BF16 &&
                          a.x.dtype != FSDP_DTYPE_F32 && (a.add.p == nullptr || a.add.dtype == FSDP_DTYPE_BF16);
        e = cudaErrorInvalidConfiguration;
#define RING_(nv, gt_, most, again, f, k)                                                                 \
    if (fast == f && kept == k)                                                                           \
        e = launch_shared<norm_backward_ring_kernel<nv, gt_, most, f, k, again>>(blocks, p.threads(), bytes, st, a, places)
#define RING(nv, gt_, most, again)                    \
    if (p.NV == nv && p.gt == gt_) {                  \
        RING_(nv, gt_, most, again, true, true);     \
        RING_(nv, gt_, most, again, true, false);     \
        RING_(nv, gt_, most, again, false, true);     \
        RING_(nv, gt_, most, again, false, false);     \
    }
        RING(1, 32, 512, false) RING(2, 32, 512, false) RING(3, 32, 512, true) RING(4, 32, 256, false) RING(5, 32, 256, false)
        RING(2, 128, 512, false) RING(3, 128, 512, true) RING(4, 128, 512, true) RING(3, 256, 512, true)
        RING(2, 512, 512, false) RING(3, 512, 512, false) RING(4, 512, 512, true) RING(5, 512, 512, true)
#undef RING
#undef RING_
    } else {
        const int comb = p.groups * 16 * (p.NV * p.gt + 4) * 4;
        e = p.NV == 1 ? launch_shared<norm_backward_kernel<1, 768>>(blocks, p.threads(), comb, st, a, p.gt)
                      : launch_shared<norm_backward_kernel<2, 768>>(blocks, p.threads(), comb, st, a, p.gt);
    }
    if (e != cudaSuccess) return e;
    return sum_partials(a.partials, count, 2 * a.cols, a.cols, a.cols, a.dgamma, a.dbeta, a.grad_dtype, a.accumulate, st);
}

cudaError_t launch_sum_partials(const float* partials, int64_t count, int64_t stride, int64_t cols, void* out,
                                int out_dtype, int accumulate, cudaStream_t st) {
    return sum_partials(partials, count, stride, 0, cols, out, nullptr, out_dtype, accumulate, st);
}

}  // namespace fsdp
