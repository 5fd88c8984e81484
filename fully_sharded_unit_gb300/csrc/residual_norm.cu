// The norms before and after a block with its gate and residual scale, forward and
// backward.
#include <algorithm>

#include "block_device.cuh"
#include "compute.hpp"
#include "rows.cuh"

namespace fsdp {
namespace {

// Sums over the block, for every thread.  `red` is free again after the next barrier.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*red)[32]) {
    const int w = threadIdx.x >> 5, n = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = warp_sum(v[i]);
        if ((threadIdx.x & 31) == 0) red[i][w] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.0f;
        for (int j = 0; j < n; ++j) v[i] += red[i][j];
    }
}

// Eight elements of a row from column c on, those inside the row; 0 past its end, and
// `otherwise` where there is no matrix or vector.
__device__ __forceinline__ void load_any(const void* p, int dtype, int64_t at, int in, float otherwise, float* v) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = otherwise;
    } else {
        load_chunks_any<1>(p, dtype, at, &in, 0, reinterpret_cast<float(*)[8]>(v));
    }
}

// ---- any rows ----
//
// A row to a block, in chunks of eight columns that start anywhere, read again (from L1
// or L2) for each of the passes that a row takes; the columns' sums of the backward pass lie in
// the block's row of the workspace.  Rows past 49152 columns have nothing else; their passes
// over L2 bound them (at 4096 x 12288 they took 253 us forward and 808 backward).

__device__ __forceinline__ void residual_chunk(const ResidualNorm& a, int64_t row, int64_t c, int in, float post_rstd, float* s) {
    float h[8], o[8], p[8], g[8];
    load_any(a.h.p, a.h.dtype, row * a.h.ld + c, in, 0.0f, h);
    load_any(a.o.p, a.o.dtype, row * a.o.ld + c, in, 0.0f, o);
    load_any(a.post, a.param_dtype, c, in, 1.0f, p);
    load_any(a.gate, a.param_dtype, c, in, 1.0f, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = fmaf(a.alpha, h[j], o[j] * post_rstd * p[j] * g[j]);
}

__global__ void __launch_bounds__(512) residual_norm_any_kernel(const ResidualNorm a) {
    __shared__ float red[2][1][32];
    starts_early();
    after_previous();
    const float n = static_cast<float>(a.cols);
    const int64_t chunks = (a.cols + 7) / 8;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float post_rstd = 1.0f;
        if (a.post != nullptr) {
            float ss[1] = {0.0f};
            for (int64_t q = threadIdx.x; q < chunks; q += blockDim.x) {
                float o[8];
                load_any(a.o.p, a.o.dtype, row * a.o.ld + q * 8, inside8(q * 8, a.cols), 0.0f, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss[0] = fmaf(o[j], o[j], ss[0]);
            }
            block_sums(ss, red[0]);
            post_rstd = 1.0f / sqrtf(ss[0] / n + a.eps);
            if (threadIdx.x == 0) a.post_rstd[row] = post_rstd;
        }
        float ss[1] = {0.0f};
        for (int64_t first = 0; first < chunks; first += blockDim.x) {   // whole warps store together
            const int64_t c = (first + threadIdx.x) * 8;
            const int in = inside8(c, a.cols);
            float s[8];
            residual_chunk(a, row, c, in, post_rstd, s);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < in) ss[0] = fmaf(s[j], s[j], ss[0]);
            if (a.y.p == nullptr) store_chunk_any(a.out.p, a.out.dtype, row * a.out.ld + c, in, s);
        }
        if (a.y.p != nullptr) {   // out behind the sum: it may lie where the residual stream does, which is read again
            block_sums(ss, red[1]);
            const float rstd = 1.0f / sqrtf(ss[0] / n + a.eps);
            if (threadIdx.x == 0) a.rstd[row] = rstd;
            for (int64_t first = 0; first < chunks; first += blockDim.x) {
                const int64_t c = (first + threadIdx.x) * 8;
                const int in = inside8(c, a.cols);
                float s[8], g[8];
                residual_chunk(a, row, c, in, post_rstd, s);
                load_any(a.gamma, a.param_dtype, c, in, 1.0f, g);
                store_chunk_any(a.out.p, a.out.dtype, row * a.out.ld + c, in, s);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = s[j] * rstd * g[j];
                store_chunk_any(a.y.p, a.y.dtype, row * a.y.ld + c, in, s);
            }
        }
        __syncthreads();
    }
}

// A chunk of the backward pass.
struct GradChunk {
    float dy[8], xh[8], g[8], k[8], u[8], t[8];   // k: gate * post_gamma; t: dout so far
};
__device__ __forceinline__ void grad_chunk(const ResidualNormGrad& a, int64_t row, int64_t c, int in, float rstd, float post_rstd,
                                           GradChunk& v) {
    load_any(a.dy.p, a.dy.dtype, row * a.dy.ld + c, in, 0.0f, v.dy);
    load_any(a.dout.p, a.dout.dtype, row * a.dout.ld + c, in, 0.0f, v.t);
    load_any(a.o.p, a.o.dtype, row * a.o.ld + c, in, 0.0f, v.u);
    load_any(a.dy.p != nullptr ? a.out.p : nullptr, a.out.dtype, row * a.out.ld + c, in, 0.0f, v.xh);
    float w[8];
    load_any(a.post, a.param_dtype, c, in, 1.0f, v.k);
    load_any(a.gate, a.param_dtype, c, in, 1.0f, w);
    load_any(a.gamma, a.param_dtype, c, in, 1.0f, v.g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v.k[j] *= w[j];
        v.u[j] *= post_rstd;
        v.xh[j] *= rstd;
        v.g[j] *= v.dy[j];
    }
}

__global__ void __launch_bounds__(512) residual_norm_any_backward_kernel(const ResidualNormGrad a) {
    __shared__ float red[3][32];
    starts_early();
    after_previous();
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    const int64_t chunks = (a.cols + 7) / 8;
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.dy.p != nullptr ? a.rstd[row] : 0.0f, post_rstd = a.post != nullptr ? a.post_rstd[row] : 1.0f;
        // with e = t k and t = dout + rstd (g - xh c1), sum(e u) is linear in c1
        float s[3] = {0.0f, 0.0f, 0.0f};
        for (int64_t q = threadIdx.x; q < chunks; q += blockDim.x) {
            GradChunk v;
            grad_chunk(a, row, q * 8, inside8(q * 8, a.cols), rstd, post_rstd, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float ku = v.k[j] * v.u[j];
                s[0] = fmaf(v.g[j], v.xh[j], s[0]);
                s[1] = fmaf(ku, fmaf(rstd, v.g[j], v.t[j]), s[1]);
                s[2] = fmaf(ku, v.xh[j], s[2]);
            }
        }
        block_sums(s, red);
        const float c1 = s[0] * inv_n, c2 = a.post != nullptr ? (s[1] - rstd * c1 * s[2]) * inv_n : 0.0f;
        const bool fresh = row == blockIdx.x;
        for (int64_t first = 0; first < chunks; first += blockDim.x) {
            const int64_t c = (first + threadIdx.x) * 8;
            const int in = inside8(c, a.cols);
            GradChunk v;
            grad_chunk(a, row, c, in, rstd, post_rstd, v);
            float dh[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = fmaf(rstd, fmaf(-v.xh[j], c1, v.g[j]), v.t[j]);
                dh[j] = a.alpha * t;
                v.dy[j] *= v.xh[j];
                v.t[j] = t * v.u[j];
                v.u[j] = post_rstd * fmaf(-v.u[j], c2, t * v.k[j]);
                if (j < in) {
                    if (a.dgamma != nullptr) part[c + j] = (fresh ? 0.0f : part[c + j]) + v.dy[j];
                    if (a.o.p != nullptr) part[a.cols + c + j] = (fresh ? 0.0f : part[a.cols + c + j]) + v.t[j];
                }
            }
            store_chunk_any(a.dh.p, a.dh.dtype, row * a.dh.ld + c, in, dh);
            if (a.dblock.p != nullptr) store_chunk_any(a.dblock.p, a.dblock.dtype, row * a.dblock.ld + c, in, v.u);
        }
        __syncthreads();
    }
}

// ---- a chunk to a thread ----
//
// Rows of any type and alignment in registers: a row to a block, or to a cluster of blocks
// that join their sums through one another's shared memory.  Bound by a row's latency, one
// row of up to 6144 columns at a time to an SM in the backward pass, with nothing of the next row under way: 1031 x 5121
// 52 us (1.2 TB/s).  What the ring does not take comes here.  At 4096 x 1280 and 4096 x 12288: F32 forward 25 and 324 us,
// backward 46 and 351; BF16 without a block (a model's first norm) 16 and 206, 38 and 281; without dout (its last) 42 and 315.

constexpr int kMostThreads = 768;   // of a block, which leaves a thread the 80 registers that the backward pass takes

// Sums over the cluster's blocks, for every thread.  `mine` of each block is free again after
// the cluster's next barrier but one.
template <int N>
__device__ __forceinline__ void cluster_sums(float (&v)[N], float (*mine)[4], int cluster) {
    if (cluster == 1) return;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x < static_cast<unsigned>(cluster)) {
        const uint32_t to = remote_addr(shared_at(mine[rank]), threadIdx.x);
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * i), "f"(v[i]) : "memory");
    }
    cluster_meet();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.0f;
        for (int j = 0; j < cluster; ++j) v[i] += mine[j][i];
    }
}

// load_any, or from 16-byte boundaries.
template <bool ANY>
__device__ __forceinline__ void load_part(const void* p, int dtype, int64_t at, int in, float otherwise, float* v) {
    if (!ANY && p != nullptr) {
        if (in > 0) {
            load8(p, dtype, at, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
    } else {
        load_any(p, dtype, at, in, otherwise, v);
    }
}
template <bool ANY>
__device__ __forceinline__ void store_part(const Mat& m, int64_t at, int in, const float* v) {
    if (ANY) store_chunk_any(m.p, m.dtype, at, in, v);
    else if (in > 0) store8(m.p, m.dtype, at, v);
}

template <bool ANY>
__global__ void __launch_bounds__(kMostThreads) residual_norm_kernel(const ResidualNorm a, int cluster) {
    __shared__ float red[2][1][32];
    __shared__ float joined[2][8][4];
    starts_early();
    after_previous();
    if (cluster > 1) cluster_sync();   // the others' shared memory is there
    const float n = static_cast<float>(a.cols);
    const int64_t c = (static_cast<int64_t>(cluster > 1 ? cluster_rank() : 0) * blockDim.x + threadIdx.x) * 8;
    const int in = inside8(c, a.cols);
    for (int64_t row = blockIdx.x / cluster; row < a.rows; row += gridDim.x / cluster) {
        float s[8], o[8], p[8], g[8], w[8];
        load_part<ANY>(a.o.p, a.o.dtype, row * a.o.ld + c, in, 0.0f, o);
        load_part<ANY>(a.h.p, a.h.dtype, row * a.h.ld + c, in, 0.0f, s);
        load_part<ANY>(a.post, a.param_dtype, c, in, 1.0f, p);
        load_part<ANY>(a.gate, a.param_dtype, c, in, 1.0f, g);
        load_part<ANY>(a.gamma, a.param_dtype, c, in, 1.0f, w);
        float post_rstd = 1.0f;
        if (a.post != nullptr) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < 8; ++j) ss[0] = fmaf(o[j], o[j], ss[0]);
            block_sums(ss, red[0]);
            cluster_sums(ss, joined[0], cluster);
            post_rstd = 1.0f / sqrtf(ss[0] / n + a.eps);
            if (c == 0) a.post_rstd[row] = post_rstd;
        }
        float ss[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = fmaf(a.alpha, s[j], o[j] * post_rstd * p[j] * g[j]);
            if (j < in) ss[0] = fmaf(s[j], s[j], ss[0]);
        }
        store_part<ANY>(a.out, row * a.out.ld + c, in, s);
        if (a.y.p != nullptr) {
            block_sums(ss, red[1]);
            cluster_sums(ss, joined[1], cluster);
            const float rstd = 1.0f / sqrtf(ss[0] / n + a.eps);
            if (c == 0) a.rstd[row] = rstd;
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = s[j] * rstd * w[j];
            store_part<ANY>(a.y, row * a.y.ld + c, in, s);
        }
        if (a.post == nullptr || a.y.p == nullptr) {   // one barrier a row does not keep the rows' sums apart
            if (cluster > 1) cluster_sync();
            else __syncthreads();
        }
    }
}

template <bool ANY>
__global__ void __launch_bounds__(kMostThreads) residual_norm_backward_kernel(const ResidualNormGrad a, int cluster) {
    __shared__ float red[2][3][32];
    __shared__ float joined[2][8][4];
    starts_early();
    after_previous();
    if (cluster > 1) cluster_sync();   // the others' shared memory is there
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    const int64_t c = (static_cast<int64_t>(cluster > 1 ? cluster_rank() : 0) * blockDim.x + threadIdx.x) * 8;
    const int in = inside8(c, a.cols);
    float dg[8], du[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[j] = du[j] = 0.0f;
    int flip = 0;
    for (int64_t row = blockIdx.x / cluster; row < a.rows; row += gridDim.x / cluster) {
        const float rstd = a.dy.p != nullptr ? a.rstd[row] : 0.0f, post_rstd = a.post != nullptr ? a.post_rstd[row] : 1.0f;
        float t[8], xh[8], u[8], k[8], w[8], g[8];
        load_part<ANY>(a.dy.p, a.dy.dtype, row * a.dy.ld + c, in, 0.0f, g);
        load_part<ANY>(a.dy.p != nullptr ? a.out.p : nullptr, a.out.dtype, row * a.out.ld + c, in, 0.0f, xh);
        load_part<ANY>(a.dout.p, a.dout.dtype, row * a.dout.ld + c, in, 0.0f, t);
        load_part<ANY>(a.o.p, a.o.dtype, row * a.o.ld + c, in, 0.0f, u);
        load_part<ANY>(a.gamma, a.param_dtype, c, in, 1.0f, w);
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            xh[j] *= rstd;
            dg[j] = fmaf(g[j], xh[j], dg[j]);
            g[j] *= w[j];
            s[0] = fmaf(g[j], xh[j], s[0]);
            t[j] = fmaf(rstd, g[j], t[j]);
        }
        load_part<ANY>(a.post, a.param_dtype, c, in, 1.0f, k);
        load_part<ANY>(a.gate, a.param_dtype, c, in, 1.0f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            k[j] *= w[j];
            u[j] *= post_rstd;
            s[1] = fmaf(k[j] * u[j], t[j], s[1]);
            s[2] = fmaf(k[j] * u[j], xh[j], s[2]);
        }
        block_sums(s, red[flip]);
        cluster_sums(s, joined[flip], cluster);
        flip ^= 1;
        // with e = t k and t = dout + rstd (g - xh c1), sum(e u) is linear in c1
        const float c1 = s[0] * inv_n, c2 = a.post != nullptr ? (s[1] - rstd * c1 * s[2]) * inv_n : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            t[j] = fmaf(-rstd * c1, xh[j], t[j]);
            du[j] = fmaf(t[j], u[j], du[j]);
            u[j] = post_rstd * fmaf(-u[j], c2, t[j] * k[j]);
            t[j] *= a.alpha;
        }
        store_part<ANY>(a.dh, row * a.dh.ld + c, in, t);
        if (a.dblock.p != nullptr) store_part<ANY>(a.dblock, row * a.dblock.ld + c, in, u);
    }
    float* part = a.partials + static_cast<int64_t>(blockIdx.x / cluster) * 2 * a.cols + c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j < in) {
            part[j] = dg[j];
            part[a.cols + j] = du[j];
        }
    }
}

// ---- rows staged through shared memory ----
//
// BF16 rows, as they come in training.  A block holds G groups of GT threads, each with a
// row (or, in a cluster, a run of its columns); thread t of a group owns its chunks of eight
// columns t + k GT, k < NV, and copies the ones of the rows ahead into a ring of shared
// memory (cp.async), so that it waits for its own copies alone.  ANY: rows start anywhere;
// a chunk is then the two 16-byte words that hold it, moved together when it is read.
// Forward, 4096 x 12288: 66 us, 6.1 TB/s; 4096 x 1280 15 us; 4096 x 5121 (ANY) 91.  Backward, 4096 x 1280: 22 us with 4 us
// for the sums over the blocks, bound by a row's latency at three rows to an SM; 1031 x 5121 (ANY): 35 us,
// seven rows to an SM behind one another; 4096 x 5121 107.

constexpr int kMostPlaces = 4;      // rows of a group in the ring
// Threads of a block by the chunks of one.  The backward pass holds a row's words and its columns' sums:
// 128 registers, or 168 for two chunks (with the 96 and 128 that more threads leave, what is
// spilled goes to L2, for the ring takes L1's room: 4096 x 1280 27 us against 23).
constexpr int forward_threads(int nv) { return nv == 1 ? 768 : 512; }
constexpr int backward_threads(int nv) { return nv == 1 ? 512 : 384; }
constexpr int keep_threads = 512;
constexpr int kRingWarps = 24;

struct RingShape {
    int gt, groups, places, cluster;   // clusters have two chunks to a thread
    int chunks;                     // of a block's share of a row, but for the last one's
};

// A thread's place: its group, its number there, its block's first chunk.  Only a thread's last
// chunk can be short or lie past the share's end (ring_shape has the shares so).
template <int NV>
struct Place {
    int gt, groups, g, t;
    int64_t first;
    int last;                       // columns of the last chunk
    __device__ Place(const RingShape& s, int64_t cols) : gt(s.gt), groups(s.groups), g(threadIdx.x / s.gt), t(threadIdx.x % s.gt) {
        first = NV == 2 && s.cluster > 1 ? static_cast<int64_t>(cluster_rank()) * s.chunks : 0;
        last = t + (NV - 1) * gt < s.chunks ? inside8(column(NV - 1), cols) : 0;
    }
    __device__ int64_t column(int k) const { return (first + t + k * gt) * 8; }
    __device__ int in(int k) const { return k + 1 < NV ? 8 : last; }
};

template <int NV, int M, bool ANY>
struct Ring {
    uint8_t* base;
    static constexpr int kHalves = ANY ? 2 : 1;
    __device__ uint8_t* slot(const Place<NV>& at, int place, int m, int k) const {
        return base + ((((place * M + m) * at.groups + at.g) * NV + k) * kHalves * at.gt + at.t) * 16;
    }
    __device__ void copy(const Place<NV>& at, const Mat& x, int64_t row, int place, int m) const {
        const uint8_t* from = static_cast<const uint8_t*>(x.p) + (row * x.ld + (at.first + at.t) * 8) * 2;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (at.in(k) == 0) continue;
            const uint32_t to = shared_at(slot(at, place, m, k));
            if (ANY) {
                const uintptr_t chunk = reinterpret_cast<uintptr_t>(from + k * at.gt * 16), word = chunk & ~uintptr_t(15);
                copy16(to, reinterpret_cast<const void*>(word));
                if (static_cast<int>(chunk & 15) + 2 * at.in(k) > 16) copy16(to + at.gt * 16, reinterpret_cast<const void*>(word + 16));
            } else {
                copy16(to, from + k * at.gt * 16);
            }
        }
    }
    // The chunk; zeros past the row's end.  (What no copy has written is read too, and dropped: a
    // branch here would keep the reads behind one another, 78 us against 66.)
    __device__ uint4 read(const Place<NV>& at, const Mat& x, int64_t row, int place, int m, int k) const {
        const uint4 lo = *reinterpret_cast<const uint4*>(slot(at, place, m, k));
        if (!ANY) return k + 1 < NV || at.last != 0 ? lo : make_uint4(0, 0, 0, 0);
        const uint4 hi = *reinterpret_cast<const uint4*>(slot(at, place, m, k) + at.gt * 16);
        uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x.p) + static_cast<uintptr_t>(row * x.ld) * 2) & 15u;
        if (off & 8) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (off & 4) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        if (off & 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
        if (k + 1 == NV) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] &= 2 * i + 1 < at.last ? 0xffffffffu : 2 * i < at.last ? 0xffffu : 0u;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ void pairs(uint4 w, f32x2* v) {
    v[0] = pair(bf16_lo(w.x), bf16_hi(w.x));
    v[1] = pair(bf16_lo(w.y), bf16_hi(w.y));
    v[2] = pair(bf16_lo(w.z), bf16_hi(w.z));
    v[3] = pair(bf16_lo(w.w), bf16_hi(w.w));
}
__device__ __forceinline__ void half_pairs(uint4 w, int h, f32x2* v) {
    const uint32_t x = h ? w.z : w.x, y = h ? w.w : w.y;
    v[0] = pair(bf16_lo(x), bf16_hi(x));
    v[1] = pair(bf16_lo(y), bf16_hi(y));
}
__device__ __forceinline__ f32x2 twice(float v) { return pair(v, v); }

// A chunk of an output row; whole warps take part.
template <int NV, bool ANY>
__device__ __forceinline__ void put(const Place<NV>& at, const Mat& m, int64_t row, int k, const f32x2* v) {
    float o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpair(v[j], o[2 * j], o[2 * j + 1]);
    if (ANY) store_chunk_any(m.p, FSDP_DTYPE_BF16, row * m.ld + at.column(k), at.in(k), o);
    else if (at.in(k) != 0) store8(m.p, FSDP_DTYPE_BF16, row * m.ld + at.column(k), o);
}

// The vectors, which all groups share: ones where there is none.  Floats lie in two
// halves of 16 bytes a chunk, so that neighbouring threads' accesses are neighbours.
template <int NV, bool FLOATS>
struct Vectors {
    uint8_t* base;
    static constexpr int kChunk = FLOATS ? 32 : 16;
    __device__ uint8_t* slot(const Place<NV>& at, int v, int k) const { return base + (v * NV + k) * at.gt * kChunk + at.t * 16; }
    // From 16-byte boundaries, of the slots' type: asynchronous.  Places past the row's end are read too, and
    // multiplied by the row's zeros there: they hold ones, for what a kernel before left may be NaN.
    __device__ void copy(const Place<NV>& at, const void* p, int v) const {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            uint8_t* to = slot(at, v, k);
            if (p != nullptr && at.in(k) != 0) {
                const uint8_t* from = static_cast<const uint8_t*>(p) + at.column(k) / 8 * kChunk;
                copy16(shared_at(to), from);
                if (FLOATS) copy16(shared_at(to + at.gt * 16), from + 16);
            } else {
                const uint32_t one = FLOATS ? 0x3f800000u : 0x3f803f80u;
                *reinterpret_cast<uint4*>(to) = make_uint4(one, one, one, one);
                if (FLOATS) *reinterpret_cast<uint4*>(to + at.gt * 16) = make_uint4(one, one, one, one);
            }
        }
    }
    // From anywhere, of either type, to floats.
    __device__ void load(const Place<NV>& at, const void* p, int dtype, int v) const {
        float x[NV][8];
        int in[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            in[k] = at.in(k);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[k][j] = 1.0f;
        }
        if (p != nullptr) load_chunks_any<NV>(p, dtype, at.column(0), in, at.gt * 8, x);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float4* to = reinterpret_cast<float4*>(slot(at, v, k));
            to[0] = make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
            to[at.gt] = make_float4(x[k][4], x[k][5], x[k][6], x[k][7]);
        }
    }
    // All three; `ahead` issues the ring's first copies, of `groups` groups.
    template <bool ANY, typename Ahead>
    __device__ void fill(const Place<NV>& at, const void* v0, const void* v1, const void* v2, int dtype, int groups, Ahead ahead) const {
        if (!ANY) {
            if (at.g == 0) {
                copy(at, v0, 0);
                copy(at, v1, 1);
                copy(at, v2, 2);
            }
            copies_end();
        }
        ahead();
        if (ANY) {
            if constexpr (FLOATS) {
                if (at.g == 0) {
                    load(at, v0, dtype, 0);
                    load(at, v1, dtype, 1);
                    load(at, v2, dtype, 2);
                }
            }
        } else {
            copies_wait(groups);
        }
        __syncthreads();
    }
    // Half a chunk: of floats, a place of its own; of BF16, a half of `whole`.
    __device__ uint4 whole(const Place<NV>& at, int v, int k) const {
        return FLOATS ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(slot(at, v, k));
    }
    __device__ void half(const Place<NV>& at, int v, int k, int h, uint4 w, f32x2* x) const {
        if (FLOATS) {
            const float4 a = *reinterpret_cast<const float4*>(slot(at, v, k) + h * at.gt * 16);
            x[0] = pair(a.x, a.y);
            x[1] = pair(a.z, a.w);
        } else {
            half_pairs(w, h, x);
        }
    }
    __device__ void read(const Place<NV>& at, int v, int k, f32x2* x) const {
        const uint8_t* from = slot(at, v, k);
        if (FLOATS) {
            const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + at.gt * 16);
            x[0] = pair(a.x, a.y);
            x[1] = pair(a.z, a.w);
            x[2] = pair(b.x, b.y);
            x[3] = pair(b.z, b.w);
        } else {
            pairs(*reinterpret_cast<const uint4*>(from), x);
        }
    }
};

// Sums over a group, for all of its threads.  `red` is one of two buffers used in turn: a thread
// that writes one again has passed the barrier behind which every thread had read it.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float4* red, int group, int gt) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    const int warps = gt >> 5;
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float4(v[0], N > 1 ? v[N > 1] : 0.0f, N > 2 ? v[N > 2 ? 2 : 0] : 0.0f, 0.0f);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gt) : "memory");
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < warps; ++i) {
        const float4 r = red[group * warps + i];
        s.x += r.x;
        s.y += r.y;
        s.z += r.z;
    }
    v[0] = s.x;
    if (N > 1) v[N > 1] = s.y;
    if (N > 2) v[N > 2 ? 2 : 0] = s.z;
}

template <int NV, bool FLOATS, bool ANY>
__global__ void __launch_bounds__(forward_threads(NV)) residual_norm_ring_kernel(const __grid_constant__ ResidualNorm a, const RingShape shape) {
    extern __shared__ __align__(16) uint8_t ring_bytes[];
    __shared__ float4 red[2][kRingWarps];
    __shared__ float joined[2][8][4];
    starts_early();
    after_previous();
    const int places = shape.places, cluster = NV == 2 ? shape.cluster : 1;
    if (cluster > 1) cluster_sync();   // the others' shared memory is there
    const Place<NV> at(shape, a.cols);
    const Vectors<NV, FLOATS> vec{ring_bytes};
    const Ring<NV, 2, ANY> ring{ring_bytes + 3 * NV * at.gt * vec.kChunk};
    const int64_t stride = static_cast<int64_t>(gridDim.x / cluster) * at.groups, first = static_cast<int64_t>(blockIdx.x / cluster) * at.groups + at.g;
    const auto issue = [&](int64_t row, int place) {
        if (row < a.rows) {
            ring.copy(at, a.o, row, place, 0);
            ring.copy(at, a.h, row, place, 1);
        }
        copies_end();
    };
    vec.template fill<ANY>(at, a.post, a.gate, a.gamma, a.param_dtype, places - 1, [&] {
        for (int s = 0; s + 1 < places; ++s) issue(first + s * stride, s);
    });
    const float n = static_cast<float>(a.cols);
    const bool tells = at.t == 0 && at.first == 0;   // the statistics
    int place = 0;
    for (int64_t row = first; row < a.rows; row += stride) {
        issue(row + (places - 1) * stride, place == 0 ? places - 1 : place - 1);
        copies_wait(places - 1);
        f32x2 o[NV][4], s[NV][4];
        f32x2 ss = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            pairs(ring.read(at, a.o, row, place, 0, k), o[k]);
            pairs(ring.read(at, a.h, row, place, 1, k), s[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fma2(o[k][j], o[k][j], ss);
        }
        place = place + 1 == places ? 0 : place + 1;
        float post_rstd = 1.0f;
        if (a.post != nullptr) {
            float sum[1] = {both(ss)};
            group_sums(sum, red[0], at.g, at.gt);
            cluster_sums(sum, joined[0], cluster);
            post_rstd = 1.0f / sqrtf(sum[0] / n + a.eps);
            if (tells) a.post_rstd[row] = post_rstd;
        }
        ss = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            f32x2 p[4], w[4];
            vec.read(at, 0, k, p);
            vec.read(at, 1, k, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x2 b = mul2(mul2(mul2(o[k][j], twice(post_rstd)), p[j]), w[j]);
                s[k][j] = fma2(s[k][j], twice(a.alpha), b);
                ss = fma2(s[k][j], s[k][j], ss);   // 0 past the row's end
            }
            put<NV, ANY>(at, a.out, row, k, s[k]);
        }
        float sum[1] = {both(ss)};
        group_sums(sum, red[1], at.g, at.gt);
        cluster_sums(sum, joined[1], cluster);
        const float rstd = 1.0f / sqrtf(sum[0] / n + a.eps);
        if (tells) a.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            f32x2 w[4];
            vec.read(at, 2, k, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[k][j] = mul2(mul2(s[k][j], twice(rstd)), w[j]);
            put<NV, ANY>(at, a.y, row, k, s[k]);
        }
        if (a.post == nullptr) {   // one barrier a row does not keep the rows' sums apart
            if (cluster > 1) cluster_sync();
            else asm volatile("bar.sync %0, %1;" ::"r"(1 + at.g), "r"(at.gt) : "memory");
        }
    }
}

template <int NV, bool FLOATS, bool ANY>
__global__ void __launch_bounds__(backward_threads(NV)) residual_norm_backward_ring_kernel(const __grid_constant__ ResidualNormGrad a,
                                                                                   const RingShape shape) {
    extern __shared__ __align__(16) uint8_t ring_bytes[];
    __shared__ float4 red[2][kRingWarps];
    __shared__ float joined[2][8][4];
    starts_early();
    after_previous();
    const int places = shape.places, cluster = NV == 2 ? shape.cluster : 1;
    if (cluster > 1) cluster_sync();   // the others' shared memory is there
    const Place<NV> at(shape, a.cols);
    const Vectors<NV, FLOATS> vec{ring_bytes};
    const Ring<NV, 4, ANY> ring{ring_bytes + 3 * NV * at.gt * vec.kChunk};
    const int64_t stride = static_cast<int64_t>(gridDim.x / cluster) * at.groups, first = static_cast<int64_t>(blockIdx.x / cluster) * at.groups + at.g;
    const auto issue = [&](int64_t row, int place) {
        if (row < a.rows) {
            ring.copy(at, a.dy, row, place, 0);
            ring.copy(at, a.dout, row, place, 1);
            ring.copy(at, a.out, row, place, 2);
            ring.copy(at, a.o, row, place, 3);
        }
        copies_end();
    };
    vec.template fill<ANY>(at, a.post, a.gate, a.gamma, a.param_dtype, places, [&] {
        for (int s = 0; s < places; ++s) issue(first + s * stride, s);
    });
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    f32x2 dg[NV][4], du[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[k][j] = du[k][j] = 0;
    int place = 0, flip = 0;
    float next1 = 1.0f, next2 = 1.0f;   // the next row's statistics
    const auto statistics = [&](int64_t row) {
        if (row < a.rows) {
            next1 = a.rstd[row];
            if (a.post != nullptr) next2 = a.post_rstd[row];
        }
    };
    statistics(first);
    for (int64_t row = first; row < a.rows; row += stride) {
        const float r1 = next1, r2 = next2;
        statistics(row + stride);
        const f32x2 rstd = twice(r1), post_rstd = twice(r2);
        copies_wait(places - 1);
        // the row's words stay in registers, and their places take the rows ahead at once
        uint4 raw[NV][4];
        f32x2 s1 = 0, s2 = 0, s3 = 0;
        // half a chunk at a time: what is expanded takes fewer registers
        const auto expand = [&](const uint4* w, const uint4* vw, int k, int h, f32x2* xh, f32x2* tt, f32x2* u, f32x2* gr, f32x2* dy, f32x2* kk) {
            half_pairs(w[0], h, dy);
            half_pairs(w[1], h, tt);
            half_pairs(w[2], h, xh);
            half_pairs(w[3], h, u);
            f32x2 g2[2];
            vec.half(at, 0, k, h, vw[0], kk);
            vec.half(at, 1, k, h, vw[1], g2);
            vec.half(at, 2, k, h, vw[2], gr);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                xh[j] = mul2(xh[j], rstd);
                gr[j] = mul2(dy[j], gr[j]);
                tt[j] = fma2(rstd, gr[j], tt[j]);
                u[j] = mul2(u[j], post_rstd);
                kk[j] = mul2(kk[j], g2[j]);
            }
        };
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            raw[k][0] = ring.read(at, a.dy, row, place, 0, k);
            raw[k][1] = ring.read(at, a.dout, row, place, 1, k);
            raw[k][2] = ring.read(at, a.out, row, place, 2, k);
            raw[k][3] = ring.read(at, a.o, row, place, 3, k);
            const uint4 vw[3] = {vec.whole(at, 0, k), vec.whole(at, 1, k), vec.whole(at, 2, k)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x2 xh[2], tt[2], u[2], gr[2], dy[2], kk[2];
                expand(raw[k], vw, k, h, xh, tt, u, gr, dy, kk);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    dg[k][2 * h + j] = fma2(dy[j], xh[j], dg[k][2 * h + j]);
                    s1 = fma2(gr[j], xh[j], s1);
                    const f32x2 ku = mul2(kk[j], u[j]);
                    s2 = fma2(ku, tt[j], s2);
                    s3 = fma2(ku, xh[j], s3);
                }
            }
        }
        issue(row + places * stride, place);
        place = place + 1 == places ? 0 : place + 1;
        float sum[3] = {both(s1), both(s2), both(s3)};
        group_sums(sum, red[flip], at.g, at.gt);
        cluster_sums(sum, joined[flip], cluster);
        flip ^= 1;
        const float c1 = sum[0] * inv_n, c2 = a.post != nullptr ? (sum[1] - r1 * c1 * sum[2]) * inv_n : 0.0f;
        const f32x2 less1 = twice(-r1 * c1), less2 = twice(-c2), alpha = twice(a.alpha);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint4 vw[3] = {vec.whole(at, 0, k), vec.whole(at, 1, k), vec.whole(at, 2, k)};
            f32x2 dh[4], db[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x2 xh[2], tt[2], u[2], gr[2], dy[2], kk[2];
                expand(raw[k], vw, k, h, xh, tt, u, gr, dy, kk);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    tt[j] = fma2(less1, xh[j], tt[j]);
                    du[k][2 * h + j] = fma2(tt[j], u[j], du[k][2 * h + j]);
                    db[2 * h + j] = mul2(post_rstd, fma2(u[j], less2, mul2(tt[j], kk[j])));
                    dh[2 * h + j] = mul2(tt[j], alpha);
                }
            }
            put<NV, ANY>(at, a.dh, row, k, dh);
            put<NV, ANY>(at, a.dblock, row, k, db);
        }
    }
    // the groups' column sums meet in shared memory: element j of chunk i at j * slots + i
    copies_wait(0);
    __syncthreads();
    const int slots = NV * at.gt + 4;
    float* comb = reinterpret_cast<float*>(ring_bytes);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float* to = comb + (at.g * 16 + 2 * j) * slots + at.t + k * at.gt;
            unpair(dg[k][j], to[0], to[slots]);
            unpair(du[k][j], to[8 * slots], to[9 * slots]);
        }
    __syncthreads();
    float* part = a.partials + static_cast<int64_t>(blockIdx.x / cluster) * 2 * a.cols + at.first * 8;
    const int columns = static_cast<int>(max(int64_t(0), min(a.cols - at.first * 8, static_cast<int64_t>(shape.chunks) * 8)));
#pragma unroll
    for (int o = 0; o < 2; ++o)
        for (int c = threadIdx.x; c < columns; c += blockDim.x) {
            const float* from = comb + (o * 8 + (c & 7)) * slots + (c >> 3);
            float s = from[0];
            for (int h = 1; h < at.groups; ++h) s += from[h * 16 * slots];
            part[o * a.cols + c] = s;
        }
}

// The same for rows of 4104 to 12288 columns on 16-byte boundaries, a row to a block: the vectors lie
// in registers, as BF16, and two whole rows in the ring, from which both passes over a
// row read.  (With the vectors in shared memory there is room for one row of 12288; and a thread's three
// chunks, with their columns' sums, leave no registers to hold a row in between, 187 us at 4096 x 12288;
// two blocks to a row, 222: their barrier waits for the slower one's copies.)  4096 x 12288: 116 us, 5.2
// TB/s; the two passes over shared memory and a row's one barrier take as long as its copies.  With a gate, whose
// vector takes registers that are not left, three chunks to a thread spill 200 bytes: 174 us; 4096 x 5120 68.
template <int NV, bool GATE>
__global__ void __launch_bounds__(keep_threads) residual_norm_backward_keep_kernel(const __grid_constant__ ResidualNormGrad a, const RingShape shape) {
    extern __shared__ __align__(16) uint8_t ring_bytes[];
    __shared__ float4 red[2][kRingWarps];
    starts_early();
    after_previous();
    const Place<NV> at(shape, a.cols);
    const Ring<NV, 4, false> ring{ring_bytes};
    const int64_t stride = gridDim.x;
    const auto issue = [&](int64_t row, int place) {
        if (row < a.rows) {
            ring.copy(at, a.dy, row, place, 0);
            ring.copy(at, a.out, row, place, 2);
            ring.copy(at, a.dout, row, place, 1);
            ring.copy(at, a.o, row, place, 3);
        }
        copies_end();
    };
    issue(blockIdx.x, 0);
    uint4 gammas[NV], posts[NV], gates[NV];
    const auto vector = [&](const void* p, uint4* v) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            v[k] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
            if (p != nullptr && at.in(k) != 0) v[k] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at.column(k) * 2);
        }
    };
    vector(a.gamma, gammas);
    vector(a.post, posts);
    if (GATE) vector(a.gate, gates);
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    f32x2 dg[NV][4], du[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[k][j] = du[k][j] = 0;
    int place = 0;
    float next1 = 1.0f, next2 = 1.0f;   // the next row's statistics
    const auto statistics = [&](int64_t row) {
        if (row < a.rows) {
            next1 = a.rstd[row];
            if (a.post != nullptr) next2 = a.post_rstd[row];
        }
    };
    statistics(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += stride) {
        const float r1 = next1, r2 = next2;
        statistics(row + stride);
        issue(row + stride, place ^ 1);
        copies_wait(1);
        const f32x2 rstd = twice(r1), post_rstd = twice(r2);
        // half a chunk at a time, which keeps what is expanded in the registers that are left
        const auto read = [&](int k, uint4* raw) {
            raw[0] = ring.read(at, a.dy, row, place, 0, k);
            raw[1] = ring.read(at, a.dout, row, place, 1, k);
            raw[2] = ring.read(at, a.out, row, place, 2, k);
            raw[3] = ring.read(at, a.o, row, place, 3, k);
        };
        const auto expand = [&](const uint4* raw, int k, int half, f32x2* xh, f32x2* tt, f32x2* u, f32x2* gr, f32x2* dy, f32x2* kk) {
            half_pairs(raw[0], half, dy);
            half_pairs(raw[1], half, tt);
            half_pairs(raw[2], half, xh);
            half_pairs(raw[3], half, u);
            half_pairs(gammas[k], half, gr);
            half_pairs(posts[k], half, kk);
            f32x2 w[2];
            if (GATE) half_pairs(gates[k], half, w);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                xh[j] = mul2(xh[j], rstd);
                gr[j] = mul2(dy[j], gr[j]);
                tt[j] = fma2(rstd, gr[j], tt[j]);
                u[j] = mul2(u[j], post_rstd);
                if (GATE) kk[j] = mul2(kk[j], w[j]);
            }
        };
        f32x2 s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            uint4 raw[4];
            read(k, raw);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                f32x2 xh[2], tt[2], u[2], gr[2], dy[2], kk[2];
                expand(raw, k, half, xh, tt, u, gr, dy, kk);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    dg[k][2 * half + j] = fma2(dy[j], xh[j], dg[k][2 * half + j]);
                    s1 = fma2(gr[j], xh[j], s1);
                    const f32x2 ku = mul2(kk[j], u[j]);
                    s2 = fma2(ku, tt[j], s2);
                    s3 = fma2(ku, xh[j], s3);
                }
            }
        }
        float sum[3] = {both(s1), both(s2), both(s3)};
        group_sums(sum, red[place], 0, at.gt);
        const float c1 = sum[0] * inv_n, c2 = a.post != nullptr ? (sum[1] - r1 * c1 * sum[2]) * inv_n : 0.0f;
        const f32x2 less1 = twice(-r1 * c1), less2 = twice(-c2), alpha = twice(a.alpha);
        uint8_t* dh = static_cast<uint8_t*>(a.dh.p) + (row * a.dh.ld + at.t * 8) * 2;
        uint8_t* db = static_cast<uint8_t*>(a.dblock.p) + (row * a.dblock.ld + at.t * 8) * 2;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            uint32_t h[4], b[4];
            uint4 raw[4];
            read(k, raw);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                f32x2 xh[2], tt[2], u[2], gr[2], dy[2], kk[2];
                expand(raw, k, half, xh, tt, u, gr, dy, kk);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    tt[j] = fma2(less1, xh[j], tt[j]);
                    du[k][2 * half + j] = fma2(tt[j], u[j], du[k][2 * half + j]);
                    u[j] = mul2(post_rstd, fma2(u[j], less2, mul2(tt[j], kk[j])));
                    tt[j] = mul2(tt[j], alpha);
                    float x, y;
                    unpair(tt[j], x, y);
                    h[2 * half + j] = to_bf16x2(x, y);
                    unpair(u[j], x, y);
                    b[2 * half + j] = to_bf16x2(x, y);
                }
            }
            if (k + 1 < NV || at.last != 0) {
                *reinterpret_cast<uint4*>(dh + k * at.gt * 16) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(db + k * at.gt * 16) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
        place ^= 1;
    }
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (k + 1 < NV || at.last != 0) {
            float x[8], y[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                unpair(dg[k][j], x[2 * j], x[2 * j + 1]);
                unpair(du[k][j], y[2 * j], y[2 * j + 1]);
            }
            store8(part, FSDP_DTYPE_F32, at.column(k), x);
            store8(part + a.cols, FSDP_DTYPE_F32, at.column(k), y);
        }
    }
}

// The columns' sums over the blocks, in their order: dgamma from the first half of the
// partial rows, dpost_gamma and dgate from the second.  16 threads of V columns across and
// 16 slices of the blocks down.  Bound by latency: 152 rows of 2 x 1280, 4 us.
template <int V>
__global__ void __launch_bounds__(256) residual_norm_sums_kernel(const ResidualNormGrad a, int64_t count) {
    __shared__ float part[16][16 * V];
    starts_early();
    after_previous();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 16 + tx) * V;
    const float* p = a.partials + blockIdx.y * a.cols + c;
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.0f;
    if (c < a.cols) {
#pragma unroll 10
        for (int64_t i = ty; i < count; i += 16) {
            if constexpr (V == 4) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(p + i * 2 * a.cols));
                s[0] += f.x; s[1] += f.y; s[2] += f.z; s[3] += f.w;
            } else {
                s[0] += __ldcg(p + i * 2 * a.cols);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) part[ty][tx * V + j] = s[j];
    __syncthreads();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 * V + threadIdx.x;
    if (threadIdx.x >= 16 * V || col >= a.cols) return;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += part[i][threadIdx.x];
    const auto put = [&](void* out, const void* by) {
        if (out == nullptr) return;
        float v = by != nullptr ? sum * load1(by, a.param_dtype, col) : sum;
        if (a.accumulate) v += load1(out, a.grad_dtype, col);
        store1(out, a.grad_dtype, col, v);
    };
    if (blockIdx.y == 0) {
        put(a.dgamma, nullptr);
    } else {
        put(a.dpost, a.gate);
        put(a.dgate, a.post);
    }
}

int round32(int64_t n) { return static_cast<int>((n + 31) / 32 * 32); }

// How a chunk to a thread is laid out: 0 threads where eight blocks do not hold a row.
struct Spread {
    int threads = 0, cluster = 1, blocks = 1;   // blocks (or clusters) that run at once on an SM (or its share of SMs)
};
Spread spread(int64_t cols) {
    const int64_t chunks = (cols + 7) / 8;
    Spread s;
    while (s.cluster <= 8 && chunks > static_cast<int64_t>(s.cluster) * kMostThreads) s.cluster *= 2;
    if (s.cluster > 8) return s;
    s.threads = round32((chunks + s.cluster - 1) / s.cluster);
    s.blocks = std::min(8, kMostThreads / s.threads);
    return s;
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned_or_none(const Mat& m) { return m.p == nullptr || rows_aligned(m); }

// How the ring takes `matrices` rows of BF16: chunks to a thread (0: it does not), threads, groups,
// clusters and places.  threads: of a block, by its chunks to a thread; `most` of these at most.
int ring_shape(int64_t rows, int64_t cols, int matrices, bool floats, bool any, int (*threads)(int), int most, int least_places,
               RingShape* s, int* bytes) {
    const int64_t chunks = (cols + 7) / 8;
    for (s->cluster = 1; s->cluster <= 8; s->cluster *= 2) {
        const int64_t share = (chunks + s->cluster - 1) / s->cluster;
        const int nv = s->cluster > 1 ? 2 : share <= threads(1) ? 1 : static_cast<int>((share + threads(2) - 1) / threads(2));
        if (nv > most || share > static_cast<int64_t>(nv) * threads(nv)) continue;
        s->chunks = static_cast<int>(share);
        s->gt = round32((share + nv - 1) / nv);
        s->groups = s->cluster > 1 ? 1 : static_cast<int>(std::min<int64_t>(std::min(threads(nv) / s->gt, 15), rows));
        const int keep = 3 * nv * s->gt * (floats ? 32 : 16), row = matrices * nv * s->gt * (any ? 32 : 16);
        while (s->groups > 1 && keep + least_places * s->groups * row > kSharedMost) --s->groups;
        s->places = std::min(kMostPlaces, (kSharedMost - keep) / (row * s->groups));
        // only a thread's last chunk may lie past the end of a share, the last and smallest one too
        if (s->places < least_places || static_cast<int64_t>(nv - 1) * s->gt > chunks - (s->cluster - 1) * share) continue;
        *bytes = keep + s->places * s->groups * row;
        return nv;
    }
    return 0;
}

}  // namespace

int64_t residual_norm_blocks(int64_t rows, int64_t cols) { return std::min<int64_t>(rows, kSms * spread(cols).blocks); }

cudaError_t launch_residual_norm_forward(const ResidualNorm& a, int sms, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const bool aligned = a.cols % 8 == 0 && rows_aligned(a.h) && aligned_or_none(a.o) && rows_aligned(a.out) && aligned_or_none(a.y) &&
                         on16(a.post) && on16(a.gate) && on16(a.gamma);
    const bool half = a.o.p != nullptr && a.y.p != nullptr && a.h.dtype == FSDP_DTYPE_BF16 && a.o.dtype == FSDP_DTYPE_BF16 &&
                      a.out.dtype == FSDP_DTYPE_BF16 && a.y.dtype == FSDP_DTYPE_BF16;
    const bool floats = !aligned || a.param_dtype == FSDP_DTYPE_F32;
    RingShape shape;
    int bytes = 0;
    const int nv = half ? ring_shape(a.rows, a.cols, 2, floats, !aligned, forward_threads, 3, 2, &shape, &bytes) : 0;
    if (nv != 0 && a.rows * shape.cluster >= 2 * static_cast<int64_t>(sms) * shape.groups) {   // rows enough for every group to walk two
        const unsigned clusters = static_cast<unsigned>(std::min<int64_t>((a.rows + shape.groups - 1) / shape.groups, sms / shape.cluster));
        const int threads = shape.gt * shape.groups;
#define RING_(nv_, f, any)                                                                                                       \
    if (nv == nv_ && floats == f && aligned != any)                                                                              \
        return launch_shared_clusters<residual_norm_ring_kernel<nv_, f, any>>(clusters * shape.cluster, threads, bytes, shape.cluster, st, a, shape);
#define RING(nv_) RING_(nv_, false, false) RING_(nv_, true, false) RING_(nv_, true, true)
        RING(1) RING(2) RING(3)
#undef RING
#undef RING_
    }
    const Spread s = spread(a.cols);
    if (s.threads != 0) {
        const int64_t most = std::max<int64_t>(1, static_cast<int64_t>(sms) * std::min(16, 2048 / s.threads) / s.cluster);
        const dim3 grid(static_cast<unsigned>(std::min(a.rows, most) * s.cluster));
        return launch_early_clusters(aligned ? residual_norm_kernel<false> : residual_norm_kernel<true>, grid, s.threads, 0, s.cluster, st, a, s.cluster);
    }
    return launch_early(residual_norm_any_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t(1) << 30))), 512, 0, st, a);
}

cudaError_t launch_residual_norm_backward(const ResidualNormGrad& a, int sms, cudaStream_t st) {
    const bool aligned = a.cols % 8 == 0 && aligned_or_none(a.dy) && aligned_or_none(a.dout) && aligned_or_none(a.out) && aligned_or_none(a.o) &&
                         rows_aligned(a.dh) && aligned_or_none(a.dblock) && on16(a.post) && on16(a.gate) && on16(a.gamma);
    const bool half = a.dy.p != nullptr && a.dout.p != nullptr && a.o.p != nullptr && a.dy.dtype == FSDP_DTYPE_BF16 &&
                      a.dout.dtype == FSDP_DTYPE_BF16 && a.out.dtype == FSDP_DTYPE_BF16 && a.o.dtype == FSDP_DTYPE_BF16 &&
                      a.dh.dtype == FSDP_DTYPE_BF16 && a.dblock.dtype == FSDP_DTYPE_BF16;
    const bool floats = !aligned || a.param_dtype == FSDP_DTYPE_F32;
    int64_t count = 0;   // of partial rows
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) {
        RingShape shape;
        int bytes = 0;
        const int nv = half ? ring_shape(a.rows, a.cols, 4, floats, !aligned, backward_threads, 2, 1, &shape, &bytes) : 0;
        const Spread s = spread(a.cols);
        const int64_t chunks = a.cols / 8;
        if (half && !floats && chunks > backward_threads(1) && chunks <= 3 * keep_threads) {
            const int keep = chunks <= 2 * keep_threads ? 2 : 3;
            shape.cluster = shape.groups = 1;
            shape.places = 2;
            shape.chunks = static_cast<int>(chunks);
            shape.gt = round32((chunks + keep - 1) / keep);
            count = std::min<int64_t>(a.rows, sms);
            bytes = 2 * 4 * keep * shape.gt * 16;
            const unsigned blocks = static_cast<unsigned>(count);
#define KEEP(nv_, g) launch_shared<residual_norm_backward_keep_kernel<nv_, g>>(blocks, shape.gt, bytes, st, a, shape)
            if (a.gate != nullptr) e = keep == 2 ? KEEP(2, true) : KEEP(3, true);
            else e = keep == 2 ? KEEP(2, false) : KEEP(3, false);
#undef KEEP
        } else if (nv != 0) {
            count = std::min<int64_t>((a.rows + shape.groups - 1) / shape.groups, sms / shape.cluster);
            const unsigned blocks = static_cast<unsigned>(count * shape.cluster);
            const int threads = shape.gt * shape.groups;
            bytes = std::max(bytes, shape.groups * 16 * (nv * shape.gt + 4) * 4);
            e = cudaErrorInvalidConfiguration;
#define RING_(nv_, f, any)                                                                                                       \
    if (nv == nv_ && floats == f && aligned != any)                                                                              \
        e = launch_shared_clusters<residual_norm_backward_ring_kernel<nv_, f, any>>(blocks, threads, bytes, shape.cluster, st, a, shape);
#define RING(nv_) RING_(nv_, false, false) RING_(nv_, true, false) RING_(nv_, true, true)
            RING(1) RING(2)
#undef RING
#undef RING_
        } else if (s.threads != 0) {
            count = std::min(a.rows, std::max<int64_t>(1, static_cast<int64_t>(sms) * s.blocks / s.cluster));
            e = launch_early_clusters(aligned ? residual_norm_backward_kernel<false> : residual_norm_backward_kernel<true>,
                                      dim3(static_cast<unsigned>(count * s.cluster)), s.threads, 0, s.cluster, st, a, s.cluster);
        } else {
            count = std::min<int64_t>(a.rows, sms);
            e = launch_early(residual_norm_any_backward_kernel, dim3(static_cast<unsigned>(count)), 512, 0, st, a);
        }
    }
    if (e != cudaSuccess || (a.dgamma == nullptr && a.dpost == nullptr && a.dgate == nullptr)) return e;
    const bool vec = a.cols % 4 == 0;   // the workspace is aligned
    const dim3 grid(static_cast<unsigned>(vec ? (a.cols + 63) / 64 : (a.cols + 15) / 16), 2);
    return launch_early(vec ? residual_norm_sums_kernel<4> : residual_norm_sums_kernel<1>, grid, 256, 0, st, a, count);
}

}  // namespace fsdp
