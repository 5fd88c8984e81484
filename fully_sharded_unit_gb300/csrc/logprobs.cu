// Log probabilities of given tokens, their entropy and most likely alternatives, and
// the logits' gradient.
#include <algorithm>
#include <cmath>

#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {
namespace {

constexpr int kMostThreads = 512;
constexpr int kWords = 4;            // 16-byte words of a thread in a group
constexpr int kMostCluster = 8;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kNone = -200.0f;     // 2^kNone is 0 in fp32
constexpr unsigned kAll = 0xffffffffu;
constexpr float kInf = __builtin_inff();

// A row's logits as the 16-byte words that hold them: rows start anywhere, and the
// elements of the first and last word that are not the row's count as -inf.
template <bool BF16>
struct RowWords {
    static constexpr int E = BF16 ? 8 : 4;
    const uint4* words;
    int count, cols;
    int lead;        // elements of the first word before the row

    __device__ RowWords(const Mat& z, int64_t row, int64_t cols_) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(z.p) + static_cast<uintptr_t>(row * z.ld) * (16 / E);
        words = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
        lead = static_cast<int>(at & 15) / (16 / E);
        cols = static_cast<int>(cols_);
        count = (lead + cols + E - 1) / E;
    }
    __device__ int column(int w, int j) const { return w * E - lead + j; }
    __device__ bool inside(int i) const { return i >= 0 && i < cols; }
    __device__ static uint4 none() {
        const uint32_t x = BF16 ? 0xff80ff80u : 0xff800000u;
        return make_uint4(x, x, x, x);
    }
    // The first or last word, or one behind it.
    __device__ uint4 edge(int w) const {
        uint4 v = none();
        if (w >= count) return v;
        v = words[w];
        uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if (inside(column(w, j))) continue;
            if (BF16) x[j / 2] = j & 1 ? (x[j / 2] & 0xffffu) | 0xff800000u : (x[j / 2] & 0xffff0000u) | 0xff80u;
            else x[j] = 0xff800000u;
        }
        return make_uint4(x[0], x[1], x[2], x[3]);
    }
    __device__ uint4 load(int w) const {
        return w > 0 && w < count - 1 ? words[w] : edge(w);
    }
    __device__ static void floats(uint4 v, float* f) {
        if constexpr (BF16) {
            unpack8(v, f);
        } else {
            f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
        }
    }
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest of N words' elements; NaN are passed over.
template <bool BF16, int N>
__device__ __forceinline__ float largest(const uint4* v) {
    if constexpr (BF16) {
        uint32_t m = 0xff80ff80u;
#pragma unroll
        for (int k = 0; k < N; ++k) m = max_bf16x2(m, max_bf16x2(max_bf16x2(v[k].x, v[k].y), max_bf16x2(v[k].z, v[k].w)));
        return fmaxf(bf16_lo(m), bf16_hi(m));
    } else {
        float m = -kInf;
#pragma unroll
        for (int k = 0; k < N; ++k)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[k].x), __uint_as_float(v[k].y)), fmaxf(__uint_as_float(v[k].z), __uint_as_float(v[k].w))));
        return m;
    }
}

// The running maximum m of some logits, S = sum 2^((z - m) c) and Q = sum of
// 2^((z - m) c) (z - m) c, c = scale log2(e).
struct Soft {
    float m, S, Q;
};

__device__ __forceinline__ float grown(float from, float to, float c) { return fmaxf((from - to) * c, kNone); }

__device__ __forceinline__ void rescale(Soft& s, float to, float c) {
    const float d = grown(s.m, to, c), f = exp2_fast(d);
    s.Q = f * fmaf(d, s.S, s.Q);
    s.S *= f;
    s.m = to;
}

__device__ __forceinline__ Soft join(Soft a, Soft b, float c) {
    const float m = fmaxf(a.m, b.m);
    rescale(a, m, c);
    rescale(b, m, c);
    return Soft{m, a.S + b.S, a.Q + b.Q};
}

// Adds a word's elements to s, whose m is at least as large as they are.
// Q's terms must not have d = -inf.  A bf16 logit is held at -2^100 first, two at a time, which
// is as good as masked while m is below 2^99 in magnitude and c is small enough for d to stay finite
// (`plain`); otherwise d itself is held.
template <bool BF16, bool ENTROPY>
__device__ __forceinline__ void add_word(Soft& s, f32x2& S2, f32x2& Q2, uint4 v, float ref, float c, bool plain) {
    constexpr int E = RowWords<BF16>::E;
    float z[8];
    if (BF16 && ENTROPY && plain) {
        constexpr uint32_t kFloor = 0xf180f180u;   // -2^100
        v = make_uint4(max_nan_bf16x2(v.x, kFloor), max_nan_bf16x2(v.y, kFloor), max_nan_bf16x2(v.z, kFloor), max_nan_bf16x2(v.w, kFloor));
    }
    RowWords<BF16>::floats(v, z);
    const f32x2 less = pair(-ref, -ref), c2 = pair(c, c);
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        float d0, d1;
        unpair(mul2(add2(pair(z[j], z[j + 1]), less), c2), d0, d1);
        if (ENTROPY && !(BF16 && plain)) {
            d0 = max_nan(d0, kNone);
            d1 = max_nan(d1, kNone);
        }
        const f32x2 e = pair(exp2_fast(d0), exp2_fast(d1));
        S2 = add2(S2, e);
        if (ENTROPY) Q2 = fma2(e, pair(d0, d1), Q2);
    }
}

// Orders like the logits, -0 like 0.
__device__ __forceinline__ uint32_t order(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unorder(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

// Larger logits first, lower indices first among equals; no two of a row are equal,
// and none is 0.
using Key = unsigned long long;
__device__ __forceinline__ Key key_of(float z, int64_t i) {
    return (static_cast<Key>(order(z)) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
}

constexpr int kLists = 64;      // of as many neighbouring threads each
constexpr int kRoom = 2048;     // candidates

struct TopShared {
    Key best[kLists];
    Key found[kRoom];
    Key got[kMostTop];
    Key floor;
    int count;
};

// Puts the `top` largest of `count` keys into `to`, in order.
__device__ __forceinline__ void rank_keys(const Key* keys, int count, int top, Key* to) {
    for (int i = threadIdx.x; i < count; i += blockDim.x) {
        const Key k = keys[i];
        int above = 0;
        for (int j = 0; j < count; ++j) above += keys[j] > k;
        if (above < top && k != 0) to[above] = k;
    }
}

// The `top` largest keys of the words [first, end), in order, into s.got (0 where the words
// hold fewer).  Every one of them is at least the top-th largest of the lists' maxima; a
// warp looks through the elements of each of its threads whose largest key (`mine`) reaches that.
template <bool BF16>
__device__ void top_keys(const RowWords<BF16>& r, int first, int end, int top, Key mine, TopShared& s) {
    constexpr int E = RowWords<BF16>::E;
    const int t = threadIdx.x, lane = t & 31, threads = blockDim.x, width = threads / kLists;
    Key list = mine;
    for (int d = 1; d < width; d <<= 1) list = max(list, __shfl_xor_sync(kAll, list, d));
    if ((t & (width - 1)) == 0) s.best[t / width] = list;
    if (t < kMostTop) s.got[t] = 0;
    if (t == 0) {
        s.count = 0;
        s.floor = 0;
    }
    __syncthreads();
    if (t < kLists) {
        const Key k = s.best[t];
        int above = 0;
        for (int i = 0; i < kLists; ++i) above += s.best[i] > k;
        if (above == top - 1 && k != 0) s.floor = k;   // one list's, or none if fewer than `top` hold any
    }
    __syncthreads();
    const Key floor = s.floor;
    const auto each = [&](int from, int step, auto f) {
        for (int w = from; w < end; w += step) {
            float z[8];
            RowWords<BF16>::floats(r.load(w), z);
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (r.inside(r.column(w, j))) f(key_of(z[j], r.column(w, j)));
        }
    };
    for (unsigned who = __ballot_sync(kAll, mine >= floor && mine != 0); who != 0; who &= who - 1) {
        const int thread = (t & ~31) + __ffs(who) - 1;
        each(first + thread + lane * threads, 32 * threads, [&](Key k) {
            if (k >= floor) {
                const int at = atomicAdd(&s.count, 1);
                if (at < kRoom) s.found[at] = k;
            }
        });
    }
    __syncthreads();
    const int count = s.count;
    if (count <= kRoom) {
        rank_keys(s.found, count, top, s.got);
    } else {   // more than there is room for: one after the other
        Key last = ~Key(0);
        for (int n = 0; n < top; ++n) {
            Key k = 0;
            each(first + t, threads, [&](Key x) { k = x < last ? max(k, x) : k; });
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) k = max(k, __shfl_xor_sync(kAll, k, d));
            if (lane == 0) s.best[t >> 5] = k;
            __syncthreads();
            for (int i = 0; i < threads / 32; ++i) k = max(k, s.best[i]);
            last = k;
            if (t == 0) s.got[n] = k;
            __syncthreads();
        }
    }
    __syncthreads();
}

// ---- gradient ----

struct RowGrad {
    float a, b;       // scale a (0 without a token), scale b
    float m, ln2s;    // max z, log2 S
    float h;          // entropy
    int64_t token;    // -1: none
    bool zero;        // the whole row
};

// p (-(a + b h) - b ln p) of eight logits; and a at the token.
__device__ __forceinline__ void logit_grads(float* v, float c, const RowGrad& g) {
    const f32x2 less = pair(-g.m, -g.m), c2 = pair(c, c), l = pair(-g.ln2s, -g.ln2s);
    const float a1 = -fmaf(g.b, g.h, g.a), b1 = -g.b * kLn2;
    const f32x2 a2 = pair(a1, a1), b2 = pair(b1, b1);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float x0, x1;
        unpair(fma2(add2(pair(v[j], v[j + 1]), less), c2, l), x0, x1);
        if (b1 != 0.0f) {
            x0 = max_nan(x0, kNone);
            x1 = max_nan(x1, kNone);
            unpair(mul2(pair(exp2_fast(x0), exp2_fast(x1)), fma2(pair(x0, x1), b2, a2)), v[j], v[j + 1]);
        } else {
            unpair(mul2(pair(exp2_fast(x0), exp2_fast(x1)), a2), v[j], v[j + 1]);
        }
    }
}

__device__ __forceinline__ int grad_lead(const TokenLogprobs& a, int64_t row) {
    const bool half = a.dz.dtype == FSDP_DTYPE_BF16;
    const uintptr_t to = reinterpret_cast<uintptr_t>(a.dz.p) + static_cast<uintptr_t>(row * a.dz.ld) * (half ? 2 : 4);
    return static_cast<int>(to & 15) / (half ? 2 : 4);
}
__device__ __forceinline__ int grad_chunks(const TokenLogprobs& a, int64_t row) {
    return (grad_lead(a, row) + static_cast<int>(a.vocab) + 7) / 8;
}

// dz of the row's chunks of eight in [begin, end), by all the threads of a block.  Chunks start
// on 16-byte boundaries of dz; logits that do not start with them are read as the words that
// hold them.
template <bool ZHALF, bool DHALF>
__device__ __forceinline__ void row_gradient(const TokenLogprobs& a, int64_t row, const RowGrad& g, int begin, int end) {
    constexpr int kZ = ZHALF ? FSDP_DTYPE_BF16 : FSDP_DTYPE_F32, kD = DHALF ? FSDP_DTYPE_BF16 : FSDP_DTYPE_F32;
    constexpr int N = ZHALF ? 4 : 2, W = ZHALF ? 1 : 2;   // chunks in flight; words of a chunk
    const float c = a.scale * kLog2e;
    const int lead = grad_lead(a, row), vocab = static_cast<int>(a.vocab), t = threadIdx.x, threads = blockDim.x;
    const int64_t zrow = row * a.z.ld, drow = row * a.dz.ld;
    // a row's ends, an element to a thread
    const int last = (lead + vocab - 1) / 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int q = h == 0 ? 0 : last, i = q * 8 - lead + t;
        if ((h == 0 ? lead > 0 || vocab < 8 : last > 0 && (lead + vocab) % 8 != 0) && q >= begin && q < end && t < 8 && i >= 0 && i < vocab) {
            float x[8] = {};
            if (!g.zero) {
                x[0] = load1(a.z.p, kZ, zrow + i);
                logit_grads(x, c, g);
                if (g.token == i) x[0] += g.a;
            }
            store1(a.dz.p, kD, drow + i, x[0]);
        }
    }
    begin = max(begin, lead > 0 ? 1 : 0);
    end = min(end, (lead + vocab) / 8);
    const bool direct = ((reinterpret_cast<uintptr_t>(a.z.p) + static_cast<uintptr_t>((zrow - lead) * (ZHALF ? 2 : 4))) & 15) == 0;
    const int hit = g.token >= 0 && g.token < vocab ? (static_cast<int>(g.token) + lead) / 8 : -1;   // the token's chunk
    const auto finish = [&](int q, float* v) {
        logit_grads(v, c, g);
        if (q == hit) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (static_cast<int>(g.token) + lead == q * 8 + j) v[j] += g.a;
        }
        store8(a.dz.p, kD, drow + q * 8 - lead, v);
    };
    if (g.zero) {
        const float v[8] = {};
        for (int q = begin + t; q < end; q += threads) store8(a.dz.p, kD, drow + q * 8 - lead, v);
    } else if (direct) {
        const uint4* words = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.z.p) + (zrow - lead) * (ZHALF ? 2 : 4));
        for (int q0 = begin + t; q0 < end; q0 += N * threads) {
            uint4 w[N][W];
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (q0 + k * threads < end) w[k][i] = words[(q0 + k * threads) * W + i];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (q0 + k * threads < end) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < W; ++i) RowWords<ZHALF>::floats(w[k][i], v + 4 * i);
                    finish(q0 + k * threads, v);
                }
            }
        }
    } else {
        for (int q = begin + t; q < end; q += threads) {
            float v[8];
            const int n = 8;
            load_chunks_any<1>(a.z.p, kZ, zrow + q * 8 - lead, &n, 0, &v);
            finish(q, v);
        }
    }
}

template <bool ZHALF>
__device__ __forceinline__ void row_gradient(const TokenLogprobs& a, int64_t row, const RowGrad& g, int begin, int end) {
    if (a.dz.dtype == FSDP_DTYPE_BF16) row_gradient<ZHALF, true>(a, row, g, begin, end);
    else row_gradient<ZHALF, false>(a, row, g, begin, end);
}

__device__ RowGrad row_grad(const TokenLogprobs& a, int64_t row, float m, float ln_s, float h) {
    RowGrad g;
    g.token = a.dlogprob != nullptr ? a.tokens[row] : -1;
    g.a = g.token >= 0 ? a.dlogprob[row] * a.scale : 0.0f;
    g.b = a.dentropy != nullptr ? a.dentropy[row] * a.scale : 0.0f;
    // a masked row's S is 0; a token that does not exist leaves nothing to say
    g.zero = (g.a == 0.0f && g.b == 0.0f) || ln_s == -kInf;
    if (g.token >= a.vocab) {
        g.a = __uint_as_float(0x7fc00000u);
        g.zero = false;
    }
    g.m = m;
    g.ln2s = ln_s * kLog2e;
    g.h = g.b != 0.0f ? h : 0.0f;
    return g;
}

// ---- kernels ----

// A row to a block, or to a cluster of blocks that have a run of its words each.
template <bool BF16, bool ENTROPY, bool GRAD>
__global__ void __launch_bounds__(kMostThreads, 2) token_logprobs_kernel(const TokenLogprobs a, int cluster) {
    constexpr int E = RowWords<BF16>::E;
    __shared__ TopShared tops;
    __shared__ Soft softs[kMostThreads / 32], joined[kMostCluster];
    starts_early();
    after_previous();
    if (cluster > 1) cluster_sync();   // the others' shared memory is there
    const int t = threadIdx.x, lane = t & 31, threads = blockDim.x;
    const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const float c = a.scale * kLog2e;
    for (int64_t row = blockIdx.x / cluster; row < a.rows; row += gridDim.x / cluster) {
        const RowWords<BF16> r(a.z, row, a.vocab);
        const int first = static_cast<int>(static_cast<int64_t>(r.count) * rank / cluster);
        const int end = static_cast<int>(static_cast<int64_t>(r.count) * (rank + 1) / cluster);
        Soft s{-kInf, 0.0f, 0.0f};
        int best = first + t;   // the first word of the group that holds the largest logit
        const auto load = [&](int w) { return w < end ? r.load(w) : r.none(); };
        uint4 next[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k) next[k] = load(first + t + k * threads);
        for (int w = first + t; w < end; w += kWords * threads) {
            uint4 v[kWords];
#pragma unroll
            for (int k = 0; k < kWords; ++k) v[k] = next[k];
#pragma unroll
            for (int k = 0; k < kWords; ++k) next[k] = load(w + (kWords + k) * threads);
            const float top = largest<BF16, kWords>(v);
            if (top > s.m) {
                rescale(s, top, c);
                best = w;
            }
            const float ref = s.m == -kInf ? 0.0f : s.m;
            f32x2 S2 = pair(s.S, 0.0f), Q2 = pair(s.Q, 0.0f);
            if (fabsf(s.m) < 0x1p99f && c < 0x1p20f) {
#pragma unroll
                for (int k = 0; k < kWords; ++k) add_word<BF16, ENTROPY>(s, S2, Q2, v[k], ref, c, true);
            } else {
#pragma unroll
                for (int k = 0; k < kWords; ++k) add_word<BF16, ENTROPY>(s, S2, Q2, v[k], ref, c, false);
            }
            float x, y;
            unpair(S2, x, y);
            s.S = x + y;
            unpair(Q2, x, y);
            s.Q = x + y;
        }
        // the thread's largest logit's key: the first of its group that equals it
        Key mine = 0;
        if (a.top > 0) {
            for (int k = 0; k < kWords; ++k) {
                const int w = best + k * threads;
                if (w >= end) break;
                float z[8];
                RowWords<BF16>::floats(r.load(w), z);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (mine == 0 && z[j] == s.m && r.inside(r.column(w, j))) mine = key_of(z[j], r.column(w, j));
            }
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            s = join(s, Soft{__shfl_xor_sync(kAll, s.m, d), __shfl_xor_sync(kAll, s.S, d), __shfl_xor_sync(kAll, s.Q, d)}, c);
        if (lane == 0) softs[t >> 5] = s;
        __syncthreads();
        s = softs[0];
        for (int i = 1; i < threads / 32; ++i) s = join(s, softs[i], c);
        if (cluster > 1) {
            if (t < cluster) {
                const uint32_t to = remote_addr(static_cast<uint32_t>(__cvta_generic_to_shared(&joined[rank])), t);
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(s.m) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(s.S) : "memory");
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(s.Q) : "memory");
            }
            cluster_sync();
            s = joined[0];
            for (int i = 1; i < cluster; ++i) s = join(s, joined[i], c);
        }
        const bool bad = !(s.S == s.S);
        const float ln_s = logf(s.S);
        const float h = s.S == 0.0f ? 0.0f : fmaf(-kLn2, s.Q / s.S, ln_s);
        if (t == 0 && rank == 0) {
            if (a.tokens != nullptr) {
                const int64_t token = a.tokens[row];
                float lp = 0.0f;
                if (token >= a.vocab) {
                    lp = __uint_as_float(0x7fc00000u);
                    atomicOr(a.status, FSDP_KSTATUS_BAD_TOKEN);
                } else if (token >= 0) {
                    lp = s.S == 0.0f ? -kInf : fmaf(load1(a.z.p, a.z.dtype, row * a.z.ld + token) - s.m, a.scale, -ln_s);
                }
                a.logprob[row] = lp;
            }
            if (ENTROPY && a.entropy != nullptr) a.entropy[row] = h;
            if (a.stats != nullptr) {
                a.stats[2 * row] = s.m;
                a.stats[2 * row + 1] = ln_s;
            }
        }
        if (a.top > 0) {
            if (!bad) top_keys<BF16>(r, first, end, a.top, mine, tops);
            if (cluster > 1) {   // the blocks' lists meet in the first one's candidates
                const uint32_t to = remote_addr(static_cast<uint32_t>(__cvta_generic_to_shared(&tops.found[rank * kMostTop])), 0);
                const Key k = t < kMostTop ? tops.got[t] : 0;
                cluster_sync();
                if (t < kMostTop) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to + 8 * t), "l"(k) : "memory");
                cluster_sync();
                if (rank == 0 && !bad) rank_keys(tops.found, cluster * kMostTop, a.top, tops.got);
                __syncthreads();
            }
            if (rank == 0 && t < a.top) {
                const Key k = bad ? 0 : tops.got[t];
                a.top_tokens[row * a.top + t] = bad ? -1 : static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(k));
                a.top_logprobs[row * a.top + t] = bad ? __uint_as_float(0x7fc00000u)
                                                      : s.S == 0.0f ? -kInf : fmaf(unorder(static_cast<uint32_t>(k >> 32)) - s.m, a.scale, -ln_s);
            }
        }
        // what the next row or the gradient writes is read: the sums, the alternatives, the token's logit
        if (cluster > 1) cluster_sync();
        else __syncthreads();
        if constexpr (GRAD) {
            const int chunks = grad_chunks(a, row);
            row_gradient<BF16>(a, row, row_grad(a, row, s.m, ln_s, h), static_cast<int>(static_cast<int64_t>(chunks) * rank / cluster),
                               static_cast<int>(static_cast<int64_t>(chunks) * (rank + 1) / cluster));
        }
    }
}

// `parts` blocks to a row, which have a run of its chunks each.
template <bool BF16>
__global__ void __launch_bounds__(256) token_logprobs_backward_kernel(const TokenLogprobs a, int parts) {
    starts_early();
    after_previous();
    const int part = blockIdx.x % parts;
    for (int64_t row = blockIdx.x / parts; row < a.rows; row += gridDim.x / parts) {
        const float m = a.stats[2 * row], ln_s = a.stats[2 * row + 1];
        const RowGrad g = row_grad(a, row, m, ln_s, a.entropy != nullptr ? a.entropy[row] : 0.0f);
        if (threadIdx.x == 0 && part == 0 && g.token >= a.vocab) atomicOr(a.status, FSDP_KSTATUS_BAD_TOKEN);
        const int chunks = grad_chunks(a, row);
        row_gradient<BF16>(a, row, g, static_cast<int>(static_cast<int64_t>(chunks) * part / parts),
                           static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / parts));
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenLogprobs& a, int sms, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const bool half = a.z.dtype == FSDP_DTYPE_BF16, grad = a.dz.p != nullptr;
    const bool entropy = a.entropy != nullptr || a.dentropy != nullptr;
    // threads to a row: as many as fill the SMs, in blocks of 128 to 512 and clusters of up to
    // eight, but two words at least to each
    const int64_t words = a.vocab * (half ? 2 : 4) / 16 + 1;
    const int64_t wanted = std::min<int64_t>(static_cast<int64_t>(sms) * 1024 / a.rows, words / 2);
    int threads = 128, cluster = 1;
    while (threads < kMostThreads && threads < wanted) threads *= 2;
    while (cluster < kMostCluster && threads * cluster < wanted) cluster *= 2;
    const int64_t rows = std::min<int64_t>(a.rows, int64_t(1) << 27);
#define RUN(h, e, g) return launch_early_clusters(token_logprobs_kernel<h, e, g>, dim3(static_cast<unsigned>(rows * cluster)), threads, 0, cluster, st, a, cluster)
    if (half) {
        if (entropy) { if (grad) RUN(true, true, true); RUN(true, true, false); }
        if (grad) RUN(true, false, true);
        RUN(true, false, false);
    }
    if (entropy) { if (grad) RUN(false, true, true); RUN(false, true, false); }
    if (grad) RUN(false, false, true);
    RUN(false, false, false);
#undef RUN
}

cudaError_t launch_token_logprobs_backward(const TokenLogprobs& a, int sms, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    // few rows are shared by blocks, down to a group of chunks to a thread
    const int64_t most = a.vocab / (8 * 4 * 256) + 1;
    const int64_t parts = std::max<int64_t>(1, std::min(most, static_cast<int64_t>(sms) * 8 / a.rows));
    const int64_t rows = std::min(a.rows, (int64_t(1) << 30) / parts);
    return launch_early(a.z.dtype == FSDP_DTYPE_BF16 ? token_logprobs_backward_kernel<true> : token_logprobs_backward_kernel<false>,
                        dim3(static_cast<unsigned>(rows * parts)), 256, 0, st, a, static_cast<int>(parts));
}

}  // namespace fsdp
