// Log probabilities of given tokens, their entropy and most likely alternatives, and
// the logits' gradient.
#include <algorithm>
#include <cmath>

#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {
namespace {

constexpr int kThreads = 512;
constexpr int kWords = 4;            // 16-byte words of a thread in flight
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
    int64_t count;
    int lead;        // elements of the first word before the row
    int64_t cols;

    __device__ RowWords(const Mat& z, int64_t row, int64_t cols_) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(z.p) + static_cast<uintptr_t>(row * z.ld) * (16 / E);
        words = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
        lead = static_cast<int>(at & 15) / (16 / E);
        cols = cols_;
        count = (lead + cols + E - 1) / E;
    }
    static __device__ uint4 none() { return BF16 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                                                 : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    // Word w, none() past the end.
    __device__ uint4 load(int64_t w, int64_t end) const {
        uint4 v = none();
        if (w < end) v = words[w];
        return v;
    }
    // The word's elements as floats.
    __device__ void floats(uint4 v, int64_t w, float* f) const {
        if constexpr (BF16) {
            unpack8(v, f);
        } else {
            f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
        }
        if (w == 0 || w + 1 == count) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int64_t i = w * E - lead + j;
                if (i < 0 || i >= cols) f[j] = -kInf;
            }
        }
    }
};

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

constexpr int kLists = kThreads / 8;   // eight lanes' largest keys make a list
constexpr int kRoom = 2048;            // candidates

struct TopShared {
    Key best[kLists];
    Key found[kRoom];
    Key got[kMostTop];
    Key floor;
    int count;
};

// The `top` largest keys of the words [first, end), in order, into s.got (0 where the row
// has fewer).  Every element that is among them is at least the top-th largest of the
// lists' maxima, of which the threads that hold one such look through their elements
// again.  `mine`: the thread's largest key.
template <bool BF16>
__device__ void top_keys(const RowWords<BF16>& r, int64_t first, int64_t end, int top, Key mine, TopShared& s) {
    constexpr int E = RowWords<BF16>::E;
    const int t = threadIdx.x, lane = t & 31;
    Key list = mine;
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) list = max(list, __shfl_xor_sync(kAll, list, d));
    if ((lane & 7) == 0) s.best[t >> 3] = list;
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
    const auto each = [&](auto f) {
        for (int64_t w = first + t; w < end; w += kThreads) {
            float z[E];
            r.floats(r.words[w], w, z);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int64_t i = w * E - r.lead + j;
                if (i >= 0 && i < r.cols) f(key_of(z[j], i));
            }
        }
    };
    if (mine >= floor && mine != 0) {
        each([&](Key k) {
            if (k >= floor) {
                const int at = atomicAdd(&s.count, 1);
                if (at < kRoom) s.found[at] = k;
            }
        });
    }
    __syncthreads();
    const int count = s.count;
    if (count <= kRoom) {
        for (int i = t; i < count; i += kThreads) {
            const Key k = s.found[i];
            int above = 0;
            for (int j = 0; j < count; ++j) above += s.found[j] > k;
            if (above < top) s.got[above] = k;
        }
    } else {   // more than there is room for: one after the other
        Key last = ~Key(0);
        for (int n = 0; n < top; ++n) {
            Key k = 0;
            each([&](Key x) { k = x < last ? max(k, x) : k; });
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) k = max(k, __shfl_xor_sync(kAll, k, d));
            if (lane == 0) s.best[t >> 5] = k;
            __syncthreads();
            for (int i = 0; i < kThreads / 32; ++i) k = max(k, s.best[i]);
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

// p (-(a + b h) - b ln p), and a at the token.
__device__ __forceinline__ float logit_grad(float z, float c, const RowGrad& g, float a1, float b1) {
    const float x = max_nan(fmaf(z - g.m, c, -g.ln2s), kNone);
    return exp2_fast(x) * fmaf(x, b1, a1);
}

// dz of the row's chunks of eight from `first` on, `stride` apart.  Chunks start on
// 16-byte boundaries of dz; logits that do not start with them are read as the
// words that hold them.
__device__ void row_gradient(const TokenLogprobs& a, int64_t row, const RowGrad& g, int64_t first, int64_t stride) {
    const float c = a.scale * kLog2e;
    const bool half = a.dz.dtype == FSDP_DTYPE_BF16;
    const uintptr_t to = reinterpret_cast<uintptr_t>(a.dz.p) + static_cast<uintptr_t>(row * a.dz.ld) * (half ? 2 : 4);
    const int lead = half ? static_cast<int>(to & 15) / 2 : static_cast<int>(to & 15) / 4;
    const int64_t chunks = (lead + a.vocab + 7) / 8;
    const int64_t zrow = row * a.z.ld, drow = row * a.dz.ld;
    const int esz = a.z.dtype == FSDP_DTYPE_BF16 ? 2 : 4;
    const bool direct = ((reinterpret_cast<uintptr_t>(a.z.p) + static_cast<uintptr_t>((zrow - lead) * esz)) & 15) == 0;
    const float b1 = -g.b * kLn2, a1 = -fmaf(g.b, g.h, g.a);
    for (int64_t q = first; q < chunks; q += stride) {
        const int64_t c0 = q * 8 - lead;
        if (c0 >= 0 && c0 + 8 <= a.vocab) {
            float v[8];
            if (g.zero) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            } else {
                if (direct) {
                    load8(a.z.p, a.z.dtype, zrow + c0, v);
                } else {
                    const int n = 8;
                    load_chunks_any<1>(a.z.p, a.z.dtype, zrow + c0, &n, 0, &v);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = logit_grad(v[j], c, g, a1, b1);
                if (g.token >= c0 && g.token < c0 + 8) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (g.token == c0 + j) v[j] += g.a;
                }
            }
            store8(a.dz.p, a.dz.dtype, drow + c0, v);
        } else {
            for (int64_t i = max(c0, int64_t(0)); i < min(c0 + 8, a.vocab); ++i) {
                float v = 0.0f;
                if (!g.zero) {
                    v = logit_grad(load1(a.z.p, a.z.dtype, zrow + i), c, g, a1, b1);
                    if (g.token == i) v += g.a;
                }
                store1(a.dz.p, a.dz.dtype, drow + i, v);
            }
        }
    }
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

// A row to a block.
template <bool BF16, bool GRAD>
__global__ void __launch_bounds__(kThreads, 2) token_logprobs_kernel(const TokenLogprobs a) {
    constexpr int E = RowWords<BF16>::E;
    __shared__ TopShared tops;
    __shared__ Soft softs[kThreads / 32];
    starts_early();
    after_previous();
    const int t = threadIdx.x, lane = t & 31;
    const float c = a.scale * kLog2e;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowWords<BF16> r(a.z, row, a.vocab);
        Soft s{-kInf, 0.0f, 0.0f};
        int64_t best = t;   // the first word of the group that holds the largest logit
        for (int64_t w = t; w < r.count; w += kWords * kThreads) {
            float z[kWords][E];
            uint4 v[kWords];
#pragma unroll
            for (int k = 0; k < kWords; ++k) v[k] = r.load(w + k * kThreads, r.count);
            float top = -kInf;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                r.floats(v[k], w + k * kThreads, z[k]);
#pragma unroll
                for (int j = 0; j < E; ++j) top = fmaxf(top, z[k][j]);
            }
            if (top > s.m) {
                rescale(s, top, c);
                best = w;
            }
            const float ref = s.m == -kInf ? 0.0f : s.m;
#pragma unroll
            for (int k = 0; k < kWords; ++k)
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float d = max_nan((z[k][j] - ref) * c, kNone), e = exp2_fast(d);
                    s.S += e;
                    s.Q = fmaf(e, d, s.Q);
                }
        }
        // the thread's largest logit's key: the first of its group that equals it
        Key mine = 0;
        if (a.top > 0) {
            for (int k = 0; k < kWords; ++k) {
                const int64_t w = best + k * kThreads;
                if (w >= r.count) break;
                float z[E];
                r.floats(r.words[w], w, z);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const int64_t i = w * E - r.lead + j;
                    if (mine == 0 && i >= 0 && i < r.cols && z[j] == s.m) mine = key_of(z[j], i);
                }
            }
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            s = join(s, Soft{__shfl_xor_sync(kAll, s.m, d), __shfl_xor_sync(kAll, s.S, d), __shfl_xor_sync(kAll, s.Q, d)}, c);
        if (lane == 0) softs[t >> 5] = s;
        __syncthreads();
        s = softs[0];
        for (int i = 1; i < kThreads / 32; ++i) s = join(s, softs[i], c);
        const bool bad = !(s.S == s.S);
        const float ln_s = logf(s.S);
        const float h = s.S == 0.0f ? 0.0f : fmaf(-kLn2, s.Q / s.S, ln_s);
        if (t == 0) {
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
            if (a.entropy != nullptr) a.entropy[row] = h;
            if (a.stats != nullptr) {
                a.stats[2 * row] = s.m;
                a.stats[2 * row + 1] = ln_s;
            }
        }
        if (a.top > 0) {
            if (!bad) top_keys<BF16>(r, 0, r.count, a.top, mine, tops);
            if (t < a.top) {
                const Key k = bad ? 0 : tops.got[t];
                a.top_tokens[row * a.top + t] = bad ? -1 : static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(k));
                a.top_logprobs[row * a.top + t] = bad ? __uint_as_float(0x7fc00000u)
                                                      : s.S == 0.0f ? -kInf : fmaf(unorder(static_cast<uint32_t>(k >> 32)) - s.m, a.scale, -ln_s);
            }
        }
        __syncthreads();   // the token's logit is read before the gradient may take its place
        if constexpr (GRAD) row_gradient(a, row, row_grad(a, row, s.m, ln_s, h), t, kThreads);
    }
}

__global__ void __launch_bounds__(kThreads, 2) token_logprobs_backward_kernel(const TokenLogprobs a) {
    starts_early();
    after_previous();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float m = a.stats[2 * row], ln_s = a.stats[2 * row + 1];
        const RowGrad g = row_grad(a, row, m, ln_s, a.entropy != nullptr ? a.entropy[row] : 0.0f);
        if (threadIdx.x == 0 && g.token >= a.vocab) atomicOr(a.status, FSDP_KSTATUS_BAD_TOKEN);
        row_gradient(a, row, g, threadIdx.x, kThreads);
    }
}

unsigned blocks_for(int64_t rows) { return static_cast<unsigned>(std::min<int64_t>(rows, int64_t(1) << 30)); }

}  // namespace

cudaError_t launch_token_logprobs(const TokenLogprobs& a, int, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const bool half = a.z.dtype == FSDP_DTYPE_BF16, grad = a.dz.p != nullptr;
    const auto kernel = half ? (grad ? token_logprobs_kernel<true, true> : token_logprobs_kernel<true, false>)
                             : (grad ? token_logprobs_kernel<false, true> : token_logprobs_kernel<false, false>);
    return launch_early(kernel, dim3(blocks_for(a.rows)), kThreads, 0, st, a);
}

cudaError_t launch_token_logprobs_backward(const TokenLogprobs& a, int, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    return launch_early(token_logprobs_backward_kernel, dim3(blocks_for(a.rows)), kThreads, 0, st, a);
}

}  // namespace fsdp
