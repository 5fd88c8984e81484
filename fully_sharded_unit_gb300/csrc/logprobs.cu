// Log probabilities of given tokens, their entropy and most likely alternatives, and
// the logits' gradient.
#include <algorithm>
#include <cmath>

#include "block_device.cuh"
#include "compute.hpp"
#include "rows.cuh"

namespace fsdp {
namespace {

constexpr int kThreads = 128;         // of a block; each of them costs a row some work of its own
constexpr int kWords = 8;            // 16-byte words of a thread in a group
constexpr int kPlaces = 2;           // groups of a thread in shared memory
constexpr int kBlocks = 5;           // on an SM
constexpr int kRingBytes = kPlaces * kWords * kThreads * 16;
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
    // Word w, whose bits are v, without what is not the row's.
    __device__ uint4 masked(uint4 v, int w) const {
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
        return w > 0 && w < count - 1 ? words[w] : masked(words[w], w);
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

// The running maximum m of some logits, S = sum of 2^d and Q = sum of 2^d d over them, where
// d = z c - mc, c = scale log2(e) and mc = m c as fp32 has it: one rounding a term, and
// what mc is off by is the same for all of a row's terms and is put right in ln S at the end.
// Where that could be more than a sixteenth (|mc| from 2^20), and for c beyond what logits
// ask for, d is (z - m) c instead.
struct Soft {
    float m, S, Q;
};

__device__ __forceinline__ bool plain(float m, float c) { return fabsf(m * c) < 0x1p20f && c > 0x1p-79f && c < 0x1p20f; }

// By how much a term's d under the maximum m is below (z - m) c: what mc is off by, or nothing.
__device__ __forceinline__ float anchor_gap(float m, float c) { return plain(m, c) ? fmaf(-m, c, __fmul_rn(m, c)) : 0.0f; }

// d of the old maximum under the new one; at kNone what is behind it vanishes.  The two may stand on either
// side of plain()'s limits, where one maximum's terms carry a gap and the other's do not.
__device__ __forceinline__ float grown(float from, float to, float c) {
    if (plain(from, c) && plain(to, c)) return fmaxf(__fmul_rn(from, c) - __fmul_rn(to, c), kNone);
    return fmaxf((from - to) * c + (anchor_gap(from, c) - anchor_gap(to, c)), kNone);
}

__device__ __forceinline__ void rescale(Soft& s, float to, float c) {
    if (s.m != -kInf) {   // else the sums are 0, or NaN
        const float d = grown(s.m, to, c), f = exp2_fast(d);
        s.Q = f * fmaf(d, s.S, s.Q);
        s.S *= f;
    }
    s.m = to;
}

// Joined over a warp's lanes, for each of them: all brought to the largest maximum, then added.
__device__ __forceinline__ Soft join_lanes(Soft s, float c) {
    float m = s.m;
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
    rescale(s, m, c);
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        s.S += __shfl_xor_sync(kAll, s.S, d);
        s.Q += __shfl_xor_sync(kAll, s.Q, d);
    }
    return s;
}

// Adds N words' elements to s, whose m is at least as large as they are.  Q's terms must not have
// d = -inf: a bf16 logit is held at -2^100 first, two at a time, which is as good as masked
// where d is a plain one (below -2^20); otherwise d itself is held.
template <bool BF16, bool ENTROPY, bool PLAIN, int N>
__device__ __forceinline__ void add_words(Soft& s, const uint4* words, float c) {
    constexpr int E = RowWords<BF16>::E;
    const f32x2 c2 = pair(c, c);
    const float m = s.m == -kInf ? 0.0f : s.m;   // nothing but masked logits so far
    const float mc = __fmul_rn(m, c);
    const f32x2 less = PLAIN ? pair(-mc, -mc) : pair(-m, -m);
    f32x2 S2 = pair(s.S, 0.0f), Q2 = pair(s.Q, 0.0f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint4 v = words[k];
        float z[8];
        if (BF16 && ENTROPY && PLAIN) {
            constexpr uint32_t kFloor = 0xf180f180u;   // -2^100
            v = make_uint4(max_nan_bf16x2(v.x, kFloor), max_nan_bf16x2(v.y, kFloor), max_nan_bf16x2(v.z, kFloor), max_nan_bf16x2(v.w, kFloor));
        }
        RowWords<BF16>::floats(v, z);
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            f32x2 d = pair(z[j], z[j + 1]);
            d = PLAIN ? fma2(d, c2, less) : mul2(add2(d, less), c2);
            float d0, d1;
            unpair(d, d0, d1);
            if (ENTROPY && !(BF16 && PLAIN)) {
                d0 = max_nan(d0, kNone);
                d1 = max_nan(d1, kNone);
            }
            const f32x2 e = pair(exp2_fast(d0), exp2_fast(d1));
            S2 = add2(S2, e);
            if (ENTROPY) Q2 = fma2(e, pair(d0, d1), Q2);
        }
    }
    float x, y;
    unpair(S2, x, y);
    s.S = x + y;
    unpair(Q2, x, y);
    s.Q = x + y;
}

// The same with s.m brought up to them.
template <bool BF16, bool ENTROPY, int N>
__device__ __forceinline__ void take_words(Soft& s, const uint4* words, float c) {
    const float top = largest<BF16, N>(words);
    if (top > s.m) rescale(s, top, c);
    if (plain(s.m, c)) add_words<BF16, ENTROPY, true, N>(s, words, c);
    else add_words<BF16, ENTROPY, false, N>(s, words, c);
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

constexpr int kLists = 32;      // of neighbouring threads' logits: a lane's each when the floor is found
constexpr int kRoom = 1024;     // candidates

struct TopShared {
    uint32_t lists[kLists];     // order() of their largest logits
    uint8_t who[kThreads];      // threads that hold candidates
    Key found[kRoom];
    Key got[kMostTop];
    int asked, count;
};
static_assert(kThreads % kLists == 0 && kThreads <= 256);

// Before the block's next barrier: the lists' maxima.  `mine`: order() of the thread's largest
// logit, 0 if it has none.
__device__ __forceinline__ void top_lists(uint32_t mine, TopShared& s) {
    constexpr int width = kThreads / kLists;
#pragma unroll
    for (int d = 1; d < width; d <<= 1) mine = max(mine, __shfl_xor_sync(kAll, mine, d));
    if (threadIdx.x % width == 0) s.lists[threadIdx.x / width] = mine;
    if (threadIdx.x < kMostTop) s.got[threadIdx.x] = 0;
    if (threadIdx.x == 0) s.asked = s.count = 0;
}

// Puts the `top` largest of `count` keys into `to`, in order.
__device__ __forceinline__ void rank_keys(const Key* keys, int count, int top, Key* to) {
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const Key k = keys[i];
        int above = 0;
        for (int j = 0; j < count; ++j) above += keys[j] > k;
        if (above < top && k != 0) to[above] = k;
    }
}

// Behind that barrier: the `top` largest keys of the words [first, end), in order, into s.got (0
// where the words hold fewer).  Every one of them is at least the top-th largest of the lists'
// maxima, and the words of the few threads whose own largest logit reaches that are read again,
// by the whole block.
template <bool BF16>
__device__ void top_keys(const RowWords<BF16>& r, int first, int end, int top, uint32_t mine, TopShared& s) {
    constexpr int E = RowWords<BF16>::E;
    const int t = threadIdx.x, lane = t & 31;
    const uint32_t list = s.lists[lane];
    int above = 0;
#pragma unroll
    for (int i = 0; i < kLists; ++i) above += __shfl_sync(kAll, list, i) > list;
    const bool enough = __popc(__ballot_sync(kAll, list != 0)) >= top;
    const uint32_t floor = enough ? __reduce_min_sync(kAll, above < top ? list : 0xffffffffu) : 1u;
    if (mine >= floor) s.who[atomicAdd(&s.asked, 1)] = static_cast<uint8_t>(t);
    __syncthreads();
    const unsigned each = static_cast<unsigned>((end - first + kThreads - 1) / kThreads), items = each * static_cast<unsigned>(s.asked);
    const float least = unorder(floor);
    for (unsigned i = t; i < items; i += kThreads) {
        const int w = first + s.who[i / each] + static_cast<int>(i % each) * kThreads;
        if (w >= end) continue;
        const uint4 v = r.load(w);
        if (largest<BF16, 1>(&v) < least) continue;   // (not so where the floor is no number)
        float z[8];
        RowWords<BF16>::floats(v, z);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if (order(z[j]) >= floor && r.inside(r.column(w, j))) {
                const int at = atomicAdd(&s.count, 1);
                if (at < kRoom) s.found[at] = key_of(z[j], r.column(w, j));
            }
        }
    }
    __syncthreads();
    const int count = s.count;
    if (count <= kRoom) {
        rank_keys(s.found, count, top, s.got);
    } else {   // more than there is room for (many equal logits): one after the other
        Key last = ~Key(0);
        for (int n = 0; n < top; ++n) {
            Key k = 0;
            for (int w = first + t; w < end; w += kThreads) {
                float z[8];
                RowWords<BF16>::floats(r.load(w), z);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const Key x = key_of(z[j], r.column(w, j));
                    if (r.inside(r.column(w, j)) && x < last) k = max(k, x);
                }
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) k = max(k, __shfl_xor_sync(kAll, k, d));
            if (lane == 0) s.found[t >> 5] = k;
            __syncthreads();
            for (int i = 0; i < kThreads / 32; ++i) k = max(k, s.found[i]);
            last = k;
            if (t == 0) s.got[n] = k;
            __syncthreads();
        }
    }
    __syncthreads();
}

// ---- gradient ----

// dz = 2^d (A + B d), and a at the token; d as above.  With p = 2^d / S and ln p = d ln 2 - ln S, these
// are A = -(a + b (h - ln S)) / S and B = -b ln 2 / S.
struct RowGrad {
    float a, A, B;
    float m, mc;
    int64_t token;    // -1: none
    bool zero;        // the whole row
};

template <int N, bool ENTROPY, bool PLAIN>
__device__ __forceinline__ void logit_grads(float* v, float c, const RowGrad& g) {
    const f32x2 c2 = pair(c, c), less = PLAIN ? pair(-g.mc, -g.mc) : pair(-g.m, -g.m), A2 = pair(g.A, g.A), B2 = pair(g.B, g.B);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        f32x2 d = pair(v[j], v[j + 1]);
        d = PLAIN ? fma2(d, c2, less) : mul2(add2(d, less), c2);
        float d0, d1;
        unpair(d, d0, d1);
        if (ENTROPY) {
            d0 = max_nan(d0, kNone);
            d1 = max_nan(d1, kNone);
        }
        const f32x2 e = pair(exp2_fast(d0), exp2_fast(d1));
        unpair(mul2(e, ENTROPY ? fma2(pair(d0, d1), B2, A2) : A2), v[j], v[j + 1]);
    }
}
template <int N = 8>
__device__ __forceinline__ void logit_grads(float* v, float c, const RowGrad& g) {
    if (!plain(g.m, c)) logit_grads<N, true, false>(v, c, g);
    else if (g.B != 0.0f) logit_grads<N, true, true>(v, c, g);
    else logit_grads<N, false, true>(v, c, g);
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
    const int lead = grad_lead(a, row), vocab = static_cast<int>(a.vocab), t = threadIdx.x;
    constexpr int threads = kThreads;
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

// What the caller gives for a row, and the gradient's constants made of it: ln S and 1 / S are those of this d.
struct RowGiven {
    int64_t token;
    float a, b;
    __device__ RowGiven(const TokenLogprobs& x, int64_t row)
        : token(x.tokens != nullptr ? x.tokens[row] : -1), a(x.dlogprob != nullptr ? x.dlogprob[row] : 0.0f),
          b(x.dentropy != nullptr ? x.dentropy[row] : 0.0f) {}
};
__device__ __forceinline__ RowGrad row_grad(const TokenLogprobs& x, const RowGiven& given, float m, float ln, float inv, float h) {
    RowGrad g;
    const float c = x.scale * kLog2e, b = given.b * x.scale;
    g.token = x.dlogprob != nullptr ? given.token : -1;
    g.a = g.token >= 0 ? given.a * x.scale : 0.0f;
    // a masked row's S is 0; a token that does not exist leaves nothing to say
    g.zero = (g.a == 0.0f && b == 0.0f) || ln == -kInf;
    if (given.token >= x.vocab) {   // with the entropy's gradient alone too
        g.a = __uint_as_float(0x7fc00000u);
        g.zero = false;
    }
    g.m = m;
    g.mc = __fmul_rn(m, c);
    g.A = -inv * (b != 0.0f ? fmaf(b, h - ln, g.a) : g.a);
    g.B = -inv * b * kLn2;
    return g;
}

// ---- kernels ----

// A block's share of a row's words: all of them, or a run of them in a cluster of blocks, of
// which there are a power of two (a division here, for every thread and row, took a tenth of
// the forward pass's instructions and a fifth of the loss's).
struct Share {
    int first, end;
    __device__ Share(int count, int rank, int cluster) {
        const int shift = 31 - __clz(cluster);
        first = static_cast<int>((static_cast<int64_t>(count) * rank) >> shift);
        end = static_cast<int>((static_cast<int64_t>(count) * (rank + 1)) >> shift);
    }
};

// The threads' sums joined over a block's WARPS warps, and over the cluster: for every thread.
template <int WARPS>
__device__ __forceinline__ Soft join_all(Soft s, float c, Soft* softs, Soft* joined, int rank, int cluster) {
    const int t = threadIdx.x, lane = t & 31;
    const Soft none{-kInf, 0.0f, 0.0f};
    s = join_lanes(s, c);
    if (lane == 0) softs[t >> 5] = s;
    __syncthreads();
    s = join_lanes(lane < WARPS ? softs[lane] : none, c);
    if (cluster > 1) {
        if (t < cluster) {
            const uint32_t to = remote_addr(shared_at(&joined[rank]), t);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(s.m) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(s.S) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(s.Q) : "memory");
        }
        cluster_meet();
        s = join_lanes(lane < cluster ? joined[lane] : none, c);
    }
    return s;
}

// A row's results, by one thread.  z: the token's logit.
template <bool ENTROPY>
__device__ __forceinline__ void row_results(const TokenLogprobs& a, int64_t row, const Soft& s, float ln_s, float h, int64_t token, float z) {
    if (a.tokens != nullptr) {
        float lp = 0.0f;
        if (token >= a.vocab) {
            lp = __uint_as_float(0x7fc00000u);
            atomicOr(a.status, FSDP_KSTATUS_BAD_TOKEN);
        } else if (token >= 0) {
            lp = s.S == 0.0f ? -kInf : fmaf(z - s.m, a.scale, -ln_s);
        }
        a.logprob[row] = lp;
    }
    if (ENTROPY && a.entropy != nullptr) a.entropy[row] = h;
    if (a.stats != nullptr) {
        a.stats[2 * row] = s.m;
        a.stats[2 * row + 1] = ln_s;
    }
}

__device__ __forceinline__ float token_logit(const TokenLogprobs& a, int64_t row, int64_t token) {
    return token >= 0 && token < a.vocab ? load1(a.z.p, a.z.dtype, row * a.z.ld + token) : 0.0f;
}

// Rows to blocks, or to clusters of blocks.  A thread copies the words that it will look at itself,
// in groups and row after row, into its own places in shared memory (cp.async), so
// that while the block joins a row's sums and looks for its alternatives the next row's
// words are under way.  8192 x 50257 bf16: 134 us, 6.1 TB/s; with entropy 137; with entropy and five
// alternatives 176, 4.7 TB/s.  2048 x 50257 fp32: 76 us, 5.4 TB/s, and 92.  What the alternatives
// add is steps that a block takes together, with five blocks to an SM: neither DRAM (55 % by the counters) nor the issue
// slots (10 instructions a logit, 2.4 of 4 a cycle) are at their limit.  (A row to 256 threads, whose
// joint work weighs more, 286 us before that was cut down; words ahead in registers, 229.)
template <bool BF16, bool ENTROPY, bool GRAD>
__global__ void __launch_bounds__(kThreads, kBlocks) token_logprobs_kernel(const __grid_constant__ TokenLogprobs a, int cluster) {
    constexpr int threads = kThreads;
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ TopShared tops;
    __shared__ Soft softs[kThreads / 32], joined[kMostCluster];
    starts_early();
    after_previous();
    if (cluster > 1) cluster_sync();   // the others' shared memory is there
    const int t = threadIdx.x;
    const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const float c = a.scale * kLog2e;
    const int64_t stride = gridDim.x / cluster;
    const uint32_t slots = shared_at(ring + t);
    // the group to copy next: its row, that row's words, its first word and the share's end
    int64_t ahead = blockIdx.x / cluster;
    const uint4* words = nullptr;
    int w_ahead = 0, end_ahead = 0;
    const auto look_ahead = [&] {   // to a row of which the thread has words
        for (; ahead < a.rows; ahead += stride) {
            const RowWords<BF16> r(a.z, ahead, a.vocab);
            const Share share(r.count, rank, cluster);
            words = r.words;
            w_ahead = share.first + t;
            end_ahead = share.end;
            if (w_ahead < end_ahead) return;
        }
    };
    const auto copy_ahead = [&](int place) {
        if (ahead < a.rows) {
#pragma unroll
            for (int k = 0; k < kWords; ++k)
                if (w_ahead + k * threads < end_ahead)
                    copy16(slots + (place * kWords + k) * threads * 16, words + w_ahead + k * threads);
            w_ahead += kWords * threads;
            if (w_ahead >= end_ahead) {
                ahead += stride;
                look_ahead();
            }
        }
        copies_end();
    };
    look_ahead();
    for (int i = 0; i < kPlaces; ++i) copy_ahead(i);
    int place = 0;
    for (int64_t row = blockIdx.x / cluster; row < a.rows; row += stride) {
        const RowWords<BF16> r(a.z, row, a.vocab);
        const Share share(r.count, rank, cluster);
        const int first = share.first, end = share.end;
        const int64_t token = t == 0 && a.tokens != nullptr ? a.tokens[row] : -1;
        const float z_token = token_logit(a, row, token);
        Soft s{-kInf, 0.0f, 0.0f};
        for (int w = first + t; w < end; w += kWords * threads) {
            copies_wait(kPlaces - 1);
            uint4 v[kWords];
#pragma unroll
            for (int k = 0; k < kWords; ++k) v[k] = ring[(place * kWords + k) * threads + t];
            if (w == 0 || w + (kWords - 1) * threads >= min(end, r.count - 1)) {   // a row's ends
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    const int i = w + k * threads;
                    if (i >= end) v[k] = r.none();
                    else if (i == 0 || i == r.count - 1) v[k] = r.masked(v[k], i);
                }
            }
            take_words<BF16, ENTROPY, kWords>(s, v, c);
            copy_ahead(place);   // the words are in registers
            place = place + 1 == kPlaces ? 0 : place + 1;
        }
        const uint32_t mine = first + t < end ? order(s.m) : 0;
        if (a.top > 0) top_lists(mine, tops);
        s = join_all<kThreads / 32>(s, c, softs, joined, rank, cluster);
        const bool bad = !(s.S == s.S);
        const float ln = logf(s.S), ln_s = ln + kLn2 * anchor_gap(s.m, c);
        const float h = s.S == 0.0f ? 0.0f : fmaf(-kLn2, s.Q / s.S, ln);
        if (t == 0 && rank == 0) row_results<ENTROPY>(a, row, s, ln_s, h, token, z_token);
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
            const Share part(chunks, rank, cluster);
            row_gradient<BF16>(a, row, row_grad(a, RowGiven(a, row), s.m, ln, 1.0f / s.S, h), part.first, part.end);
        }
    }
}

// Forward and backward with the row's words held in shared memory in between: kMostSlots words
// to a thread, copied by itself.  Where a word has given its gradient, the next row's
// takes its place, so a block's loads run on under its second pass.  dz lies on its words as z does.
// 8192 x 50257 bf16: 299 us, 5.5 TB/s of reads and writes (the second pass from L2: 458), with entropy 330; the SMs
// issue 2.7 of 4 a cycle.  2048 x 50257 fp32 (1024 threads, one block on an SM) 164 us, 2048 x 128256 bf16 (two such
// blocks to a row) 246.  Where dz does not lie on its words as z does, token_logprobs_kernel gives the gradient too, from
// L2: 2048 x 50257 bf16 to fp32 215 us, fp32 to bf16 244, bf16 off by an element 186.
constexpr int kMostSlots = 13;      // of 512 threads: 104 KB, two blocks on an SM

template <bool BF16, bool ENTROPY, int T>
__global__ void __launch_bounds__(T, 1024 / T) token_loss_kernel(const __grid_constant__ TokenLogprobs a, int cluster, int slots) {
    constexpr int E = RowWords<BF16>::E, G = 4;   // words of a group
    extern __shared__ __align__(16) uint4 held[];
    __shared__ Soft softs[2][T / 32], joined[2][kMostCluster];   // used in turn: there is one barrier a row
    starts_early();
    after_previous();
    if (cluster > 1) cluster_sync();   // the others' shared memory is there
    const int t = threadIdx.x;
    const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const float c = a.scale * kLog2e;
    const int64_t stride = gridDim.x / cluster;
    const uint32_t mine = shared_at(held + t);
    int64_t row = blockIdx.x / cluster;
    if (row < a.rows) {
        const RowWords<BF16> r(a.z, row, a.vocab);
        const Share share(r.count, rank, cluster);
        for (int k = 0; k < slots; ++k)
            if (share.first + t + k * T < share.end) copy16(mine + k * T * 16, r.words + share.first + t + k * T);
        copies_end();
    }
    int flip = 0;
    for (; row < a.rows; row += stride) {
        const RowWords<BF16> r(a.z, row, a.vocab);
        const Share share(r.count, rank, cluster);
        const RowGiven given(a, row);
        const float z_token = t == 0 && rank == 0 ? token_logit(a, row, given.token) : 0.0f;
        copies_wait(0);
        Soft s{-kInf, 0.0f, 0.0f};
        for (int k0 = 0; share.first + t + k0 * T < share.end; k0 += G) {
            uint4 v[G];
            const int w = share.first + t + k0 * T;
#pragma unroll
            for (int k = 0; k < G; ++k) v[k] = k0 + k < slots ? held[(k0 + k) * T + t] : r.none();
            if (w == 0 || w + (G - 1) * T >= min(share.end, r.count - 1)) {   // a row's ends
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    const int i = w + k * T;
                    if (i >= share.end) v[k] = r.none();
                    else if (i == 0 || i == r.count - 1) v[k] = r.masked(v[k], i);
                }
            }
            take_words<BF16, ENTROPY, G>(s, v, c);
        }
        s = join_all<T / 32>(s, c, softs[flip], joined[flip], rank, cluster);
        flip ^= 1;
        const float ln = logf(s.S), ln_s = ln + kLn2 * anchor_gap(s.m, c);
        const float h = s.S == 0.0f ? 0.0f : fmaf(-kLn2, s.Q / s.S, ln);
        if (t == 0 && rank == 0) row_results<ENTROPY>(a, row, s, ln_s, h, given.token, z_token);
        const RowGrad g = row_grad(a, given, s.m, ln, 1.0f / s.S, h);
        const int hit = !g.zero && g.token >= 0 && g.token < a.vocab ? (static_cast<int>(g.token) + r.lead) / E : -1;   // the token's word
        uint4* out = reinterpret_cast<uint4*>((reinterpret_cast<uintptr_t>(a.dz.p) + static_cast<uintptr_t>(row * a.dz.ld) * (16 / E)) & ~uintptr_t(15));
        const bool more = row + stride < a.rows;
        const RowWords<BF16> next(a.z, more ? row + stride : row, a.vocab);
        const Share ahead(next.count, rank, cluster);
        const uint4* from = next.words + ahead.first + t;
        const int left = more ? ahead.end - ahead.first - t : 0;   // of the next row's words, from this thread's first
        const auto second_pass = [&](auto grads) {
#pragma unroll 2
            for (int k = 0; k < slots; ++k) {
                const int w = share.first + t + k * T;
                if (w < share.end) {
                    float v[8];
                    RowWords<BF16>::floats(held[k * T + t], v);
                    grads(v);
                    if (w == hit) {
#pragma unroll
                        for (int j = 0; j < E; ++j)
                            if (r.column(w, j) == static_cast<int>(g.token)) v[j] += g.a;
                    }
                    if (static_cast<unsigned>(w - 1) < static_cast<unsigned>(r.count - 2)) {
                        out[w] = BF16 ? make_uint4(to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]), to_bf16x2(v[E - 4], v[E - 3]), to_bf16x2(v[E - 2], v[E - 1]))
                                      : make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
                    } else {   // a row's ends
#pragma unroll
                        for (int j = 0; j < E; ++j)
                            if (r.inside(r.column(w, j))) store1(a.dz.p, a.dz.dtype, row * a.dz.ld + r.column(w, j), v[j]);
                    }
                }
                if (k * T < left) copy16(mine + k * T * 16, from + k * T);
            }
        };
        if (!g.zero && plain(g.m, c)) second_pass([&](float* v) { logit_grads<E, ENTROPY, true>(v, c, g); });
        else second_pass([&](float* v) {
            logit_grads<E, true, false>(v, c, g);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = g.zero ? 0.0f : v[j];
        });
        copies_end();
    }
}

// `parts` blocks to a row, which have a run of its chunks each.  One read, one write and an
// exponential a logit: 2048 x 50257 fp32 126 us, 6.5 TB/s; 8192 x 50257 bf16 250, 6.6 TB/s.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) token_logprobs_backward_kernel(const TokenLogprobs a, int parts) {
    starts_early();
    after_previous();
    const int part = blockIdx.x % parts;
    for (int64_t row = blockIdx.x / parts; row < a.rows; row += gridDim.x / parts) {
        const float m = a.stats[2 * row], ln_s = a.stats[2 * row + 1];
        const float c = a.scale * kLog2e, ln = ln_s - kLn2 * anchor_gap(m, c);
        const RowGrad g = row_grad(a, RowGiven(a, row), m, ln, expf(-ln), a.entropy != nullptr ? a.entropy[row] : 0.0f);
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
    // blocks to a row: as many as fill the SMs, but two words at least to a thread
    const int64_t words = a.vocab * (half ? 2 : 4) / 16 + 2;   // and where a row begins inside one
    // dz on its words as z is on its own, row by row
    const int64_t size = half ? 2 : 4;
    if (grad && a.dz.dtype == a.z.dtype && (((reinterpret_cast<uintptr_t>(a.z.p) ^ reinterpret_cast<uintptr_t>(a.dz.p)) | static_cast<uintptr_t>((a.z.ld - a.dz.ld) * size)) & 15) == 0) {
        // blocks to a row: what holds it in shared memory, and as many as fill the SMs
        int parts = 1;
        while (parts < kMostCluster && (words > static_cast<int64_t>(parts) * 1024 * kMostSlots ||
                                        (a.rows * parts * 2 <= 2 * sms && words >= static_cast<int64_t>(parts) * 2 * 512 * 2))) parts *= 2;
        const int64_t share = (words + parts - 1) / parts + 1;
        const int threads = share <= 512 * kMostSlots ? 512 : 1024;
        const int slots = static_cast<int>((share + threads - 1) / threads);
        if (slots <= kMostSlots) {
            const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(a.rows, std::max(1, sms * (1024 / threads) / parts)) * parts);
#define RUN(h, e, t) return launch_shared_clusters<token_loss_kernel<h, e, t>>(blocks, threads, slots * threads * 16, parts, st, a, parts, slots)
#define RUN_(h, e) do { if (threads == 512) RUN(h, e, 512); RUN(h, e, 1024); } while (0)
            if (half && entropy) RUN_(true, true);
            if (half) RUN_(true, false);
            if (entropy) RUN_(false, true);
            RUN_(false, false);
#undef RUN_
#undef RUN
        }
    }
    const int64_t most = static_cast<int64_t>(sms) * kBlocks;
    int cluster = 1;
    while (cluster < kMostCluster && a.rows * cluster * 2 <= most && words >= static_cast<int64_t>(cluster) * 2 * kThreads * 2) cluster *= 2;
    const int64_t rows = std::min(a.rows, std::max<int64_t>(1, most / cluster));
#define RUN(h, e, g) return launch_shared_clusters<token_logprobs_kernel<h, e, g>, kRingBytes>(static_cast<unsigned>(rows * cluster), kThreads, kRingBytes, cluster, st, a, cluster)
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
    const int64_t most = a.vocab / (8 * 4 * kThreads) + 1;
    const int64_t parts = std::max<int64_t>(1, std::min(most, static_cast<int64_t>(sms) * 8 / a.rows));
    const int64_t rows = std::min(a.rows, (int64_t(1) << 30) / parts);
    return launch_early(a.z.dtype == FSDP_DTYPE_BF16 ? token_logprobs_backward_kernel<true> : token_logprobs_backward_kernel<false>,
                        dim3(static_cast<unsigned>(rows * parts)), kThreads, 0, st, a, static_cast<int>(parts));
}

}  // namespace fsdp
