// The linear layer's products, and the column sums of its bias's gradient.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "block_device.cuh"
#include "compute.hpp"
#include "epilogue.cuh"
#include "product_plan.hpp"

namespace fsdp {
namespace {

// ---- the matrix product ------------------------------------------------------
//
// C[m, n] = sum_k A(m, k) B(n, k) on the 5th-generation tensor cores.  A pair
// of CTAs (a cluster of two) computes one 256 x BN tile with
// tcgen05.mma.cta_group::2: each CTA holds 128 rows of A and BN/2 rows of B in
// shared memory, and 128 rows of the fp32 sums in its tensor memory.
//
//   warps 0 and 3  producers: TMA copies of 64-deep slices of A and of B into a
//            ring of stages (one warp for both took 250 cycles to issue a stage)
//   warp 1   issues the pair's matrix instructions (first CTA only)
//   warp 2   tensor memory allocation
//   warps 4-11  epilogue: sums to registers, then bias, activation, residual,
//            checkpoint, stores; while the next tile's products run into the
//            other half of tensor memory
//
// Either operand may be contiguous along k or along its own rows (W is read
// both ways, x and dy too): the copies take boxes of 64 elements along the
// contiguous direction, and only the shared-memory descriptors differ.
//
// What bounds it: the tensor cores where k and the tiles are many (8192 x 8192 x
// 8192 in BF16: 1980 TFLOP/s, the rate of the library's product there; for
// seconds on end, the power limit: 1740), an epilogue that takes as long as a
// tile's products where k is short (4096 x 1280 -> 5120: 32.5 us, 1650 TFLOP/s,
// plain; 49 with bias, GELU and an 8-bit checkpoint kept, whose sums are cut three
// times; 42.5 with a residual; 46 for an input gradient with GELU's slope from a
// checkpoint; by ncu its latencies, with no unit over 60 % busy), and the latency of one tile where there are few (64 x 1280 -> 5120: 7.5 us).
// Pairs of CTAs, since a pair halves B's copies; tiles as wide as tensor memory
// holds twice, since a tile's copies for a product fall with its width; one
// persistent pair to two SMs, so that an epilogue runs beside the next tile.

constexpr int kEpiWarps = 8;
constexpr int kEpiBytes = 32 * 32 * 4;           // a warp's transposing buffer
constexpr int kThreads = 384;
constexpr int kPiece = 32 * 128;                 // floats of a warp's part of a tile
constexpr int kPieces = 2 * kEpiWarps;           // parts of a tile
constexpr size_t kSmemBytes = 1024 + kRingBytes + kEpiWarps * kEpiBytes + 320;

struct Bars {
    uint64_t full[kStagesMost];      // first CTA's: both CTAs' copies of a stage, A's and B's, have landed
    uint64_t empty[kStagesMost];     // the products that read a stage are done
    uint64_t tmem_full[2];       // a tile's sums are complete
    uint64_t tmem_empty[2];      // first CTA's: both CTAs' epilogues have read them
    uint64_t drain;
    uint32_t tmem_base;
    uint32_t abort;              // a wait of this CTA ran out
    uint32_t pair_abort;         // one of the other CTA did
    uint32_t issued[2];          // stages the producers issued: of A, of B
    uint32_t consumed;           // stages the matrix instructions read
};
static_assert(sizeof(Bars) <= 320, "the barriers' room");

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

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

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive_remote(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void bar_expect_remote(uint32_t addr, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(addr), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t addr, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    return done != 0;
}

// Wait for a phase; false if it has not completed within the limit (in clock
// cycles), or if another wait of this CTA has run out already.  The clock is
// read from the 16th try on: most waits end before, and reading the global
// timer in each of them cost more than half of the products' rate.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, long long limit, const volatile uint32_t* abort) {
    const uint32_t addr = smem_addr(bar);
    long long t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (bar_try(addr, parity)) return true;
        if (i == 16) t0 = clock64();
        else if (i > 16 && (i & 15) == 0 && (*abort != 0 || clock64() - t0 > limit)) return false;
    }
}

// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool bar_wait_warp(uint32_t addr, uint32_t parity, long long limit, const volatile uint32_t* abort) {
    long long t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (__all_sync(0xffffffffu, bar_try(addr, parity))) return true;
        if (i == 16) t0 = clock64();
        else if (i > 16 && (i & 15) == 0 && __any_sync(0xffffffffu, *abort != 0 || clock64() - t0 > limit)) return false;
    }
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// One 16-deep product of the pair, d = a b (add == 0) or d += a b, issued by the
// lane where `leader` is set.  The predicate is inside the statement: the code
// around it stays that of a whole warp, and its operands uniform.
__device__ __forceinline__ void mma(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{ .reg .pred e, p; setp.ne.u32 e, %5, 0; setp.ne.u32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(leader)
        : "memory");
}

// 1 in one lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r;
}

// Arrives on the barrier at this offset in both CTAs once the matrix
// instructions issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t leader, uint32_t bar) {
    asm volatile(
        "{ .reg .pred e; setp.ne.u32 e, %2, 0;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1; }" ::"r"(bar),
        "h"(static_cast<uint16_t>(3)), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void tmem_load32(uint32_t addr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_store32(uint32_t addr, const float* v) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Shared-memory descriptor of an operand slice, 128-byte swizzled.  Contiguous
// along k: rows of 64 elements, 8-row groups 1024 bytes apart.  Contiguous
// along its rows: blocks of 64 rows x 64 k, kBlock apart, 8-k groups 1024
// bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool by_rows) {
    const uint64_t lead = by_rows ? kBlock >> 4 : 1;
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | lead << 16 | static_cast<uint64_t>(1024 >> 4) << 32 |
           uint64_t(1) << 46 | uint64_t(2) << 61;
}

struct Plan : Tiling {
    int swapped;               // the tile's rows are C's columns (few tokens)
    int vec;                   // 1: every row of the epilogue's matrices starts on a 16-byte boundary and N % 8 == 0;
                               // 2: on a 32-byte boundary and N % 16 == 0; 0: neither, or swapped
    float* partials;           // sums of the shared tiles: tile, part, piece, kPiece floats
    int32_t* status;
    long long wait_cycles;      // bound of every wait
    int withhold;

    // One warp's part of a shared tile: chunk i of it at 256 * i, 16 bytes to a lane, eight times.
    __device__ float4* sums(int64_t shared, int part, int piece) const {
        return reinterpret_cast<float4*>(partials) + ((shared * parts + part) * kPieces + piece) * static_cast<int64_t>(kPiece / 4);
    }
};

struct Unit {
    int tm, tn, k0, k1, part;
    int shared;                // index among the shared tiles, or -1
};

// Bands of 8 tiles down, walked along n: a wave of clusters shares few slices
// of A and B in L2.
__device__ __forceinline__ void place_tile(const Plan& p, uint32_t t, int* tm, int* tn) {
    const uint32_t band = 8u * p.tiles_n;
    const uint32_t b = t / band, in = t - b * band;
    const uint32_t high = min(8u, p.tiles_m - b * 8);
    *tm = static_cast<int>(b * 8 + in % high);
    *tn = static_cast<int>(in / high);
}

__device__ __forceinline__ Unit unit_of(const Plan& p, uint32_t u) {
    Unit r;
    uint32_t t = u;
    r.k0 = 0;
    r.k1 = p.ks;
    r.part = 0;
    r.shared = -1;
    if (u >= p.whole) {
        const uint32_t v = u - p.whole;
        r.shared = static_cast<int>(v / p.parts);
        r.part = static_cast<int>(v - r.shared * p.parts);
        t = p.whole + r.shared;
        r.k0 = static_cast<int>(static_cast<int64_t>(p.ks) * r.part / p.parts);
        r.k1 = static_cast<int>(static_cast<int64_t>(p.ks) * (r.part + 1) / p.parts);
    }
    place_tile(p, t, &r.tm, &r.tn);
    return r;
}

// One 32 x 32 chunk whose rows lie one to a lane: v[j] is tile row `row0 +
// lane`, tile column `col0 + j`; `bias` that of tile column `col0 + lane`.  buf:
// 4 KiB of shared memory for rows that are not aligned.
template <int VEC, bool SLOPE>
__device__ __forceinline__ void finish_chunk(const Product& p, const Plan& pl, int64_t row0, int64_t col0, float* v,
                                             float4* buf, int lane, float bias, uint32_t* byte) {
    if constexpr (VEC > 0) {
        if (col0 < p.N) finish_row<VEC == 2, SLOPE>(p, row0 + lane, col0, row0 + lane < p.M, bias, v, byte);
    } else if (!pl.swapped) {
        if (col0 < p.N && row0 < p.M) finish_rows_any<SLOPE>(p, row0, col0, lane, bias, v, buf);
    } else {
        // the lane's tile row is a column of C
        const int64_t n = row0 + lane;
        const int count = static_cast<int>(min(static_cast<int64_t>(32), p.M - col0));
        if (count <= 0 || row0 >= p.N) return;   // the same for the whole warp
        bias = p.bias != nullptr && n < p.N ? load1(p.bias, p.bias_dtype, n) : 0.0f;
        finish_column<32, SLOPE>(p, col0, count, n, bias, v, lane);
    }
}

// VEC: the alignment of the epilogue's matrices (Plan::vec).  SLOPE: the
// epilogue multiplies by an activation's slope.
template <int VEC, bool SLOPE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ Product p, const __grid_constant__ Plan pl) {
    extern __shared__ uint8_t smem_raw[];
    // the swizzle pattern repeats every 1024 bytes of the shared address; both
    // CTAs of the pair compute the same offset
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* stage_a = smem;
    uint8_t* stage_b = smem + pl.stages * kStageA;
    float4* epi = reinterpret_cast<float4*>(smem + kRingBytes);
    Bars* bars = reinterpret_cast<Bars*>(smem + kRingBytes + kEpiWarps * kEpiBytes);
    volatile uint32_t* abort = &bars->abort;
    const uint32_t stages = pl.stages;

    // through a shuffle, which makes it uniform to the compiler: so are then the
    // branches on it, and what the warps' roles compute in them
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < pl.stages; ++i) {
            bar_init(&bars->full[i], 4);
            bar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&bars->tmem_full[i], 1);
            bar_init(&bars->tmem_empty[i], 2 * kEpiWarps);
        }
        bar_init(&bars->drain, 1);
        bars->abort = bars->pair_abort = bars->issued[0] = bars->issued[1] = bars->consumed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_a) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_b) : "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars->tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    __syncthreads();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    starts_early();
    after_previous();
    // The producers' and the matrix warp's loops run in whole warps, one lane of
    // which issues: their counters and descriptors are then uniform.  What the
    // matrix warp does in a stage has to fit into the time of the stage's
    // products (512 cycles at BN = 256): in a branch of one lane, with the clock
    // or the progress written in every stage, it took 520 to 600.
    if (warp == 0 || warp == 3) {
        // ---- producers: A's, and B's ----
        const bool is_a = warp == 0;
        const CUtensorMap* map = is_a ? &map_a : &map_b;
        const bool by_rows = is_a ? p.a_trans : p.b_trans;
        const int extent = is_a ? 128 : pl.bn / 2;                     // rows of the operand in a stage, per CTA
        const bool second = by_rows && extent > 64;                    // a box holds 64 of them
        const uint32_t bytes = is_a ? kStageA : pl.stage_b;
        const uint32_t full0 = remote_addr(smem_addr(&bars->full[0]), 0), empty0 = smem_addr(&bars->empty[0]);
        const uint32_t stage0 = smem_addr(is_a ? stage_a : stage_b), stride = is_a ? kStageA : pl.stage_b;
        const uint32_t leader = elect_one();
        bool withhold = pl.withhold && blockIdx.x < 2;                 // the first stage's copies
        uint32_t q = 0, s = 0, use = 0;   // stages issued, the next one's place and how often the ring went round (parity)
        bool ok = true;
        for (uint32_t u = cluster; u < pl.units && ok; u += clusters) {
            const Unit un = unit_of(pl, u);
            const int at = (is_a ? un.tm * 256 : un.tn * pl.bn) + static_cast<int>(rank) * extent;
            for (int k = un.k0; k < un.k1; ++k) {
                if (q >= stages && !bar_wait_warp(empty0 + s * 8, use ^ 1u, pl.wait_cycles, abort)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    const uint32_t full = full0 + s * 8, dst = stage0 + s * stride;
                    bar_expect_remote(full, bytes);
                    if (!withhold) {
                        if (!by_rows) {
                            tma_load(dst, map, k * kDepth, at, full);
                        } else {
                            tma_load(dst, map, at, k * kDepth, full);
                            if (second) tma_load(dst + kBlock, map, at + 64, k * kDepth, full);
                        }
                    }
                    withhold = false;
                }
                ++q;
                if (++s == stages) {
                    s = 0;
                    use ^= 1u;
                }
            }
        }
        // the stages still being read: their commits arrive here before this CTA leaves
        for (uint32_t i = q > stages ? q - stages : 0; ok && i < q; ++i)
            ok = bar_wait_warp(empty0 + (i % stages) * 8, (i / stages) & 1u, pl.wait_cycles, abort);
        if (lane == 0) {
            bars->issued[is_a ? 0 : 1] = q;
            if (!ok) {
                atomicOr(pl.status, FSDP_KSTATUS_WAIT_TIMEOUT);
                *abort = 1;
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---- matrix instructions ----
        const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | static_cast<uint32_t>(p.a_trans) << 15 |
                               static_cast<uint32_t>(p.b_trans) << 16 | static_cast<uint32_t>(pl.bn >> 3) << 17 | 16u << 24;
        const uint32_t step_a = p.a_trans ? 2048 >> 4 : 32 >> 4, step_b = p.b_trans ? 2048 >> 4 : 32 >> 4;   // to the next 16 k
        const uint32_t next_b = pl.stage_b >> 4;
        const int last = static_cast<int>((p.K - static_cast<int64_t>(pl.ks - 1) * kDepth + 15) / 16);   // products of the last stage
        const uint64_t da0 = smem_desc(smem_addr(stage_a), p.a_trans), db0 = smem_desc(smem_addr(stage_b), p.b_trans);
        const uint32_t full0 = smem_addr(&bars->full[0]), empty0 = smem_addr(&bars->empty[0]);
        const uint32_t tmem_full0 = smem_addr(&bars->tmem_full[0]), tmem_empty0 = smem_addr(&bars->tmem_empty[0]);
        const uint32_t leader = elect_one();
        uint64_t da = da0, db = db0;
        uint32_t q = 0, s = 0, use = 0, tile = 0;
        bool ok = true;
        for (uint32_t u = cluster; u < pl.units && ok; u += clusters) {
            const Unit un = unit_of(pl, u);
            for (int first = un.k0; first < un.k1 && ok; first += pl.slice, ++tile) {
                const int end = min(un.k1, first + pl.slice);
                const uint32_t buf = tile & pl.two, turn = tile >> pl.two, d = tmem + buf * pl.buffer;
                if (turn > 0 && !bar_wait_warp(tmem_empty0 + buf * 8, (turn - 1) & 1u, pl.wait_cycles, abort)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                uint32_t add = 0;
                for (int k = first; k < end; ++k) {
                    if (!bar_wait_warp(full0 + s * 8, use, pl.wait_cycles, abort)) {
                        ok = false;
                        break;
                    }
                    if (k + 1 < pl.ks || last == 4) {
                        mma(leader, d, da, db, idesc, add);
                        mma(leader, d, da + step_a, db + step_b, idesc, 1u);
                        mma(leader, d, da + 2 * step_a, db + 2 * step_b, idesc, 1u);
                        mma(leader, d, da + 3 * step_a, db + 3 * step_b, idesc, 1u);
                    } else {
                        for (int i = 0; i < last; ++i) mma(leader, d, da + i * step_a, db + i * step_b, idesc, add | i);
                    }
                    add = 1;
                    mma_commit(leader, empty0 + s * 8);
                    ++q;
                    da += kStageA >> 4;
                    db += next_b;
                    if (++s == stages) {
                        s = 0;
                        use ^= 1u;
                        da = da0;
                        db = db0;
                    }
                }
                if (ok) mma_commit(leader, tmem_full0 + buf * 8);
            }
        }
        if (lane == 0) bars->consumed = q;
        if (!ok) {
            // give up: report, then wait for the matrix instructions in flight
            if (lane == 0) {
                atomicOr(pl.status, FSDP_KSTATUS_WAIT_TIMEOUT);
                *abort = 1;
            }
            mma_commit(leader, smem_addr(&bars->drain));
            const volatile uint32_t never = 0;
            if (!bar_wait_warp(smem_addr(&bars->drain), 0, pl.wait_cycles, &never) && lane == 0)
                atomicOr(pl.status, FSDP_KSTATUS_DRAIN_TIMEOUT);
        }
    } else if (warp >= 4) {
        // ---- epilogue ----
        const int w = warp - 4, quad = warp & 3, half = w >> 2;
        float4* buf4 = epi + w * (kEpiBytes / 16);
        // the warp's chunks of 32 columns: the first or the second half of the tile's
        const int chunks = pl.bn / 32, c0 = half ? (chunks + 1) / 2 : 0, c1 = half ? chunks : (chunks + 1) / 2;
        uint32_t tile = 0;
        for (uint32_t u = cluster; u < pl.units; u += clusters, ++tile) {
            const Unit un = unit_of(pl, u);
            const int64_t row0 = static_cast<int64_t>(un.tm) * 256 + rank * 128 + quad * 32;
            const int64_t col0 = static_cast<int64_t>(un.tn) * pl.bn;
            float bias[4] = {};   // of the warp's chunks, read before their sums are there
            if (p.bias != nullptr && !pl.swapped) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t n = col0 + (c0 + i) * 32 + lane;
                    if (i < c1 - c0 && n < p.N) bias[i] = load1(p.bias, p.bias_dtype, n);
                }
            }
            // the slices of a long sum are added up in tensor memory, but the last one
            // where there are two accumulators: where there is one, it has to be free
            // before the epilogue's long part begins, which then reads the running
            // sums.  The whole warp goes on or none of it.
            const uint32_t sliced = tmem + pl.running + (static_cast<uint32_t>(quad * 32) << 16);
            uint32_t buf = 0, src = 0;
            bool given_up = false;
            for (int first = un.k0;; first += pl.slice, ++tile) {
                buf = tile & pl.two;
                src = tmem + buf * pl.buffer + (static_cast<uint32_t>(quad * 32) << 16);
                given_up = !bar_wait_warp(smem_addr(&bars->tmem_full[buf]), (tile >> pl.two) & 1u, pl.wait_cycles, abort);
                if (given_up) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const bool last = first + pl.slice >= un.k1;
                if (last && pl.two) break;
                for (int c = c0; c < c1; ++c) {
                    float v[32];
                    tmem_load32(src + c * 32, v);
                    if (first > un.k0) {
                        float w[32];
                        tmem_load32(sliced + c * 32, w);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] += w[j];
                    }
                    tmem_store32(sliced + c * 32, v);
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive_remote(remote_addr(smem_addr(&bars->tmem_empty[buf]), 0));
                if (last) break;
            }
            if (given_up) {
                if (lane == 0) atomicOr(pl.status, FSDP_KSTATUS_WAIT_TIMEOUT);
                *abort = 1;
                break;
            }
            // a tile shared along k leaves its sums in the workspace, for finish_kernel
            float4* sums = un.shared < 0 ? nullptr : pl.sums(un.shared, un.part, static_cast<int>(rank) * kEpiWarps + w) + lane;
            const bool joins = pl.two && un.k1 - un.k0 > pl.slice;
            if (!pl.two) src = sliced;
            uint32_t bytes = 0;   // exponents of this warp's chunks of the lane's row
            for (int c = c0; c < c1; ++c) {
                float v[32];
                tmem_load32(src + c * 32, v);
                if (joins) {
                    float w[32];
                    tmem_load32(sliced + c * 32, w);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] += w[j];
                }
                if (c + 1 == c1 && pl.two) {
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) bar_arrive_remote(remote_addr(smem_addr(&bars->tmem_empty[buf]), 0));
                }
                if (sums != nullptr) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        sums[(c - c0) * 256 + s * 32] = make_float4(v[4 * s], v[4 * s + 1], v[4 * s + 2], v[4 * s + 3]);
                } else {
                    const int i = c - c0;
                    uint32_t byte = 0;
                    finish_chunk<VEC, SLOPE>(p, pl, row0, col0 + c * 32, v, buf4, lane,
                                             i == 0 ? bias[0] : i == 1 ? bias[1] : i == 2 ? bias[2] : bias[3], &byte);
                    bytes |= byte << (8 * i);
                }
            }
            if (VEC > 0 && !SLOPE && sums == nullptr && p.pre.p != nullptr && p.pre.dtype == FSDP_DTYPE_ACT8) {
                // four neighbouring bytes of eight rows at a time: one byte of 32
                // rows at a time is 32 partial sectors, which cost 6 us in 40
                const int i = lane & 3;
                const int64_t group = (col0 >> 5) + c0 + i;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = j * 8 + (lane >> 2);
                    const uint32_t w = __shfl_sync(0xffffffffu, bytes, r);
                    if (i < c1 - c0 && group < p.pre.eld && row0 + r < p.M)
                        p.pre.e[(row0 + r) * p.pre.eld + group] = static_cast<uint8_t>(w >> (8 * i));
                }
            }
            if (c0 >= c1 && pl.two && lane == 0) bar_arrive_remote(remote_addr(smem_addr(&bars->tmem_empty[buf]), 0));
        }
    }

    __syncthreads();
    if (threadIdx.x == 0 && *abort != 0)   // the pair gives up together
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote_addr(smem_addr(&bars->pair_abort), rank ^ 1u)), "r"(1) : "memory");
    // no CTA leaves while its pair may still read its shared memory or arrive on its barriers
    cluster_sync();
    if (*abort != 0 || *static_cast<volatile uint32_t*>(&bars->pair_abort) != 0) {
        if (rank == 0 && threadIdx.x == 0) {
            uint32_t issued[4] = {bars->issued[0], bars->issued[1], 0, 0}, most = 0;
            for (int i = 0; i < 2; ++i)
                asm volatile("ld.shared::cluster.u32 %0, [%1];"
                             : "=r"(issued[2 + i])
                             : "r"(remote_addr(smem_addr(&bars->issued[i]), 1))
                             : "memory");
            for (int i = 0; i < 4; ++i) most = max(most, issued[i]);
            // after a give-up: copies in flight still land before either CTA leaves.
            // A stage that only some of the four producers issued gets the others'
            // arrivals here.
            const volatile uint32_t never = 0;
            for (uint32_t q = bars->consumed; q < most; ++q) {
                const uint32_t bar = remote_addr(smem_addr(&bars->full[q % stages]), 0);
                if (pl.withhold && blockIdx.x < 2 && q == 0) continue;   // armed, but no copy was issued
                for (int i = 0; i < 4; ++i)
                    if (q >= issued[i]) bar_arrive_remote(bar);
                if (!bar_wait(&bars->full[q % stages], (q / stages) & 1u, pl.wait_cycles, &never))
                    atomicOr(pl.status, FSDP_KSTATUS_DRAIN_TIMEOUT);
            }
        }
        cluster_sync();
    }
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// Column sums of dy: V columns to a thread (8 from a 16-byte boundary, or 1),
// 32 threads across and 8 slices of rows down to a block, which joins them and
// leaves one row of sums, for sum_partials_kernel to add in order (atomics'
// order would change results).  Bound by the latency of a thread's loads, of which
// eight are in flight: 2048 x 49152 in 43 us (4.7 TB/s), 4096 x 5120 in 13 (3.2),
// 4096 x 1280 in 6.
template <int V>
__global__ void __launch_bounds__(256) column_sum_kernel(int64_t rows, int64_t cols, Mat dy, float* partials) {
    __shared__ float part[8][32 * V + 1];
    starts_early();
    after_previous();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + tx) * V;
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.0f;
    if (c < cols) {
        const int64_t step = static_cast<int64_t>(gridDim.y) * 8;
        int64_t r = static_cast<int64_t>(blockIdx.y) * 8 + ty;
        for (; r + 7 * step < rows; r += 8 * step) {
            float v[8][V];
#pragma unroll
            for (int i = 0; i < 8; ++i) loadv<V>(dy.p, FSDP_DTYPE_BF16, (r + i * step) * dy.ld + c, v[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += v[i][j];
        }
        for (; r < rows; r += step) {
            float v[V];
            loadv<V>(dy.p, FSDP_DTYPE_BF16, r * dy.ld + c, v);
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] += v[j];
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) part[ty][j * 32 + tx] = s[j];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += part[k][i];
        const int64_t col = (static_cast<int64_t>(blockIdx.x) * 32 + (i & 31)) * V + (i >> 5);
        if (col < cols) partials[static_cast<int64_t>(blockIdx.y) * cols + col] = t;
    }
}

// The shared tiles: the parts' sums, then the same epilogue.  A block finishes
// one 32 x 32 chunk: each of its warps adds up a quarter of the parts, in their
// order, and the first warp adds the four.  (Done by the last cluster to reach
// a tile instead, the sums of 19 parts took 60 us of its two SMs' time; by one
// warp a chunk, 15 us.)  Bound by the latency of the parts' sums from L2.
template <int VEC, bool SLOPE>
__global__ void __launch_bounds__(128) finish_kernel(const __grid_constant__ Product p, const __grid_constant__ Plan pl) {
    __shared__ float4 buf[4][256];
    starts_early();
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per_tile = pl.bn / 4;   // chunks of a tile: 8 x bn/32
    const uint32_t shared = blockIdx.x / per_tile;
    const int in = static_cast<int>(blockIdx.x - shared * per_tile), c = in >> 3, rank = in >> 2 & 1, quad = in & 3;
    int tm, tn;
    place_tile(pl, static_cast<uint32_t>(pl.whole) + shared, &tm, &tn);
    const int j0 = pl.parts * warp / 4, j1 = pl.parts * (warp + 1) / 4;
    const int first = (pl.bn / 32 + 1) / 2, half = c >= first ? 1 : 0;   // as the product's epilogue divides a tile
    const float4* q = pl.sums(shared, j0, rank * kEpiWarps + half * 4 + quad) + (c - half * first) * 256 + lane;
    const int64_t next = static_cast<int64_t>(kPieces) * (kPiece / 4);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
#pragma unroll 2
    for (int j = j0; j < j1; ++j, q += next) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float4 f = __ldcg(q + s * 32);
            v[4 * s] += f.x; v[4 * s + 1] += f.y; v[4 * s + 2] += f.z; v[4 * s + 3] += f.w;
        }
    }
    if (warp > 0) {
#pragma unroll
        for (int s = 0; s < 8; ++s) buf[warp][s * 32 + lane] = make_float4(v[4 * s], v[4 * s + 1], v[4 * s + 2], v[4 * s + 3]);
    }
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < 4; ++w) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float4 f = buf[w][s * 32 + lane];
            v[4 * s] += f.x; v[4 * s + 1] += f.y; v[4 * s + 2] += f.z; v[4 * s + 3] += f.w;
        }
    }
    const int64_t col0 = static_cast<int64_t>(tn) * pl.bn + c * 32;
    const int64_t row0 = static_cast<int64_t>(tm) * 256 + rank * 128 + quad * 32;
    const float bias = p.bias != nullptr && !pl.swapped && col0 + lane < p.N ? load1(p.bias, p.bias_dtype, col0 + lane) : 0.0f;
    uint32_t byte = 0;
    finish_chunk<VEC, SLOPE>(p, pl, row0, col0, v, buf[0], lane, bias, &byte);
    if (VEC > 0 && !SLOPE && p.pre.dtype == FSDP_DTYPE_ACT8 && p.pre.p != nullptr && row0 + lane < p.M && col0 < p.N)
        p.pre.e[(row0 + lane) * p.pre.eld + (col0 >> 5)] = static_cast<uint8_t>(byte);
}

// Rows of a bf16 matrix that do not start on 16-byte boundaries, copied to ones
// that do (dst.ld a multiple of 8): eight elements to a thread, from the two
// 16-byte words that hold them, moved together.  A word is read only if it holds
// a byte between the matrix's first element and its last; what dst gets past a
// row's end is not defined.  Bound by latency at the sizes that come unaligned:
// 5121 x 1283 in 6.0 us.
__global__ void __launch_bounds__(256) align_rows_kernel(int64_t rows, int64_t cols, Mat src, Mat dst, uint32_t chunks) {
    starts_early();
    after_previous();
    const uintptr_t end = reinterpret_cast<uintptr_t>(src.p) + ((rows - 1) * src.ld + cols) * 2;
    const int64_t count = rows * chunks, stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < count; i += stride) {
        const int64_t row = i <= 0xffffffffll ? static_cast<uint32_t>(i) / chunks : i / chunks;
        const int64_t c = (i - row * chunks) * 8;
        const uintptr_t from = reinterpret_cast<uintptr_t>(src.p) + (row * src.ld + c) * 2;
        const uintptr_t word = from & ~uintptr_t(15);
        const uint4 a = *reinterpret_cast<const uint4*>(word);
        uint4 b = make_uint4(0, 0, 0, 0);
        if (from != word && word + 16 < end) b = *reinterpret_cast<const uint4*>(word + 16);
        const uint32_t shift = static_cast<uint32_t>(from & 2) * 8;
        uint4 o;
        switch ((from >> 2) & 3) {
            case 0:
                o = make_uint4(__funnelshift_r(a.x, a.y, shift), __funnelshift_r(a.y, a.z, shift), __funnelshift_r(a.z, a.w, shift),
                               __funnelshift_r(a.w, b.x, shift));
                break;
            case 1:
                o = make_uint4(__funnelshift_r(a.y, a.z, shift), __funnelshift_r(a.z, a.w, shift), __funnelshift_r(a.w, b.x, shift),
                               __funnelshift_r(b.x, b.y, shift));
                break;
            case 2:
                o = make_uint4(__funnelshift_r(a.z, a.w, shift), __funnelshift_r(a.w, b.x, shift), __funnelshift_r(b.x, b.y, shift),
                               __funnelshift_r(b.y, b.z, shift));
                break;
            default:
                o = make_uint4(__funnelshift_r(a.w, b.x, shift), __funnelshift_r(b.x, b.y, shift), __funnelshift_r(b.y, b.z, shift),
                               __funnelshift_r(b.z, b.w, shift));
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst.p) + row * dst.ld + c) = o;
    }
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

bool tma_ready(const Mat& m) { return m.dtype == FSDP_DTYPE_BF16 && rows_aligned(m); }

// The driver's tensor-map encoder, looked up once (no link against libcuda).
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
    static std::once_flag once;
    static Encode fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) == cudaSuccess &&
            found == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<Encode>(p);
    });
    return fn;
}

// rows x cols of bf16, copied in boxes of box_rows x 64 columns.
cudaError_t make_map(CUtensorMap* map, const Mat& m, int64_t rows, int64_t cols, int box_rows) {
    const Encode fn = encoder();
    if (fn == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(m.ld) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, m.p, dims, strides, box, steps,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

using FinishKernel = void (*)(Product, Plan);
const FinishKernel kFinishKernels[2][3] = {
    {finish_kernel<0, false>, finish_kernel<1, false>, finish_kernel<2, false>},
    {finish_kernel<0, true>, finish_kernel<1, true>, finish_kernel<2, true>}};
using ProductKernel = void (*)(CUtensorMap, CUtensorMap, Product, Plan);
const ProductKernel kProductKernels[2][3] = {
    {product_kernel<0, false>, product_kernel<1, false>, product_kernel<2, false>},
    {product_kernel<0, true>, product_kernel<1, true>, product_kernel<2, true>}};

}  // namespace

int product_clusters(int sms) {
    const int most = once_per_device([] {
        for (const ProductKernel* row : kProductKernels)
            for (int i = 0; i < 3; ++i)
                if (cudaFuncSetAttribute(row[i], cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2 * kMaxClusters);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        int n = 0;
        return cudaOccupancyMaxActiveClusters(&n, kProductKernels[0][0], &cfg) == cudaSuccess ? n : 0;
    });
    return std::min(std::min(most, sms / 2), kMaxClusters);
}

size_t product_copy_bytes(const Mat& m, int64_t rows, int64_t cols) {
    return tma_ready(m) ? 0 : static_cast<size_t>(round_up(rows * round_up(cols, 8) * 2, 256));
}

namespace {

// An operand as the copies need it: itself, or an aligned bf16 copy in *room.
cudaError_t settle(Mat* m, int64_t rows, int64_t cols, char** room, int sms, cudaStream_t st) {
    if (tma_ready(*m)) return cudaSuccess;
    Mat d{};
    d.p = *room;
    d.ld = round_up(cols, 8);
    d.dtype = FSDP_DTYPE_BF16;
    *room += product_copy_bytes(*m, rows, cols);
    cudaError_t e;
    if (m->dtype == FSDP_DTYPE_ACT8) {
        // the checkpoint's pad elements are zeros: whole vectors can be read
        e = launch_act8_unpack(rows, d.ld, *m, FSDP_ACTIVATION_NONE, d, sms, st);
    } else {
        const int64_t count = rows * (d.ld / 8);
        const dim3 grid(static_cast<unsigned>(std::min<int64_t>((count + 255) / 256, static_cast<int64_t>(sms) * 16)));
        e = launch_early(align_rows_kernel, grid, 256, 0, st, rows, cols, *m, d, static_cast<uint32_t>(d.ld / 8));
    }
    *m = d;
    return e;
}

}  // namespace

cudaError_t launch_product(const Product& given, const ProductRoom& room, int sms, cudaStream_t st) {
    Product p = given;
    if (p.M == 0 || p.N == 0) return cudaSuccess;
    if (p.K == 0) {   // an empty sum
        if (p.add.p == p.out.p) return cudaSuccess;
        const size_t esz = p.out.dtype == FSDP_DTYPE_F32 ? 4 : 2;
        return cudaMemset2DAsync(p.out.p, p.out.ld * esz, 0, p.N * esz, p.M, st);
    }
    if (few_rows(p)) return launch_few_rows(p, sms, st);
    const int clusters = product_clusters(sms);
    if (clusters < 1) return cudaErrorNotSupported;
    char* copies = room.copies;
    cudaError_t e = settle(&p.a, p.a_trans ? p.K : p.M, p.a_trans ? p.M : p.K, &copies, sms, st);
    if (e == cudaSuccess) e = settle(&p.b, p.b_trans ? p.K : p.N, p.b_trans ? p.N : p.K, &copies, sms, st);
    if (e != cudaSuccess) return e;

    const auto all_aligned = [&](uintptr_t to) {
        for (const Mat* m : {&p.out, &p.add, &p.pre})
            if (m->p != nullptr && !rows_aligned(*m, to)) return false;
        return p.N % static_cast<int64_t>(to / 2) == 0;
    };
    const int vec = all_aligned(32) && (reinterpret_cast<uintptr_t>(p.bias) & 15u) == 0 ? 2 : all_aligned(16) ? 1 : 0;
    // Few rows: they become the tile's columns, so that a tile of 256 is not
    // filled with rows that do not exist.
    int64_t rows = p.M, cols = p.N;
    const bool swap = swaps(p.M, p.N, p.a_trans);
    if (swap) {
        std::swap(p.a, p.b);
        std::swap(p.a_trans, p.b_trans);
        std::swap(rows, cols);
    }
    const bool keeps = !p.slope && p.pre.p != nullptr;
    const Sums sums = keeps && p.pre.dtype == FSDP_DTYPE_ACT8 ? Sums::kKept
                      : p.out.dtype == FSDP_DTYPE_F32 || (keeps && p.pre.dtype == FSDP_DTYPE_F32) ? Sums::kExact : Sums::kRounded;
    Plan pl{plan_product(rows, cols, p.K, p.b_trans, sums, clusters)};
    pl.swapped = swap;
    pl.vec = swap ? 0 : vec;
    pl.partials = room.partials;
    pl.status = room.status;
    pl.wait_cycles = static_cast<long long>(room.wait_ns) * 2;   // the SM clock is at most 2.07 GHz
    pl.withhold = room.withhold;
    CUtensorMap map_a, map_b;
    e = p.a_trans ? make_map(&map_a, p.a, p.K, rows, kDepth) : make_map(&map_a, p.a, rows, p.K, 128);
    if (e == cudaSuccess) e = p.b_trans ? make_map(&map_b, p.b, p.K, cols, kDepth) : make_map(&map_b, p.b, cols, p.K, pl.bn / 2);
    if (e != cudaSuccess) return e;
    if (static_cast<int64_t>(pl.tiles_m) * pl.tiles_n > 0x7fffffff) return cudaErrorInvalidValue;   // far beyond any memory
    const unsigned grid = 2 * static_cast<unsigned>(std::min<int64_t>(pl.units, clusters));
    e = launch_early(kProductKernels[p.slope][pl.vec], dim3(grid), kThreads, kSmemBytes, st, map_a, map_b, p, pl);
    const int64_t shared = static_cast<int64_t>(pl.tiles_m) * pl.tiles_n - pl.whole;
    if (e != cudaSuccess || shared == 0) return e;
    return launch_early(kFinishKernels[p.slope][pl.vec], dim3(static_cast<unsigned>(shared * (pl.bn / 4))), 128, 0,
                        st, p, pl);
}

int64_t column_sum_partials(int64_t rows, int64_t cols, int sms) {
    // about two blocks to an SM, of at least 32 rows each
    const int64_t blocks = (cols + 255) / 256;
    return std::max<int64_t>(1, std::min<int64_t>((rows + 31) / 32, (2 * sms + blocks - 1) / blocks));
}

cudaError_t launch_column_sum(int64_t rows, int64_t cols, const Mat& dy, float* partials, void* out, int out_dtype,
                              int accumulate, int sms, cudaStream_t st) {
    int64_t count = 0;
    if (rows > 0) {
        count = column_sum_partials(rows, cols, sms);
        const bool vec = rows_aligned(dy) && cols % 8 == 0;
        const dim3 grid(static_cast<unsigned>(vec ? (cols + 255) / 256 : (cols + 31) / 32), static_cast<unsigned>(count));
        const cudaError_t e = launch_early(vec ? column_sum_kernel<8> : column_sum_kernel<1>, grid, 256, 0, st, rows, cols, dy, partials);
        if (e != cudaSuccess) return e;
    }
    return launch_sum_partials(partials, count, cols, cols, out, out_dtype, accumulate, st);
}

}  // namespace fsdp
