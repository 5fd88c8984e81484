// How a product is cut into tiles, rounds, parts and slices.  Plain C++, so that
// tests can ask for the plan of a shape without a GPU.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace fsdp {

constexpr int kStagesMost = 10;
constexpr int kDepth = 64;                       // k per stage (3 stages of 128 were 4 % slower at 8192^3)
constexpr int kBlock = 64 * kDepth * 2;          // a box of an operand that is contiguous along its rows: 64 rows
constexpr int kStageA = 128 * kDepth * 2;        // bytes of A in a stage, per CTA
constexpr int kRingBytes = 6 * (128 + 128) * 64 * 2;   // 6 stages at BN = 256, more of narrower tiles

struct Tiling {
    int ks;                    // stages' worth of k
    int bn;                    // columns of a tile: 32 .. 256 in steps of 32
    int stages, stage_b;       // stages in the ring, and B's bytes in one, per CTA
    int slice;                 // stages after which the sums leave the tensor cores' accumulator
    int two;                   // 1: two accumulators in turn, so that an epilogue runs beside the next products; 0: one
    int buffer;                // columns of tensor memory between the two
    int running;               // the column where the running sums of slices start
    int tiles_m, tiles_n;
    uint32_t whole;            // tiles done by one cluster each
    uint32_t units;            // whole + (tiles - whole) * parts
    int parts;                 // clusters that share one of the remaining tiles, along k
};

// What a product's sums are for: a BF16 result, an F32 one, or an 8-bit checkpoint.
enum class Sums { kRounded, kExact, kKept };

// Few rows become the tile's columns, so that a tile of 256 is not filled with rows
// that do not exist.
inline bool swaps(int64_t M, int64_t N, bool a_trans) { return M <= 256 && N > M && !a_trans; }

// Tiles, and how the last ones are shared: the clusters take whole tiles in
// turn; what is left over after the last full round may be cut along k so that
// every cluster has a part.  The width and the choice are those of the least
// estimated time, in cycles.  Measured with whole rounds of tiles: a stage takes
// 2.3 cycles a column where the products bound it (256: 580, 192: 453), what its
// copies take at 75 bytes a cycle an SM (32 KiB: 442), and 275 at least; a
// tile's epilogue 13 a column.
//
// Long sums: in every step of 16 products the tensor cores cut what they add off
// below the accumulator's last bits.  Measured, in units of 2^-23 of the running
// sum a step: products of random signs err by 1.1e-9 k in all; products of one
// sign and size by 0.2 units at k = 768 and 0.75 at 300000, all one way; small
// products on one large sum by 2.3, at most 3.8.  So a cluster's k is taken in
// slices of equal length, at whose ends the accumulator is emptied and added to
// the running sums in fp32, rounded to nearest.
//
// F32 results: at most kSlice stages (768).  Random signs err by 7.3e-7 at any k,
// products of one sign by 1.3e-6.  The running sums need tensor memory, which
// leaves two accumulators of at most 160 columns: 8192 x 4608 x 4608 at 1610
// TFLOP/s against 1700 uncut, 1630 with slices of 1024 (1.0e-6 for random signs),
// 1655 with 2048 (2.1e-6), 1570 with 512 (4.7e-7).
//
// 8-bit checkpoints: their rounding shows an error of the sums by a whole step, so
// that twice the error doubles the elements which land on the wrong side.  A slice
// is also at most 16 sqrt(k) products long (256 at least), which keeps the sums'
// error within about twice that of fp32 sums in order, 8e-9 sqrt(k) measured.  4096
// x 1280 -> 5120 with GELU and checkpoint, and its unpacking: 65.4 us with slices of
// 448, 61.0 with 640, 54.7 uncut; the kept values' error, as a norm, is 1.2, 1.5 and
// 1.9 times that from fp32 sums.
//
// BF16 results: at most kSliceBf16 stages (16384), so that a drift of one way stays
// near 1e-4, where BF16's own rounding is up to 2^-8 (uncut, it reached 1.7e-3 at
// k = 300000).  There a tile is as wide as it would be uncut, with one accumulator
// beside its running sums: the products wait while a slice's sums are taken.  4096
// x 49152 -> 12288: 2864 us against 2846 uncut; with two accumulators and tiles of
// 160 columns, 3335.  Slices of 8192 cost 25 us more.
constexpr int kSlice = 12;
constexpr int kSliceBf16 = 256;
constexpr int kSlicedTwice = 160;   // columns of tensor memory that hold two accumulators and the running sums

// Stages of a slice, at most.
inline int longest_slice(int64_t k, Sums sums) {
    if (sums == Sums::kRounded) return kSliceBf16;
    if (sums == Sums::kExact) return kSlice;
    return std::min(kSlice, std::max(4, static_cast<int>(std::sqrt(static_cast<double>(k)) * 16 / kDepth)));
}

inline Tiling plan_product(int64_t rows, int64_t cols, int64_t k, bool b_by_rows, Sums sums, int clusters) {
    const int longest = longest_slice(k, sums);
    Tiling best{};
    double least = 0;
    for (int bn = 256; bn >= 32; bn -= 32) {
        if (bn < 256 && bn >= 2 * cols && bn > 32) continue;
        Tiling p{};
        p.ks = static_cast<int>((k + kDepth - 1) / kDepth);
        p.bn = bn;
        p.tiles_m = static_cast<int>((rows + 255) / 256);
        p.tiles_n = static_cast<int>((cols + bn - 1) / bn);
        const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
        const double steps = static_cast<double>((k + 15) / 16) / (kDepth / 16);   // stages, the last one in part
        p.stage_b = b_by_rows ? (bn > 128 ? 2 : 1) * kBlock : bn / 2 * kDepth * 2;   // a multiple of 1024
        p.stages = std::min(kStagesMost, kRingBytes / (kStageA + p.stage_b));
        const double copied = kStageA + p.stage_b;
        const double stage = std::max({2.3 * bn + 10.0, 275.0, copied / 75.0});
        for (int share = 0; share < 2; ++share) {
            const int64_t left = tiles % clusters;
            p.parts = share == 0 || left == 0 ? 1 : static_cast<int>(std::min<int64_t>(clusters / left, std::max(1, p.ks / 4)));
            if (share == 1 && p.parts == 1) continue;
            p.whole = static_cast<uint32_t>(p.parts > 1 ? tiles - left : tiles);
            p.units = static_cast<uint32_t>(p.whole + (tiles - p.whole) * p.parts);
            const int deepest = p.whole > 0 ? p.ks : (p.ks + p.parts - 1) / p.parts;
            const int slices = (deepest + longest - 1) / longest;
            p.slice = slices > 1 ? (deepest + slices - 1) / slices : 0x40000000;   // of equal length
            p.two = slices == 1 || bn <= kSlicedTwice;
            if (!p.two && sums != Sums::kRounded) continue;
            p.buffer = slices > 1 && p.two ? bn : 256;
            p.running = p.two ? 2 * p.buffer : p.buffer;
            const double rounds = static_cast<double>((p.whole + clusters - 1) / clusters);
            // a slice's sums: the products wait while they are taken where there is one
            // accumulator, and for an epilogue that has a checkpoint to keep besides
            const double waits = !p.two ? slices * 6.0 * bn : sums == Sums::kKept ? (slices - 1) * 1000.0 : 0.0;
            double t = rounds * (std::max(steps * stage, 400.0 + 13.0 * bn) + waits + 300.0) + 13.0 * bn;
            if (p.parts > 1) t += (p.ks + p.parts - 1) / p.parts * stage + 9000.0 + 60.0 * p.parts;
            if (least == 0 || t < least) {
                least = t;
                best = p;
            }
        }
    }
    return best;
}

}  // namespace fsdp
