// The plan of each product asked for on a line of standard input:
//     M N K a_trans b_trans sums clusters
// (sums: 0 for a BF16 result, 1 for an F32 one, 2 for an 8-bit checkpoint)
// as launch_product makes it, printed as name=value pairs.
#include <cstdio>
#include <utility>

#include "product_plan.hpp"

int main() {
    long long M, N, K;
    int at, bt, sums, clusters;
    while (std::scanf("%lld %lld %lld %d %d %d %d", &M, &N, &K, &at, &bt, &sums, &clusters) == 7) {
        const bool swapped = fsdp::swaps(M, N, at != 0);
        if (swapped) {
            std::swap(M, N);
            std::swap(at, bt);
        }
        const fsdp::Tiling t = fsdp::plan_product(M, N, K, bt != 0, static_cast<fsdp::Sums>(sums), clusters);
        std::printf("swapped=%d by_rows=%d ks=%d bn=%d stages=%d stage_b=%d slice=%d two=%d buffer=%d running=%d tiles_m=%d "
                    "tiles_n=%d whole=%u units=%u parts=%d\n",
                    swapped, bt != 0, t.ks, t.bn, t.stages, t.stage_b, t.slice, t.two, t.buffer, t.running, t.tiles_m, t.tiles_n,
                    t.whole, t.units, t.parts);
    }
    return 0;
}
