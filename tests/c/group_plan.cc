// Prints the plan of each fused product given on stdin: lines "dx experts rows
// columns contraction rank" to "tile tile_rows splits steps pairs" (pairs: CTA
// pairs that are resident together on 148 SMs).
#include <cstdio>

#include "group_plan.h"

int main() {
    int dx, E, r;
    long long M, cols, contraction;
    while (std::scanf("%d %d %lld %lld %lld %d", &dx, &E, &M, &cols, &contraction, &r) == 6) {
        const nf4lora::FusedPlan p = nf4lora::plan_fused(dx != 0, E, M, cols, contraction, r, 148);
        std::printf("%d %d %d %d %d\n", p.tile, p.tile_rows, p.splits, p.k_main, p.tile <= 64 ? 148 : 74);
    }
    return 0;
}
