// Prints the plan of each call named on a line of standard input:
//   gemm OUT IN M F32        -> kind whole slices tiles (kind -1: the few-token kernel)
//   backward M OUT IN K ASK  -> dx_slices dw_large dw_slices both (ASK: 1 dX, 2 dW, 3 both)
// Test infrastructure: built and run by tests/test_f8_plans_cpu.py.
#include <cstdio>
#include <cstring>

#include "ckpt_plan.h"
#include "f8_plan.h"

int main() {
    char what[16];
    int a, b, c, d, e;
    while (std::scanf("%15s", what) == 1) {
        if (std::strcmp(what, "gemm") == 0) {
            if (std::scanf("%d %d %d %d", &a, &b, &c, &d) != 4)
                return 1;
            if (c <= rbq::F8_FEW || !rbq::gemm_f8_tile_supports(a, b, c)) {
                std::puts("-1 0 1 0");
                continue;
            }
            const rbq::f8_plan p = rbq::plan_tiles(a, b, c, d);
            const long long rows = rbq::F8_ROWS[p.kind], tokens = rbq::F8_TOKENS[p.kind];
            std::printf("%d %d %d %lld\n", p.kind, p.whole, p.slices, (a + rows - 1) / rows * ((c + tokens - 1) / tokens));
        } else {
            if (std::scanf("%d %d %d %d %d", &a, &b, &c, &d, &e) != 5)
                return 1;
            const rbq::ck_plan p = rbq::plan_backward(a, b, c, d, e & 1, e & 2);
            std::printf("%d %d %d %d\n", p.dx_slices, p.dw_large, p.dw_slices, (int)p.both);
        }
    }
    return 0;
}
