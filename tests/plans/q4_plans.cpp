// Prints the plan of each call named on a line of standard input:
//   gemm OUT IN M      -> tiled slices four staged row_tiles lds (the few-token kernel where tiled is 0)
//   logits M VOCAB K   -> slices threads bytes
// Test infrastructure: built and run by tests/test_q4_plans_cpu.py.
#include <cstdio>
#include <cstring>

#include "logits_plan.h"
#include "q4_plan.h"

int main() {
    char what[16];
    int a, b, c;
    while (std::scanf("%15s %d %d %d", what, &a, &b, &c) == 4) {
        if (std::strcmp(what, "gemm") == 0) {
            if (rbq::q4_tiled(a, b, c)) {
                std::printf("1 %d 0 0 0 0\n", rbq::q4_slices(a, b, c));
                continue;
            }
            const rbq::q4_few_plan p = rbq::plan_q4_few(a, b, c);
            const size_t T = (b + 127) / 128, rows = 16 * p.row_tiles;
            std::printf("0 1 %d %d %d %zu\n", (int)p.four, (int)p.staged, p.row_tiles,
                        p.staged ? rbq::q4_staged_scales((int)rows, (int)T) + rows * T : (size_t)0);
        } else {
            const int S = rbq::logits_slices(a, b), vectors = (b + rbq::LG_VEC - 1) / rbq::LG_VEC;
            std::printf("%d %d %zu\n", S, rbq::logits_threads((vectors + S - 1) / S, c), rbq::logits_workspace_bytes(a, b, c, 0));
        }
    }
    return 0;
}
