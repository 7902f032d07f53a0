// For each "ROWS TOKENS IN" on a line of standard input: goes through every load of codes
// and tokens of a tile of gemm_q4 with that many rows, tokens and columns, and prints
//   <loads of codes behind the tile's end> <of tokens> <columns that do not meet their
//   tokens once> <rows or tokens that are not written once>
// Test infrastructure: built and run by tests/test_q4_loads_cpu.py.
#include <cstdio>
#include <vector>

#include "q4_plan.h"

using namespace rbq;

int main() {
    int rows, toks, in;
    while (std::scanf("%d %d %d", &rows, &toks, &in) == 3) {
        const int T = (in + 127) / 128;
        long codes_out = 0, tokens_out = 0, unmet = 0, unwritten = 0;
        std::vector<int> wrote(rows), spoke(toks);
        for (int at = 0; at < Q4_ROWS; at += 16) {
            const int first = q4_first(at, rows);
            for (int li = 0; li < 16; ++li) {
                if (first + li < rows && first + li >= at)
                    ++wrote[first + li];
                for (int t = 0; t < T; ++t)
                    for (int g = 0; g < 4; ++g) {
                        const int64_t b = (int64_t)first * (in / 2) + q4_column(in, t) / 2 + q4_lane_codes(rows, in, li, g);
                        codes_out += b + 16 > (int64_t)rows * (in / 2);
                        if (first + li < rows)      // the row's own codes
                            codes_out += b / (in / 2) != first + li || b % (in / 2) + 16 > in / 2;
                    }
            }
        }
        for (int at = 0; at < Q4_TOKENS; at += 16) {
            const int first = q4_first(at, toks);
            for (int m = 0; m < 16; ++m) {
                if (first + m < toks && first + m >= at)
                    ++spoke[first + m];
                for (int t = 0; t < T; ++t) {
                    std::vector<int> met(128);
                    const int column = q4_column(in, t);
                    // what reads as 0 passes the range, with or without the scalar part taken off it
                    const uint32_t range = at < toks ? (uint32_t)toks * in * 2 : 0, scalar = at < toks ? (uint32_t)first * in * 2 + column * 2 : 0;
                    tokens_out += Q4_BEYOND < range || Q4_BEYOND < range - scalar;
                    for (int q = 0; q < 16; ++q) {
                        const uint32_t lane = column + q * 8 >= t * 128 ? q4_lane_tokens(toks, in, m, q) : Q4_BEYOND;
                        if (lane == Q4_BEYOND)
                            continue;
                        const int64_t b = (int64_t)first * in * 2 + (int64_t)column * 2 + lane;
                        tokens_out += b + 16 > (int64_t)toks * in * 2;
                        if (first + m < toks)
                            tokens_out += b / (in * 2) != first + m || b % (in * 2) + 16 > in * 2;
                        // the 8 columns of codes that these meet: word q % 4 of lane group q / 4
                        const int c = (int)(b % (in * 2)) / 2;
                        const int w = (int)(q4_lane_codes(16, in, 0, q / 4) + column / 2) * 2 + q % 4 * 8;
                        unmet += c != w || c < t * 128;
                        for (int e = 0; e < 8 && c - t * 128 + e < 128; ++e)
                            ++met[c - t * 128 + e];
                    }
                    for (int c = 0; c < 128; ++c)
                        unmet += met[c] != (t * 128 + c < in);
                }
            }
        }
        for (int n : wrote)
            unwritten += n != 1;
        for (int n : spoke)
            unwritten += n != 1;
        std::printf("%ld %ld %ld %ld\n", codes_out, tokens_out, unmet, unwritten);
    }
    return 0;
}
