// q4_plan.h -- which kernel, tile and slices a product in 4 bits takes.  Host
// arithmetic only, so that a test can ask it without a GPU.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace rbq {

// The few-token kernel (q4.hip) up to 16 tokens, and above as long as it has little
// to do.  It took, the many-token kernel (gemm_q4.hip) took, in us:
//      32 tokens, 11008 x 4096      16.7    24
//      64          4096 x 4096      13.5    19
//     128          4096 x 4096      22.8    23.4
//      64          4096 x 11008     29      23
//      32         28672 x 8192      79      57
inline bool q4_few(int out, int in, int M) {
    return M <= 16 || (double)M * out * in <= 2e9;
}

// Groups of a row whose scales and zero points the few-token kernel takes into LDS:
// 48 rows' 3 bytes a group, beside the 32 KB of its tokens, in 64 KB.
constexpr int Q4_STAGED_GROUPS = 224;

// Bytes of the scales of some rows there.
constexpr size_t q4_staged_scales(int rows, int T) {
    return ((size_t)rows * T * 2 + 15) / 16 * 16;
}

struct q4_few_plan {
    bool four;          // up to 4 tokens
    bool staged;        // scales through LDS
    int row_tiles;      // of a workgroup
};

// Row tiles: up to 4 tokens one (11008 x 4096: 7.3 us with one, 8.0 with two;
// 128256 x 4096: 54 and 50).  Else more tiles use the tokens again: three if that
// makes one round of all workgroups (16 tokens, 11008 x 4096: 11.9 us with one, 11.7
// with two, 9.8 with three), two where there are more rounds (128256 x 4096: 110, 83,
// 92), one where the workgroups would not fill the chip (4096 x 4096: 6.0, 6.9, 8.4).
inline q4_few_plan plan_q4_few(int out, int in, int M) {
    q4_few_plan p = {M <= 4, (in + 127) / 128 <= Q4_STAGED_GROUPS, 1};
    const int64_t tiles = ((int64_t)out + 15) / 16;
    if (p.staged && !p.four)
        p.row_tiles = tiles <= 256 ? 1 : tiles > 512 && tiles <= 768 ? 3 : 2;
    return p;
}

// Tiles of the many-token kernel (gemm_q4.hip).
constexpr int Q4_ROWS = 256, Q4_TOKENS = 64;

// The loads of a tile are sixteen rows or tokens by a group of 128 columns, all inside
// the tile whatever its size: sixteen that would end behind its last one are its last
// sixteen, where there are fewer the last one is repeated (what stands twice is written
// once), and a row's short last group is its last 128 columns, with the tokens of the
// columns before that group 0.  Of rows shorter than 128 columns a lane's piece of codes
// behind the end is the last one, with tokens 0.
constexpr uint32_t Q4_BEYOND = 0x80000000u;      // an offset that reads as 0: behind every range

constexpr int q4_first(int at, int count) {      // first of the sixteen that stand for at .. at + 15
    return std::max(0, std::min(at, count - 16));
}
constexpr int q4_column(int in, int t) {         // first column of what is loaded for group t
    return std::min(t * 128, std::max(in - 128, 0));
}
// Bytes from the first of sixteen rows (tokens) and the first column on: of row li's 32
// codes from column 32 g on, of token m's 8 columns from column 8 q on.
constexpr uint32_t q4_lane_codes(int rows, int in, int li, int g) {
    return (uint32_t)std::min(li, rows - 1) * (uint32_t)(in / 2) + (uint32_t)std::min(g * 16, in / 2 - 16);
}
constexpr uint32_t q4_lane_tokens(int toks, int in, int m, int q) {
    return q * 8 < in ? (uint32_t)std::min(m, toks - 1) * (uint32_t)in * 2u + (uint32_t)q * 16u : Q4_BEYOND;
}

// Offsets inside a tile are 32-bit and the tiles are numbered in 31 bits.
inline bool q4_tiled(int out, int in, int M) {
    return !q4_few(out, in, M) && in <= (1 << 23) && ((int64_t)out / Q4_ROWS + 1) * ((int64_t)M / Q4_TOKENS + 1) < (1 << 24);
}

// Slices of the columns, by what was measured (S = 1 .. 16 at twelve sizes): a
// workgroup takes 1.1 us for a group and 7 to begin and end, every 256 take that
// long again (two on a CU take twice as long), and joining slices takes 4 us and
// their sums' way through memory.  64 tokens of 4096 x 4096: 41.8 us with one, 28.4
// two, 20.6 four, 19.1 eight, 22.7 sixteen; 128 of 11008 x 4096: 42.5, 33.1, 32.7,
// 39.7, 55.
inline int q4_slices(int out, int in, int M) {
    const int T = (in + 127) / 128;
    const int64_t tiles = (((int64_t)out + Q4_ROWS - 1) / Q4_ROWS) * (((int64_t)M + Q4_TOKENS - 1) / Q4_TOKENS);
    int best = 1;
    double least = 0.0;
    for (int S = 1; S <= 16 && 2 * S <= T + 1; ++S) {
        const double rounds = (double)((tiles * S + 255) / 256);
        double cost = rounds * ((T + S - 1) / S) * 1.1 + 7.0;
        if (S > 1)
            cost += 4.0 + (double)(S + 1) * 4.0 * (double)M * (double)out / 3.0e6;
        if (S == 1 || cost < least) {
            least = cost;
            best = S;
        }
    }
    return best;
}

}  // namespace rbq
