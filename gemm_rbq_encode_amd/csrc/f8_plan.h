// f8_plan.h -- which kernel, tile and slices a product in 8-bit floating point
// blocks takes.  Host arithmetic only, so that a test can ask it without a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace rbq {

// Up to this many tokens: the few-token kernel (f8.hip); more: the tiled ones
// (gemm_f8.hip).  The number decides the arithmetic of fp16 outputs as well
// (exact products up to it), so it is one for all sizes.  us of the few-token
// kernel and of the tiles, W from HBM, fp16 outputs:
//                    17 tokens      32 tokens      33 tokens      64 tokens
//    4096 x  1024     4.5   6.7      4.9   6.8      5.6   6.9      6.4   7.1
//    4096 x  4096     8.0  11.5      9.2  12.9     12.0  13.0     14.6  13.1
//    8192 x  4096    13.6  14.4     15.7  14.4     22    14.5     28    15.7
//   11008 x  4096    17.8  18.7     21.5  17.8     29    17.7     37    18.4
//   22016 x  4096    28.8  28.7     32.3  26.5     51    26.6     58    27.2
//    4096 x 14336    21.9  19.2     24.7  19.1     35    19.1     45    20.4
// Small layers would keep the few-token kernel up to 64 tokens, by up to 35 %;
// large ones and long rows would leave it at 17 to 24, by up to 25 %.
constexpr int F8_FEW = 32;

// Byte offsets inside a tile are 32-bit and the tiles are numbered in 31 bits.
inline bool gemm_f8_tile_supports(int out, int in, int M) {
    return in <= (1 << 23) && ((int64_t)out / 64 + 1) * ((int64_t)M / 128 + 1) < (1 << 22);
}

// Kinds of tiles (rows x tokens); the first are those of the large kernel.
constexpr int F8_LARGE = 3, F8_KINDS = 6;
constexpr int F8_ROWS[F8_KINDS] = {256, 224, 192, 128, 128, 64}, F8_TOKENS[F8_KINDS] = {256, 256, 256, 256, 128, 128};

// The kind, tiles computed whole, and slices of the others.
struct f8_plan {
    int kind, whole, slices;
};

// The choice is the least of a simple cost: every kind keeps one workgroup per
// compute unit, so a launch takes ceil(workgroups / 256) rounds of its blocks'
// stages and a start of 2.5 us each; slices add a second launch and the write
// and read of the partial sums.  Stage times measured on full launches: us per
// block 1.8, 1.62, 1.42, 1.05, 0.68, 0.47 (the 8-bit instruction; the large tiles
// serve only that), and 1.95, 1.1, 0.75 (exact products).
//
// It picked the fastest kind, or one within 8 % of it, for 48 to 2048 tokens on
// 1000 to 22016 rows (33 tokens, 4096 x 4096: 13.4 us where 64 x 128 in other
// slices takes 11.6).  us, fp16 outputs: 128 tokens, 4096 x 4096: 14.9 with 64 x
// 128 in 4 slices, 18.5 uncut, 17.1 with 128 x 128, 52 with 256 x 256; 2048
// tokens, 4096 x 4096: 40.5 with 128 x 256, 50.4 with 128 x 128, 69.7 with 64 x
// 128.  Tiles of 192 and 224 rows, one round in place of one and a third or of a
// part empty one: 1024 tokens, 11008 x 4096: 57.0 with 192 rows, 61.4 without that
// kind; 14336 x 4096: 66.9 with 224, 71.2 without; 2048 tokens, 14336 x 4096: 128
// with 224, 138 without; 6144 x 4096: 56.9 with 192, 59.4 without.  Slices for
// the last round only: exact products, 777 tokens, 5003 x 4128 (256 + 24 tiles
// of 128 x 128): 59.2, uncut 67.4; 1066 tokens, 7568 x 3040: 73.2 and 85.9; fp16,
// 300 tokens, 11008 x 4096: 33.6 and 36.7.
inline f8_plan plan_tiles(int out, int in, int M, int exact) {
    static constexpr float stage[2][F8_KINDS] = {{1.8f, 1.62f, 1.42f, 1.05f, 0.68f, 0.47f},
                                                 {0.0f, 0.0f, 0.0f, 1.95f, 1.1f, 0.75f}};
    static constexpr int splits[] = {1, 2, 3, 4, 6, 8};
    const int T = (int)(((int64_t)in + 127) / 128);
    f8_plan best = {F8_LARGE, 0, 1};
    float least = 0.0f;
    for (int k = exact ? F8_LARGE : 0; k < F8_KINDS; ++k) {
        const int64_t tiles = (((int64_t)out + F8_ROWS[k] - 1) / F8_ROWS[k]) *
                              (((int64_t)M + F8_TOKENS[k] - 1) / F8_TOKENS[k]);
        // (the whole rounds computed whole, or every tile cut)
        for (int64_t whole = tiles / 256 * 256;; whole = 0) {
            for (const int S : splits) {
                if (S > 1 && (k < F8_LARGE || 2 * S > T))
                    break;
                const int64_t cut = tiles - whole;
                float cost = (float)(whole / 256) * ((float)T * stage[exact][k] + 2.5f) +
                             (float)((cut * S + 255) / 256) * ((float)((T + S - 1) / S) * stage[exact][k] + 2.5f);
                if (S > 1)
                    cost += 4.0f + (float)S * (8.0f / 6.0e6f) *
                                       std::min((float)cut * (float)(F8_ROWS[k] * F8_TOKENS[k]), (float)M * (float)out);
                if (least == 0.0f || cost < least) {
                    least = cost;
                    best = {k, (int)whole, S};
                }
            }
            if (whole == 0)
                break;
        }
    }
    return best;
}

}  // namespace rbq
