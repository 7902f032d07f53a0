// f8_plan.h -- which kernel, tile and slices a product in 8-bit floating point
// blocks takes.  Host arithmetic only, so that a test can ask it without a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace rbq {

// Up to this many tokens: the few-token kernel (f8.hip); more: gemm_f8.hip.
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
// serve only that), and 1.95, 1.1, 0.75 (exact products).  It picked the fastest kind, or one within 7 % of it, for 65
// to 2048 tokens on 1000 to 14336 rows; e.g. 128 tokens, 4096 x 4096: 14.6 us
// with 64 x 128 in 4 slices, 48.9 with 256 x 256; 2048 tokens: 39.3 with
// 128 x 256, 54.9 with 256 x 256, 67.2 with 64 x 128; 1024 tokens, 11008 x
// 4096: 63.0 with 256 x 256, 73.4 with 128 x 256.  Tiles of 192 rows, one round
// in place of one and a third or of a part empty one: 2048 tokens, 6144 x 4096:
// 64.2 us with 256 rows, 59.1 with 192; 1024 tokens, 11008 x 4096: 63.3 and
// 56.8; of 224: 2048 tokens, 11008 x 4096: 120.3 and 113.2; 14336 x 4096: 133.3
// and 131.2.  Slices for the last round
// only: fp32 outputs, 777 tokens, 5003 x 4128 (256 + 24 tiles of 128 x 128):
// 73.0 us without, 63.1 with them; 1066 tokens, 7568 x 3040: 85.5 and 74;
// fp16, 300 tokens, 11008 x 4096: 37.3 and 33.2.
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
