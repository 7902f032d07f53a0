// q4_plan.h -- which kernel, tile and slices a product in 4 bits takes.  Host
// arithmetic only, so that a test can ask it without a GPU.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace rbq {

// The few-token kernel (q4.hip) up to 32 tokens, and above as long as it has little
// to do: it took 13.9 us for 64 tokens of 4096 x 4096, 25 of 11008 x 4096, 109 of
// 28672 x 8192, the tiled one 26, 30 and 88 (65 tokens).
inline bool q4_few(int out, int in, int M) {
    return M <= 32 || (double)M * out * in <= 3e9;
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
    int token_tiles, row_tiles;
};

inline q4_few_plan plan_q4_few(int out, int in, int M) {
    q4_few_plan p = {M <= 4, (in + 127) / 128 <= Q4_STAGED_GROUPS, M <= 16 ? 1 : 2, 1};
    const int64_t tiles = ((int64_t)out + 15) / 16;
    if (p.staged && !p.four)
        p.row_tiles = tiles <= 256 ? 1 : p.token_tiles == 1 && tiles > 512 && tiles <= 768 ? 3 : 2;
    return p;
}

// Offsets inside a tile are 32-bit and the tiles are numbered in 31 bits.
inline bool q4_tiled(int out, int in, int M) {
    return !q4_few(out, in, M) && in <= (1 << 23) && ((int64_t)out / 128 + 1) * ((int64_t)M / 64 + 1) < (1 << 24);
}

// Kinds of tiles (rows x tokens): 512 x 64, 256 x 64.
enum { Q4_512 = 0, Q4_256 = 1, Q4_KINDS = 2 };
constexpr int Q4_ROWS[Q4_KINDS] = {512, 256}, Q4_TOKENS[Q4_KINDS] = {64, 64};

struct q4_plan {
    int kind, slices;
};

inline q4_plan plan_q4(int out, int in, int M) {
    const int T = (in + 127) / 128;
    q4_plan best = {Q4_512, 1};
    float least = 0.0f;
    static constexpr float stage[Q4_KINDS] = {1.7f, 0.9f};
    for (int k = 0; k < Q4_KINDS; ++k) {
        const int64_t tiles = (((int64_t)out + Q4_ROWS[k] - 1) / Q4_ROWS[k]) *
                              (((int64_t)M + Q4_TOKENS[k] - 1) / Q4_TOKENS[k]);
        const int64_t at_once = 256 * (k == 0 ? 1 : 2);
        for (int S = 1; S <= 16 && 2 * S <= T + 1; ++S) {
            const float rounds = (float)((tiles * S + at_once - 1) / at_once);
            const int each = (T + S - 1) / S;
            const float share = std::min(1.0f, (float)(tiles * S) / (float)at_once);
            (void)share;
            float cost = rounds * ((float)each * stage[k] * (k == 0 ? 1.0f : 2.0f) + 2.5f);
            if (S > 1)
                cost += 3.0f + (float)(S + 1) * 4.0f * (float)M * (float)out / 5.0e6f;
            if (least == 0.0f || cost < least) {
                least = cost;
                best = {k, S};
            }
        }
    }
    return best;
}

}  // namespace rbq
