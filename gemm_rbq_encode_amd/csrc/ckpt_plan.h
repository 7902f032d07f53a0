// ckpt_plan.h -- which kernels, tiles and slices a backward pass from a
// checkpoint takes.  Host arithmetic only, so that a test can ask it without a
// GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace rbq {

constexpr int CW_BK = 64;        // tokens per stage of dW
constexpr int CX_BK = 64;        // rows of What per stage of dX
constexpr int CX_J = 128;        // columns of a dX tile

// How a call is split up.  Every choice is the least of a simple cost in us:
// rounds of workgroups over the compute units, each a start and end and its
// stages, and for slices a second launch and the write and read of the partial
// sums at 5 TB/s.
constexpr int CK_SPLITS[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
constexpr int CK_UNITS = 256;

struct ck_plan {
    int dx_slices;            // of dX's contraction
    int dw_large, dw_slices;  // dW's tiles (256 x 256, one workgroup per compute unit, or 128 x 128, two), slices of its tokens
    bool both;                // one launch of dX and large tiles of dW
};

inline float slice_cost(int S, int64_t n) { return S > 1 ? 4.0f + (float)n * (float)(2 * S + 1) * (4.0f / 5.0e6f) : 0.0f; }

inline int64_t ck_div(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Tokens per dX tile.
inline int dx_tokens(int M) { return M > 128 ? 256 : M > 64 ? 128 : M > 32 ? 64 : M > 16 ? 32 : 16; }

// dX: workgroups, and the time of one; stage times by tokens and planes.
inline int64_t dx_groups(int M, int in, int S) { return ck_div(in, CX_J) * ck_div(M, dx_tokens(M)) * S; }

inline float dx_time(int M, int out, int K, int S) {
    const int tm = dx_tokens(M);
    const float stage = tm <= 64 ? 0.8f : tm == 128 ? 1.4f : K > 2 ? 2.4f : 2.0f;
    return (float)ck_div(ck_div(out, CX_BK), S) * stage + (tm <= 64 ? 4.0f : 8.0f);
}

// dW: the same.
inline int64_t dw_groups(int out, int in, int large, int S) {
    const int edge = large ? 256 : 128;
    return ck_div(in, edge) * ck_div(out, edge) * S;
}

inline float dw_time(int M, int large, int S, bool two) {
    return (float)ck_div(ck_div(M, CW_BK), S) * (large ? 1.9f : two ? 1.6f : 1.1f) + (large ? 20.0f : two ? 14.0f : 10.0f);
}

// Each by itself.  Measured, dX (one slice and the choice): 16 tokens, 4096 x
// 4096: 48 and 16 us in 8; 1003 tokens, 5120 x 5120, K = 4: 191 and 158 us in 3
// (160 workgroups leave 96 compute units idle); 2048 tokens, 11008 x 4096: 339
// us in 1, 352 in 2.  dW with the scales' gradients: 2048 tokens, 11008 x 4096:
// 248 us large, 338 small; 300 tokens, 2000 x 2048: 33 large, 20 small; 2000
// tokens, 600 x 576: 38 us in one slice of 25 small tiles, 25 in 4.
//
// Both in one launch.  Up to 64 tokens, where dW is written in one stage: 16
// tokens, 4096 x 4096: 28.5 us with dX in 4 slices, 31.0 in 8; 4096 x 11008: 56
// in 2, 64 in 1, 67 in 8; so dX takes 176 of the 256 units.  More tokens: dW's
// workgroups fill the units that dX's leave, so that fewer slices do: 1003
// tokens, 5120 x 5120, K = 4: 231 us in 1 slice, 261 in 3 and two launches; 300
// tokens, 8192 x 4096, K = 3: 143 us, 151 in two launches; 955 tokens, 2896 x
// 1536, K = 1: 54 us in 3 slices, 86 in 1, 75 in two launches.  Over 17 such
// sizes the choice is the fastest or within 8 % of it.
inline ck_plan plan_backward(int M, int out, int in, int K, bool dx, bool dw) {
    ck_plan best = {1, 0, 1, false};
    const int64_t steps = ck_div(out, CX_BK), stages = ck_div(M, CW_BK);
    const bool few = M <= CW_BK;
    float dx_least = 0.0f, dw_least = 0.0f;
    for (const int S : CK_SPLITS) {
        if (!dx || (S > 1 && 2 * S > steps))
            break;
        const int room = few && dw ? 176 : CK_UNITS;
        const float cost = (float)ck_div(dx_groups(M, in, S), room) * dx_time(M, out, K, S) +
                           slice_cost(S, (int64_t)M * in);
        if (S == 1 || cost < dx_least) {
            best.dx_slices = S;
            dx_least = cost;
        }
    }
    if (few || !dw)
        return best;
    for (int large = 1; large >= 0; --large)
        for (const int S : CK_SPLITS) {
            if (S > 8 || (S > 1 && 2 * S > stages))
                break;
            const int64_t groups = dw_groups(out, in, large, S);
            const bool two = !large && groups > CK_UNITS;
            const float cost = (float)ck_div(groups, two ? 2 * CK_UNITS : CK_UNITS) * dw_time(M, large, S, two) +
                               slice_cost(S, (int64_t)out * in);
            if (dw_least == 0.0f || cost < dw_least) {
                best.dw_large = large;
                best.dw_slices = S;
                dw_least = cost;
            }
        }
    if (!dx)
        return best;
    float least = dx_least + dw_least + 3.0f;
    for (const int Sw : CK_SPLITS) {
        if (Sw > 8 || (Sw > 1 && 2 * Sw > stages))
            break;
        const float tw = dw_time(M, 1, Sw, false);
        const int64_t nw = dw_groups(out, in, 1, Sw);
        for (const int S : CK_SPLITS) {
            if (S > 1 && 2 * S > steps)
                break;
            // the units that dX's last round leaves begin with dW
            const float tx = dx_time(M, out, K, S);
            const int64_t nx = dx_groups(M, in, S), late = nx % CK_UNITS;
            float cost = (float)(nx / CK_UNITS) * tx;
            cost += late == 0 ? (float)ck_div(nw, CK_UNITS) * tw
                              : std::max(std::max(tx, tw), ((float)late * tx + (float)nw * tw) / CK_UNITS + 0.4f * tw);
            cost += slice_cost(S, (int64_t)M * in) + slice_cost(Sw, (int64_t)out * in);
            if (cost < least) {
                best = {S, 1, Sw, true};
                least = cost;
            }
        }
    }
    return best;
}

}  // namespace rbq
