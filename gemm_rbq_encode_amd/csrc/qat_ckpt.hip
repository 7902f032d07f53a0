// qat_ckpt.hip -- 8-bit activation checkpoints of the coupled forward, and
// the straight-through weight gradient that reads them.
//
// A checkpoint keeps the fp16 activations X [M][in] of one layer as int8
// codes with one fp16 scale per token and block of 128 columns.  For a block
// with A = max |x|:
//   s = A / 127 rounded up to fp16, at least 2^-24 and at most 515.5
//   c = nearest integer of x / s, ties to even, within +-127
// and the value a code stands for is x^ = fp16(c s): an fp16 number, so the
// backward is that of rbq_qat_backward with x^ in the place of X.  Rounding s
// up keeps |x| <= 127 s (nothing is cut off where s is subnormal and coarse);
// 2^-24 is the smallest fp16, for which the codes are exact; and 127 * 515.5
// is the largest maximum that fp16(c s) holds as a finite number.  A block
// with a NaN or infinite entry has scale NaN and codes 0, so x^ is NaN.
//
// c is the rounding of the exact quotient.  With q = fl(x fl(1/s)) and
// q' = fl(q + fl(x - q s) fl(1/s)), q' is the exact quotient wherever that is
// an fp32 number, ties among them, and elsewhere off by less than 2^-16; a
// quotient of two 11-bit significands in [0.25, 127] that is no tie is at
// least 2^-12 away from every half-integer.
#include <algorithm>
#include <type_traits>

#include "rbq.h"
#include "rbq_device.h"
#include "rbq_kernels.h"
#include "f8_device.h"
#include "ckpt_plan.h"

namespace rbq {

namespace {

constexpr int CK_THREADS = 256;

// fp16 bits of the scale of a block from the fp16 bits of its maximum.
__device__ __forceinline__ uint16_t ckpt_scale(uint32_t top) {
    if (top >= 0x7C00u)
        return (uint16_t)0x7E00u;
    const float A = h2f((uint16_t)top);
    uint16_t s = f2h(__fdiv_rn(A, 127.0f));
    if (h2f(s) * 127.0f < A)                  // 11 + 7 bits: the product is exact
        ++s;
    return std::min(std::max(s, (uint16_t)1), (uint16_t)0x6007u);   // 2^-24, 515.5
}

// Code of x for scale s (inv = fl(1 / s)), in the low byte.
__device__ __forceinline__ uint32_t ckpt_code(float x, float s, float inv) {
    float q = x * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, x), inv, q);
    q = fminf(fmaxf(q, -127.0f), 127.0f);
    return __float_as_uint(q + 12582912.0f) & 0xFFu;     // 1.5 * 2^23: the sum is rounded to an integer
}

// 16 lanes per block, as for the 8-bit floating point codes.  Bound by the read
// of X and the write of the codes.
template <int B>
__global__ __launch_bounds__(CK_THREADS) void qat_checkpoint_kernel(const uint16_t *__restrict__ X, int M, int in,
                                                                    int T, int8_t *__restrict__ codes,
                                                                    uint16_t *__restrict__ scales) {
    constexpr int ROWS = f8_rows(B);
    const int li = threadIdx.x & 15, sub = threadIdx.x >> 4;
    const int t0 = B == 1 ? (int)blockIdx.x * 16 + sub : (int)blockIdx.x * B;
    for (int64_t m = (int64_t)blockIdx.y * ROWS + (B == 1 ? 0 : sub); m < M; m += (int64_t)gridDim.y * ROWS) {
        const uint16_t *row = X + m * in;
        uint4 v[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int64_t c = (int64_t)(t0 + b) * F8_BLOCK + 8 * li;
            v[b] = c < in ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int64_t c = (int64_t)(t0 + b) * F8_BLOCK + 8 * li;
            const uint16_t sb = ckpt_scale(row16_max_u32(absmax8_f16(v[b])));
            const float s = h2f(sb), inv = __fdiv_rn(1.0f, s);
            const uint32_t u4[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
            uint32_t p[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t w0 = u4[2 * i], w1 = u4[2 * i + 1];
                p[i] = ckpt_code(h2f((uint16_t)w0), s, inv) | ckpt_code(h2f((uint16_t)(w0 >> 16)), s, inv) << 8 |
                       ckpt_code(h2f((uint16_t)w1), s, inv) << 16 |
                       ckpt_code(h2f((uint16_t)(w1 >> 16)), s, inv) << 24;
            }
            if (c < in)
                *reinterpret_cast<uint2 *>(codes + m * in + c) =
                    sb == 0x7E00u ? make_uint2(0u, 0u) : make_uint2(p[0], p[1]);
            if (li == 0 && t0 + b < T)
                scales[m * T + t0 + b] = sb;
        }
    }
}

// Two x^ from bytes (c0, c1) = bytes `sel` of `u` (codes with the sign bit
// flipped, c + 128): 0x6400 | (c + 128) is the fp16 number 1152 + c.
template <int HI>
__device__ __forceinline__ v2h ckpt_pair(uint32_t u, v2h s) {
    const uint32_t p = __builtin_amdgcn_perm(0x64646464u, u, HI ? 0x04030402u : 0x04010400u);
    return (__builtin_bit_cast(v2h, p) - (v2h){(_Float16)1152.0f, (_Float16)1152.0f}) * s;
}

// ---------------------------------------------------------------------------
// What both products below share.
//
// Operands pass through registers into LDS, two buffers deep: the loads of
// stage t + 2 (t + 3 for dX of up to 128 tokens) are issued, and the registers
// of stage t + 1 written to the other buffer, in pieces between the matrix
// instructions of stage t.  One barrier per stage.  Both operands of dW, and What of dX, lie with the
// contraction along the rows; the matrix instruction wants 8 consecutive
// contraction steps per lane, which ds_read_b64_tr_b16 gives: 16 lanes read
// four rows of 16 fp16 and lane i receives column i of the four.
//
// A row of LDS holds P pieces of 16 bytes, piece p of row k at position
// p ^ 2 f(k), f(k) = (bits 0, 1, 3, 4 of k) mod P / 2: the 16 rows of 32 bytes
// that one such read touches then lie in different banks.

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef v4u __attribute__((aligned(2))) v4u_a2;       // 16 bytes at any fp16
typedef v4u __attribute__((aligned(4))) v4u_a4;       // ... at any word
typedef double __attribute__((aligned(4))) f64_a4;

__device__ __forceinline__ int ck_swizzle(int k, int P) { return 2 * (((k & 3) | ((k >> 1) & 12)) & (P / 2 - 1)); }

// Eight contraction steps of one column: rows 4 h + .. of the lane's group.
__device__ __forceinline__ v8h ck_column(const unsigned char *p, int pitch) {
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * pitch));
    return __builtin_bit_cast(v8h, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Eight fp16 of a row of `n` from column c (any alignment), zero past its end
// and where `ok` is false.  Nothing outside the row is read.
__device__ __forceinline__ v4u ck_piece(const uint16_t *__restrict__ row, int64_t c, int64_t n, bool ok) {
    if (ok && c + 8 <= n)
        return *reinterpret_cast<const v4u_a2 *>(row + c);
    v4u v = {0u, 0u, 0u, 0u};
    if (ok && c < n)
        for (int i = 0; i < (int)(n - c); ++i)
            v[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
    return v;
}

__device__ __forceinline__ void ck_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---------------------------------------------------------------------------
// dW[r][j] = sum_m dY[m][r] x^[m][j] on v_mfma_f32_16x16x32_f16, 64 tokens per
// stage.  The codes are decoded to fp16 on their way into LDS.  Waves WM x WN,
// each 128 columns x 16 TN rows of dW; the columns are the side that a lane
// holds four of, so dW is written 16 bytes a lane.
//
// The gradients of the scales are sums of +-dW over groups of columns, in fp64
// as in qat.hip (entries of one size cancel): each wave adds its 128 columns
// from the registers it has just computed, which is a whole gradient where
// that is a group and all tokens, and else one fp64 value per row and plane of
// parts [slice][K][out][ceil(in / 128)], added in order at the end.
//
// Bound by the matrix instructions and their power: 2048 tokens, 11008 x 4096:
// 213 us, 866 TFLOP/s, and 240 with the scales' gradients (688 tiles are 2.7
// rounds of 256 compute units).  Their fp64 sums cost 1 to 3 % of a whole
// backward more than fp32 sums would (300 tokens, 8192 x 4096, K = 3: 134 us
// and 131), and up to 13 % of dW and the gradients alone (300 tokens, 11008 x
// 4096: 98 and 87).  LDS is not what counts: an order of its writes without
// bank conflicts (17 % of its cycles) takes the same time.

constexpr int CW_TM = 8;

// ONE: a single stage (up to 64 tokens): one buffer, and no staging between
// the products.  KP: planes whose sign words a lane holds.
template <int WM, int WN, int TN, bool ONE, int KP>
__device__ __forceinline__ void ck_dw(
    unsigned char *lds, int id, const uint16_t *__restrict__ dY, const int8_t *__restrict__ codes,
    const uint16_t *__restrict__ cscales, int M, int out, int in, int T, float *__restrict__ dW,
    const uint32_t *__restrict__ planes, int K, float *__restrict__ grads, f64_a4 *__restrict__ parts, int tiles_j,
    int tiles, int slices) {
    constexpr int THREADS = WM * WN * RBQ_WAVE;
    constexpr int CJ = WM * 128, CR = WN * TN * 16;            // tile: columns x rows of dW
    constexpr int PJ = CJ / 8, PR = CR / 8;                    // pieces of an LDS row
    constexpr int XB = CW_BK * CJ * 2, STAGE = XB + CW_BK * CR * 2;
    constexpr int NX = CW_BK * CJ / 16 / THREADS;              // 16 codes each
    constexpr int NY = CW_BK * PR / THREADS;                   // 8 values of dY each
    static_assert(NX * THREADS * 16 == CW_BK * CJ && NY * THREADS == CW_BK * PR, "staging covers the tile");
    static_assert(NX + NY <= CW_BK / 32 * CW_TM / 2, "every piece is staged within a stage");
    const int tid = threadIdx.x;
    const int lane = tid & (RBQ_WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / RBQ_WAVE);
    const int wj = wave % WM, wr = wave / WM;
    const int li = lane & 15, g = lane >> 4;
    const int tile = id % tiles, slice = id / tiles;
    const int64_t j0 = (int64_t)(tile % tiles_j) * CJ, r0 = (int64_t)(tile / tiles_j) * CR;
    dW += (int64_t)slice * out * in;

    v4f acc[CW_TM][TN];
#pragma unroll
    for (int i = 0; i < CW_TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

    // Whole stages load without a branch: columns past the last repeat column
    // 0 and rows past the last run on into the next token's (both end up in
    // elements of dW that do not exist).  The others, which that would take
    // past the end of dY, check every piece; tokens past the last are zero on
    // both sides.
    const int64_t steps = ((int64_t)M + CW_BK - 1) / CW_BK;
    const int64_t safe = ((int64_t)M * out - 7) / out / CW_BK;   // (below 1 where M out < 7 + out)
    v4u xr[NX], yr[NY];
    uint16_t xs[NX];
    uint32_t xoff[NX], soff[NX], yoff[NY];        // elements from the first of a stage
#pragma unroll
    for (int u = 0; u < NX; ++u) {
        const int c = u * THREADS + tid;
        const int64_t j = j0 + 16 * (c % (CJ / 16));
        const uint32_t jc = j < in ? (uint32_t)j : 0u;
        xoff[u] = (uint32_t)(c / (CJ / 16)) * (uint32_t)in + jc;
        soff[u] = (uint32_t)(c / (CJ / 16)) * (uint32_t)T + jc / F8_BLOCK;
    }
#pragma unroll
    for (int u = 0; u < NY; ++u) {
        const int c = u * THREADS + tid;
        const int64_t r = r0 + 8 * (c % PR);
        yoff[u] = (uint32_t)(c / PR) * (uint32_t)out + (r < out ? (uint32_t)r : 0u);
    }
    auto load_x = [&](int64_t t, int u, auto whole) {
        const int64_t m0 = t * CW_BK;
        const bool ok = decltype(whole)::value || m0 + (u * THREADS + tid) / (CJ / 16) < M;
        const int8_t *p = codes + m0 * in;
        const uint16_t *q = cscales + m0 * T;
        if (decltype(whole)::value || ok) {
            xr[u] = *reinterpret_cast<const v4u *>(p + xoff[u]);
            xs[u] = q[soff[u]];
        } else {
            xr[u] = (v4u){0u, 0u, 0u, 0u};
            xs[u] = 0;
        }
    };
    auto load_y = [&](int64_t t, int u, auto whole) {
        const uint16_t *p = dY + t * CW_BK * out;
        if constexpr (decltype(whole)::value) {
            yr[u] = *reinterpret_cast<const v4u_a2 *>(p + yoff[u]);
        } else {
            const int c = u * THREADS + tid;
            yr[u] = ck_piece(p + (int64_t)(c / PR) * out, r0 + 8 * (c % PR), out, t * CW_BK + c / PR < M);
        }
    };
    auto store_x = [&](unsigned char *at, int u) {
        const int c = u * THREADS + tid;
        const int k = c / (CJ / 16), p = 2 * (c % (CJ / 16));
        const _Float16 s1 = __builtin_bit_cast(_Float16, xs[u]);
        const v2h s = {s1, s1};
        v4u o[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = xr[u][i] ^ 0x80808080u;
            o[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, ckpt_pair<0>(w, s));
            o[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, ckpt_pair<1>(w, s));
        }
        unsigned char *q = at + k * (CJ * 2) + (p ^ ck_swizzle(k, PJ)) * 16;
        *reinterpret_cast<v4u *>(q) = o[0];
        *reinterpret_cast<v4u *>(q + 16) = o[1];
    };
    auto store_y = [&](unsigned char *at, int u) {
        const int c = u * THREADS + tid;
        const int k = c / PR, p = c % PR;
        *reinterpret_cast<v4u *>(at + XB + k * (CR * 2) + (p ^ ck_swizzle(k, PR)) * 16) = yr[u];
    };

    // this lane's place in the first four rows of its group, per tile of 16
    const int k0 = 8 * g + (li >> 2);
    uint32_t xo[CW_TM], yo[TN];
#pragma unroll
    for (int i = 0; i < CW_TM; ++i)
        xo[i] = k0 * (CJ * 2) + (((wj * CW_TM + i) * 2) ^ ck_swizzle(k0, PJ)) * 16 + 8 * (li & 3);
#pragma unroll
    for (int j = 0; j < TN; ++j)
        yo[j] = XB + k0 * (CR * 2) + (((wr * TN + j) * 2) ^ ck_swizzle(k0, PR)) * 16 + 8 * (li & 3);

    // stage t of this slice: its products, and between them, a piece after
    // every second row of tiles, stage t + 1 to LDS and stage t + 2 requested
    auto stage = [&](int64_t t, int64_t first, auto whole) {
        const unsigned char *cur = lds + ((t - first) & 1) * STAGE;
        unsigned char *nxt = lds + ((t - first + 1) & 1) * STAGE;
#pragma unroll
        for (int kk = 0; kk < CW_BK / 32; ++kk) {
            v8h a[2], b[TN];
            a[0] = ck_column(cur + xo[0] + kk * 32 * (CJ * 2), CJ * 2);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                b[j] = ck_column(cur + yo[j] + kk * 32 * (CR * 2), CR * 2);
#pragma unroll
            for (int i = 0; i < CW_TM; ++i) {
                if (i + 1 < CW_TM)
                    a[(i + 1) & 1] = ck_column(cur + xo[i + 1] + kk * 32 * (CJ * 2), CJ * 2);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i & 1], b[j], acc[i][j], 0, 0, 0);
                const int u = (kk * CW_TM + i) / 2;
                if (!ONE && (i & 1)) {
                    if (u < NX) {
                        store_x(nxt, u);
                        load_x(t + 2, u, whole);
                    } else if (u - NX < NY) {
                        store_y(nxt, u - NX);
                        load_y(t + 2, u - NX, whole);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (!ONE)
            ck_barrier();
    };
    // the sign words of this wave's columns, for the scales' gradients; they
    // arrive while dW is written
    const int64_t words = in >> 5, w0 = (j0 + wj * 128) >> 5;
    const bool add = (grads != nullptr || parts != nullptr) && w0 < words;
    v4u sign[KP][TN];
    auto load_signs = [&]() {
        if (!add)
            return;
#pragma unroll
        for (int k = 0; k < KP; ++k)
            if (k < K)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int64_t r = std::min<int64_t>(r0 + (wr * TN + j) * 16 + li, out - 1);
                    const uint32_t *p = planes + ((int64_t)k * out + r) * words + w0;
                    if (w0 + 4 <= words)
                        sign[k][j] = *reinterpret_cast<const v4u_a4 *>(p);
                    else
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            sign[k][j][q] = w0 + q < words ? p[q] : 0u;
                }
    };
    if constexpr (ONE) {
#pragma unroll
        for (int u = 0; u < NX; ++u)
            load_x(0, u, std::false_type());
#pragma unroll
        for (int u = 0; u < NY; ++u)
            load_y(0, u, std::false_type());
#pragma unroll
        for (int u = 0; u < NX; ++u)
            store_x(lds, u);
#pragma unroll
        for (int u = 0; u < NY; ++u)
            store_y(lds, u);
        load_signs();
        ck_barrier();
        stage(0, 0, std::false_type());
    } else {
        // (a slice's last stages request two past its end: checked, and unused)
        const int64_t t_lo = steps * slice / slices, t_hi = steps * (slice + 1) / slices;
#pragma unroll
        for (int u = 0; u < NX; ++u) {
            load_x(t_lo, u, std::false_type());
            store_x(lds, u);
            load_x(t_lo + 1, u, std::false_type());
        }
#pragma unroll
        for (int u = 0; u < NY; ++u) {
            load_y(t_lo, u, std::false_type());
            store_y(lds, u);
            load_y(t_lo + 1, u, std::false_type());
        }
        ck_barrier();
        int64_t t = t_lo;
        for (; t + 2 < std::min(t_hi, safe); ++t)
            stage(t, t_lo, std::true_type());
        for (; t < t_hi; ++t)
            stage(t, t_lo, std::false_type());
        load_signs();
    }

    // lane (li, g): columns 4 g + v of a column tile, row li of a row tile
    const bool vec = ((uintptr_t)dW & 15) == 0;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int64_t r = r0 + (wr * TN + j) * 16 + li;
        if (r >= out)
            continue;
#pragma unroll
        for (int i = 0; i < CW_TM; ++i) {
            const int64_t c = j0 + (wj * CW_TM + i) * 16 + 4 * g;
            float *p = dW + r * in + c;
            if (c < in) {
                if (vec) {
                    *reinterpret_cast<v4f *>(p) = acc[i][j];
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        p[v] = acc[i][j][v];
                }
            }
        }
    }
    if (!add)
        return;
    const int64_t at = (int64_t)slice * K * out * T + w0 / 4;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int64_t r = r0 + (wr * TN + j) * 16 + li;
        double s[KP];
#pragma unroll
        for (int k = 0; k < KP; ++k)
            s[k] = 0.0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (w0 + q >= words)                           // columns past the last
                break;
            // (a half at a time, for the registers)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                double d[4];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    d[v] = (double)acc[2 * q + h][j][v];
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    if (k >= K)
                        break;
                    const uint32_t w = ~sign[k][j][q] >> (4 * g);
#pragma unroll
                    for (int v = 0; v < 4; ++v)                // + d or - d: the high word of +-1.0
                        s[k] = __builtin_fma(
                            d[v], __hiloint2double((int)(((w << (31 - 16 * h - v)) & 0x80000000u) | 0x3FF00000u), 0), s[k]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            if (k >= K)
                break;
            double v = s[k];
            v += __shfl_xor(v, 16, RBQ_WAVE);
            v += __shfl_xor(v, 32, RBQ_WAVE);
            const int64_t o = at + ((int64_t)k * out + r) * T;
            if (g == 0 && r < out) {
                if (grads != nullptr)
                    grads[o] = (float)v;
                else
                    parts[o] = v;
            }
        }
    }
}

// (At least two waves per SIMD, here and below: no accumulation registers, out
// of which the sums would have to be copied.)
template <int WM, int WN, int TN>
__global__ __launch_bounds__(WM *WN *RBQ_WAVE, 2) void qat_ckpt_dw_kernel(
    const uint16_t *__restrict__ dY, const int8_t *__restrict__ codes, const uint16_t *__restrict__ cscales, int M,
    int out, int in, int T, float *__restrict__ dW, const uint32_t *__restrict__ planes, int K,
    float *__restrict__ grads, f64_a4 *__restrict__ parts, int tiles_j, int tiles, int slices) {
    extern __shared__ __align__(16) unsigned char lds[];
    ck_dw<WM, WN, TN, false, 4>(lds, xcd_run(blockIdx.x, tiles * slices), dY, codes, cscales, M, out, in, T, dW,
                                planes, K, grads, parts, tiles_j, tiles, slices);
}

// ---------------------------------------------------------------------------
// dX[m][j] = sum_r dY[m][r] What[r][j], What = sum_k a_k B_k formed in fp32 and
// split into two fp16 parts hi = fp16(w), lo = fp16(w - hi), as in qat.hip.
// Tiles of 64 TM tokens x 128 columns, 64 rows r per stage; waves 4 x 2.  A
// thread forms 16 columns of one row.  With one or two planes a row has four
// values, which a byte permute looks up from two 8-byte tables (hi and lo)
// two columns at a time; with three and four it has eight and their
// negatives, each worked out by one of the eight lanes of the row and passed
// round, in byte tables that are looked up four columns at a time (1003
// tokens, 5120 x 5120, K = 4: 145 us in 3 slices; with every sum formed by
// itself 25 more).  Bound by the matrix instructions: 2048 tokens, 11008 x 4096:
// 296 us, 1.25 PFLOP/s over both parts.

constexpr int CX_THREADS = 512;

__device__ __forceinline__ uint32_t ck_pack(_Float16 a, _Float16 b) {
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}

// Byte tables of four fp16 values v0, v1, -v1, -v0: low bytes and high bytes.
__device__ __forceinline__ void ck_table(_Float16 v0, _Float16 v1, uint32_t &lo, uint32_t &hi) {
    const uint32_t a = ck_pack(v0, v1), b = ck_pack(v1, v0) ^ 0x80008000u;
    lo = __builtin_amdgcn_perm(b, a, 0x06040200u);
    hi = __builtin_amdgcn_perm(b, a, 0x07050301u);
}

// The same byte tables of eight values, one from each of the 8 lanes that form
// a row (fj: the lane's place, v: fp16 hi | lo << 16): of the hi and of the lo
// parts, the low bytes t[0], t[1] of values 0 .. 3 and 4 .. 7, the high bytes
// t[2], t[3].  Three exchanges, each doubling what a lane holds.
__device__ __forceinline__ void ck_table8(uint32_t v, int fj, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    auto dpp = [](uint32_t x, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xF, 0xF, false);
    };
    constexpr std::integral_constant<int, 0xB1> by1;       // quad_perm 1 0 3 2
    constexpr std::integral_constant<int, 0x4E> by2;       // quad_perm 2 3 0 1
    constexpr std::integral_constant<int, 0x141> other4;   // row_half_mirror: a lane of the other four
    const uint32_t v1 = dpp(v, by1);
    // bytes L0 L1 H0 H1 of the even and the odd lane (perm: bytes 0 .. 3 are the second operand's)
    const bool b0 = fj & 1, b1 = fj & 2, b2 = fj & 4;
    const uint32_t h2 = __builtin_amdgcn_perm(v1, v, b0 ? 0x01050004u : 0x05010400u);
    const uint32_t l2 = __builtin_amdgcn_perm(v1, v, b0 ? 0x03070206u : 0x07030602u);
    const uint32_t h3 = dpp(h2, by2), l3 = dpp(l2, by2);
    const uint32_t sl = b1 ? 0x01000504u : 0x05040100u, sh = b1 ? 0x03020706u : 0x07060302u;
    const uint32_t own[4] = {__builtin_amdgcn_perm(h3, h2, sl), __builtin_amdgcn_perm(h3, h2, sh),
                             __builtin_amdgcn_perm(l3, l2, sl), __builtin_amdgcn_perm(l3, l2, sh)};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t o = dpp(own[q], other4);
        uint32_t *t = (q < 2 ? hi : lo) + 2 * (q & 1);
        t[0] = b2 ? o : own[q];
        t[1] = b2 ? own[q] : o;
    }
}

// The four nibbles of a 16-bit number, one to a byte.
__device__ __forceinline__ uint32_t ck_nibbles(uint32_t x) {
    const uint32_t z = __builtin_amdgcn_perm(0u, x, 0x0C010C00u);       // bytes 0 and 1 to 0 and 2
    return (z & 0x000F000Fu) | ((z << 4) & 0x0F000F00u);
}

template <int WM, int TM, int K>
__device__ __forceinline__ void ck_dx(
    unsigned char *lds, int id, const uint16_t *__restrict__ dY, const uint32_t *__restrict__ planes,
    const uint16_t *__restrict__ scales, int M, int out, int in, int group_size, int64_t r_slice,
    float *__restrict__ dX, int32_t *__restrict__ status, int tiles_j, int tiles_m) {
    constexpr int WJ = CX_THREADS / RBQ_WAVE / WM, TJ = CX_J / 16 / WJ;   // waves and their tiles along the columns
    constexpr int CM = 16 * WM * TM;
    constexpr int YB = CM * CX_BK * 2, HB = CX_BK * CX_J * 2, STAGE = YB + 2 * HB;
    constexpr int YP = CM * (CX_BK / 8), NY = (YP + CX_THREADS - 1) / CX_THREADS;   // 8 values of dY each
    constexpr int PJ = CX_J / 8;
    // stages whose loads are in flight: the short stages of few tokens need two
    constexpr int SETS = CM == 256 ? 1 : 2;
    const int tid = threadIdx.x;
    const int lane = tid & (RBQ_WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / RBQ_WAVE);
    const int wm = wave % WM, wj = wave / WM;
    const int li = lane & 15, g = lane >> 4;
    const int z = id / (tiles_j * tiles_m);
    const int64_t j0 = (int64_t)(id % tiles_j) * CX_J, m0 = (int64_t)(id / tiles_j % tiles_m) * CM;
    const int64_t words = in >> 5;
    const int G = group_size ? in / group_size : 1;
    const int64_t r_lo = z * r_slice, r_hi = std::min<int64_t>(out, r_lo + r_slice);
    dX += (int64_t)z * M * in;

    v4f acc[TJ][TM];
#pragma unroll
    for (int i = 0; i < TJ; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

    // staging: 8 pieces per token row, piece p of token m at p ^ (m & 7).
    // Stages that lie whole in the slice load without a branch (tokens and
    // columns past the last repeat the last: they end up in elements of dX
    // that do not exist); the last one checks, zero past the end on both sides.
    v4u yr[SETS][NY];
    const uint16_t *yrow[NY];
#pragma unroll
    for (int u = 0; u < NY; ++u) {
        const int c = u * CX_THREADS + tid;
        yrow[u] = dY + std::min<int64_t>(m0 + (c >> 3), M - 1) * out + 8 * (c & 7);
    }
    auto load_y = [&](int64_t rb, int u, auto whole, int set) {
        const int c = u * CX_THREADS + tid;
        if constexpr (decltype(whole)::value)
            yr[set][u] = *reinterpret_cast<const v4u_a2 *>(yrow[u] + rb);
        else
            yr[set][u] = ck_piece(dY + (m0 + (c >> 3)) * out, rb + 8 * (c & 7), r_hi, m0 + (c >> 3) < M);
    };
    auto store_y = [&](unsigned char *at, int u, int set) {
        const int c = u * CX_THREADS + tid;
        const int m = c >> 3, p = c & 7;
        if (c < YP)
            *reinterpret_cast<v4u *>(at + m * (CX_BK * 2) + (p ^ (m & 7)) * 16) = yr[set][u];
    };
    const int fr = tid >> 3, fj = tid & 7;                     // this thread's row of What and 16 columns
    const int64_t fw = std::min((j0 >> 5) + (fj >> 1), words - 1);
    const int64_t fg = group_size ? j0 / group_size : 0;       // 128 columns lie in one group
    uint32_t bits[SETS][K];
    uint16_t sc[SETS][K];
    bool valid[SETS] = {}, ovf = false;
    const uint32_t woff = (uint32_t)fr * (uint32_t)words + (uint32_t)fw, goff = (uint32_t)fr * (uint32_t)G + (uint32_t)fg;
    const int sh = 16 * (fj & 1);
    auto load_w = [&](int64_t rb, auto whole, int set) {
        valid[set] = decltype(whole)::value || rb + fr < r_hi;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t *p = planes + ((int64_t)k * out + rb) * words;
            const uint16_t *q = scales + ((int64_t)k * out + rb) * G;
            if (decltype(whole)::value || valid[set]) {
                bits[set][k] = p[woff] >> sh;
                sc[set][k] = q[goff];
            } else {
                bits[set][k] = 0u;
                sc[set][k] = 0;
            }
        }
    };
    uint32_t hv[8], lv[8];
    // part q = 0 .. 3 of forming: 4 columns; what is common to the row comes with part 0
    uint32_t hl = 0, hh = 0, ll = 0, lh = 0, even = 0, odd = 0;        // K <= 2
    uint32_t ht[4], lt[4], nib[K], hp[2], lp[2];                       // K >= 3
    float a[K];
    auto form = [&](int q, int set) {
        if (q == 0) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                a[k] = h2f(sc[set][k]);
                sum += __builtin_fabsf(a[k]);
            }
            // no weight of the row is beyond the sum of its scales: only
            // where that is beyond fp16 are the weights looked at
            if (valid[set] && !(sum < 65520.0f))
                for (int c = 0; c < 16; ++c) {
                    float w = 0.0f;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        w += (bits[set][k] >> c) & 1u ? a[k] : -a[k];
                    ovf = ovf || !(__builtin_fabsf(w) < 65520.0f);
                }
            if constexpr (K <= 2) {
                // index b0 + 2 b1: -a0 - a1, a0 - a1, a1 - a0, a0 + a1 (K = 1: only the first two, b1 = 0)
                const uint32_t b0 = bits[set][0], b1 = K > 1 ? bits[set][K - 1] : 0u;
                const float a1 = K > 1 ? a[K - 1] : 0.0f, w0 = -a[0] - a1, w1 = a[0] - a1;
                const _Float16 h0 = (_Float16)w0, h1 = (_Float16)w1;
                ck_table(h0, h1, hl, hh);
                ck_table((_Float16)(w0 - (float)h0), (_Float16)(w1 - (float)h1), ll, lh);
                even = (b0 & 0x5555u) | ((b1 & 0x5555u) << 1);
                odd = ((b0 >> 1) & 0x5555u) | (b1 & 0xAAAAu);
            } else {
                // the values with the last plane's bit set (the others are
                // their negatives), by the bits that differ from it
                float w = fj & 1 ? -a[0] : a[0];
#pragma unroll
                for (int k = 1; k + 1 < K; ++k)
                    w += fj >> k & 1 ? -a[k] : a[k];
                w += a[K - 1];
                const _Float16 h = (_Float16)w;
                ck_table8(ck_pack(h, (_Float16)(w - (float)h)), fj, ht, lt);
#pragma unroll
                for (int k = 0; k < K; ++k)
                    nib[k] = ck_nibbles(k + 1 < K ? bits[set][k] ^ bits[set][K - 1] : ~bits[set][k]);
            }
        }
        if constexpr (K <= 2) {
#pragma unroll
            for (int p = 2 * q; p < 2 * q + 2; ++p) {
                const uint32_t i = ((even >> (2 * p)) & 3u) | ((odd >> (2 * p)) & 3u) << 16;
                const uint32_t sel = i * 0x101u + 0x04000400u;
                hv[p] = __builtin_amdgcn_perm(hh, hl, sel);
                lv[p] = __builtin_amdgcn_perm(lh, ll, sel);
            }
        } else {
            // columns q, q + 4, q + 8, q + 12: a byte of the index each
            uint32_t sel = (nib[0] >> q) & 0x01010101u;
#pragma unroll
            for (int k = 1; k + 1 < K; ++k)
                sel |= ((nib[k] >> q) & 0x01010101u) << k;
            const uint32_t sign = ((nib[K - 1] >> q) & 0x01010101u) << 7;
            const uint32_t h0 = __builtin_amdgcn_perm(ht[1], ht[0], sel);
            const uint32_t h1 = __builtin_amdgcn_perm(ht[3], ht[2], sel) ^ sign;
            const uint32_t l0 = __builtin_amdgcn_perm(lt[1], lt[0], sel);
            const uint32_t l1 = __builtin_amdgcn_perm(lt[3], lt[2], sel) ^ sign;
            // columns q and q + 4, q + 8 and q + 12; with those of the column before, the pairs
            const uint32_t ha = __builtin_amdgcn_perm(h1, h0, 0x05010400u), hb = __builtin_amdgcn_perm(h1, h0, 0x07030602u);
            const uint32_t la = __builtin_amdgcn_perm(l1, l0, 0x05010400u), lb = __builtin_amdgcn_perm(l1, l0, 0x07030602u);
            if (q & 1) {
                const int p = q >> 1;
                hv[p] = __builtin_amdgcn_perm(ha, hp[0], 0x05040100u);
                hv[p + 2] = __builtin_amdgcn_perm(ha, hp[0], 0x07060302u);
                hv[p + 4] = __builtin_amdgcn_perm(hb, hp[1], 0x05040100u);
                hv[p + 6] = __builtin_amdgcn_perm(hb, hp[1], 0x07060302u);
                lv[p] = __builtin_amdgcn_perm(la, lp[0], 0x05040100u);
                lv[p + 2] = __builtin_amdgcn_perm(la, lp[0], 0x07060302u);
                lv[p + 4] = __builtin_amdgcn_perm(lb, lp[1], 0x05040100u);
                lv[p + 6] = __builtin_amdgcn_perm(lb, lp[1], 0x07060302u);
            } else {
                hp[0] = ha;
                hp[1] = hb;
                lp[0] = la;
                lp[1] = lb;
            }
        }
    };
    auto store_w = [&](unsigned char *at) {
        unsigned char *q = at + YB + fr * (CX_J * 2) + ((2 * fj) ^ ck_swizzle(fr, PJ)) * 16;
        *reinterpret_cast<v4u *>(q) = (v4u){hv[0], hv[1], hv[2], hv[3]};
        *reinterpret_cast<v4u *>(q + 16) = (v4u){hv[4], hv[5], hv[6], hv[7]};
        *reinterpret_cast<v4u *>(q + HB) = (v4u){lv[0], lv[1], lv[2], lv[3]};
        *reinterpret_cast<v4u *>(q + HB + 16) = (v4u){lv[4], lv[5], lv[6], lv[7]};
    };

    const int k0 = 8 * g + (li >> 2);
    uint32_t wo[TJ], yo[2];
#pragma unroll
    for (int i = 0; i < TJ; ++i)
        wo[i] = YB + k0 * (CX_J * 2) + (((wj * TJ + i) * 2) ^ ck_swizzle(k0, PJ)) * 16 + 8 * (li & 3);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
        yo[kk] = (wm * TM * 16 + li) * (CX_BK * 2) + ((4 * kk + g) ^ (li & 7)) * 16;

    // the stage at row r of What: its products, and between them, a piece after
    // every row of tiles, the next stage (from register set `next`) to LDS and
    // the one SETS behind it requested
    auto stage = [&](int64_t r, auto whole, auto next) {
        constexpr int set = decltype(next)::value;
        const int64_t t = (r - r_lo) / CX_BK, ahead = r + (1 + SETS) * CX_BK;
        const unsigned char *cur = lds + (t & 1) * STAGE;
        unsigned char *nxt = lds + ((t + 1) & 1) * STAGE;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            v8h b[TM], al[2], ah[2];
            al[0] = ck_column(cur + wo[0] + HB + kk * 32 * (CX_J * 2), CX_J * 2);
#pragma unroll
            for (int j = 0; j < TM; ++j)
                b[j] = *reinterpret_cast<const v8h *>(cur + yo[kk] + j * 16 * (CX_BK * 2));
            ah[0] = ck_column(cur + wo[0] + kk * 32 * (CX_J * 2), CX_J * 2);
#pragma unroll
            for (int i = 0; i < TJ; ++i) {
                if (i + 1 < TJ) {
                    al[(i + 1) & 1] = ck_column(cur + wo[i + 1] + HB + kk * 32 * (CX_J * 2), CX_J * 2);
                    ah[(i + 1) & 1] = ck_column(cur + wo[i + 1] + kk * 32 * (CX_J * 2), CX_J * 2);
                }
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(al[i & 1], b[j], acc[i][j], 0, 0, 0);
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ah[i & 1], b[j], acc[i][j], 0, 0, 0);
                // (8 places for the pieces)
#pragma unroll
                for (int u = (kk * TJ + i) * 4 / TJ; u < (kk * TJ + i + 1) * 4 / TJ; ++u) {
                    if (u < 4)
                        form(u, set);
                    if (u == 4) {
                        store_w(nxt);
                        load_w(ahead, whole, set);
                    }
                    if (u >= 4 && u - 4 < NY) {
                        store_y(nxt, u - 4, set);
                        load_y(ahead, u - 4, whole, set);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        static_assert(NY <= 4, "every piece is staged within a stage");
        ck_barrier();
    };
    constexpr std::integral_constant<int, 0> set0;
    constexpr std::integral_constant<int, SETS - 1> set1;     // of odd stages
    load_w(r_lo, std::false_type(), 0);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        form(q, 0);
    store_w(lds);
#pragma unroll
    for (int u = 0; u < NY; ++u) {
        load_y(r_lo, u, std::false_type(), 0);
        store_y(lds, u, 0);
    }
#pragma unroll
    for (int d = 1; d <= SETS; ++d) {
        load_w(r_lo + d * CX_BK, std::false_type(), d % SETS);
#pragma unroll
        for (int u = 0; u < NY; ++u)
            load_y(r_lo + d * CX_BK, u, std::false_type(), d % SETS);
    }
    ck_barrier();
    int64_t r = r_lo;
    for (; r + (3 + SETS) * CX_BK <= r_hi; r += 2 * CX_BK) {
        stage(r, std::true_type(), set1);
        stage(r + CX_BK, std::true_type(), set0);
    }
    for (; r < r_hi; r += CX_BK) {
        stage(r, std::false_type(), set1);
        r += CX_BK;
        if (r < r_hi)
            stage(r, std::false_type(), set0);
    }

    const bool vec = ((uintptr_t)dX & 15) == 0;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int64_t m = m0 + (wm * TM + j) * 16 + li;
        if (m >= M)
            continue;
#pragma unroll
        for (int i = 0; i < TJ; ++i) {
            const int64_t c = j0 + (wj * TJ + i) * 16 + 4 * g;
            float *p = dX + m * in + c;
            if (c < in) {
                if (vec) {
                    *reinterpret_cast<v4f *>(p) = acc[i][j];
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        p[v] = acc[i][j][v];
                }
            }
        }
    }
    if (status != nullptr && __ballot(ovf) != 0 && lane == 0)
        atomicOr(status, (int)RBQ_STATUS_SCALE_OVERFLOW);
}

template <int WM, int TM, int K>
__global__ __launch_bounds__(CX_THREADS, 2) void qat_ckpt_dx_kernel(
    const uint16_t *__restrict__ dY, const uint32_t *__restrict__ planes, const uint16_t *__restrict__ scales, int M,
    int out, int in, int group_size, int64_t r_slice, float *__restrict__ dX, int32_t *__restrict__ status,
    int tiles_j, int tiles_m, int total) {
    extern __shared__ __align__(16) unsigned char lds[];
    ck_dx<WM, TM, K>(lds, xcd_run(blockIdx.x, total), dY, planes, scales, M, out, in, group_size, r_slice, dX,
                     status, tiles_j, tiles_m);
}

// Large tiles of both in one launch, one workgroup to a compute unit: dW's
// begin on the units that dX's last round leaves free.
template <int TM, int K>
__global__ __launch_bounds__(CX_THREADS, 2) void qat_ckpt_both_kernel(
    const uint16_t *__restrict__ dY, const uint32_t *__restrict__ planes, const uint16_t *__restrict__ scales, int M,
    int out, int in, int group_size, int64_t r_slice, float *__restrict__ dX, int32_t *__restrict__ status,
    int x_tiles_j, int x_tiles_m, int x_total, const int8_t *__restrict__ codes, const uint16_t *__restrict__ cscales,
    int T, float *__restrict__ dW, float *__restrict__ grads, f64_a4 *__restrict__ parts, int w_tiles_j, int w_tiles,
    int w_slices) {
    extern __shared__ __align__(16) unsigned char lds[];
    if ((int)blockIdx.x < x_total)
        ck_dx<4, TM, K>(lds, xcd_run(blockIdx.x, x_total), dY, planes, scales, M, out, in, group_size, r_slice, dX,
                       status, x_tiles_j, x_tiles_m);
    else
        ck_dw<2, 4, 4, false, 4>(lds, xcd_run(blockIdx.x - x_total, w_tiles * w_slices), dY, codes, cscales, M, out,
                                 in, T, dW, planes, K, grads, parts, w_tiles_j, w_tiles, w_slices);
}

// Up to 64 tokens: both in one launch, two workgroups to a compute unit.  The
// write of dW bounds one, the start of every stage the other, so they go well
// beside each other; either may have no workgroups.  dX: the waves lie along
// the columns, so that each weight is read from LDS by one wave only.  16
// tokens, 4096 x 4096: 28 us for all three outputs (one after the other: 37),
// against 14.4 for dW alone.
template <int TM, int K>
__global__ __launch_bounds__(CX_THREADS, 4) void qat_ckpt_few_kernel(
    const uint16_t *__restrict__ dY, const uint32_t *__restrict__ planes, const uint16_t *__restrict__ scales, int M,
    int out, int in, int group_size, int64_t r_slice, float *__restrict__ dX, int32_t *__restrict__ status,
    int x_tiles, int x_total, const int8_t *__restrict__ codes, const uint16_t *__restrict__ cscales, int T,
    float *__restrict__ dW, float *__restrict__ grads, f64_a4 *__restrict__ parts, int w_tiles_j, int w_tiles) {
    extern __shared__ __align__(16) unsigned char lds[];
    if ((int)blockIdx.x < x_total)
        ck_dx<1, TM, K>(lds, xcd_run(blockIdx.x, x_total), dY, planes, scales, M, out, in, group_size, r_slice, dX,
                        status, x_tiles, 1);
    else
        ck_dw<1, 8, 2, true, K>(lds, xcd_run(blockIdx.x - x_total, w_tiles), dY, codes, cscales, M, out, in, T, dW,
                                planes, K, grads, parts, w_tiles_j, w_tiles, 1);
}

// What is left to add at the end, in one launch: up to three jobs, each with a
// share of the workgroups.  A job sums, for each of n outputs, `slices` fp32
// values in order (slices of dW or dX; parts = 0), or `slices` groups of
// `parts` consecutive fp64 values in a fixed order (the scales' gradients): by
// one thread where a group is one value, else by one wave.
struct ck_job {
    const void *from;
    float *to;
    int64_t n;
    int slices, parts;
    unsigned blocks;
};

struct ck_jobs {
    ck_job job[3];
};

__global__ __launch_bounds__(CK_THREADS) void qat_ckpt_join_kernel(ck_jobs jobs) {
    unsigned b = blockIdx.x;
    int q = 0;
    while (q < 2 && b >= jobs.job[q].blocks)
        b -= jobs.job[q++].blocks;
    const ck_job &o = jobs.job[q];
    const int64_t first = (int64_t)b * CK_THREADS + threadIdx.x, stride = (int64_t)o.blocks * CK_THREADS;
    if (o.parts == 0) {
        const float *from = static_cast<const float *>(o.from);
        for (int64_t i = first; i < o.n; i += stride) {
            float v = from[i];
            for (int z = 1; z < o.slices; ++z)
                v += from[z * o.n + i];
            o.to[i] = v;
        }
        return;
    }
    const f64_a4 *from = static_cast<const f64_a4 *>(o.from);
    if (o.parts == 1) {
        for (int64_t i = first; i < o.n; i += stride) {
            double v = from[i];
            for (int z = 1; z < o.slices; ++z)
                v += from[z * o.n + i];
            o.to[i] = (float)v;
        }
        return;
    }
    const int lane = threadIdx.x & (RBQ_WAVE - 1);
    constexpr int WAVES = CK_THREADS / RBQ_WAVE;
    for (int64_t i = (int64_t)b * WAVES + threadIdx.x / RBQ_WAVE; i < o.n; i += (int64_t)o.blocks * WAVES) {
        double s = 0.0;
        for (int z = 0; z < o.slices; ++z)
            for (int t = lane; t < o.parts; t += RBQ_WAVE)
                s += from[(z * o.n + i) * o.parts + t];
        s = wave_sum_f64(s);
        if (lane == 0)
            o.to[i] = (float)s;
    }
}

constexpr int LDS_MAX = 160 * 1024;

// The calls' arguments and where their partial sums go.
struct ck_call {
    const uint16_t *dY;
    const uint32_t *planes;
    const uint16_t *scales;
    const int8_t *codes;
    const uint16_t *cscales;
    int M, out, in, K, group_size;
    float *dX, *dW;                        // the results, or slices of them
    float *grads;                          // the scales' gradients, or null and
    f64_a4 *parts;                         // parts of them, or null
    int dx_slices, dw_slices;
    int32_t *status;
    hipStream_t st;
};

constexpr int64_t CK_GRID = 0x7FFFFFFF / CX_THREADS;

// Rows of What per slice of dX's contraction.
int64_t dx_rows(const ck_call &c) {
    return (((int64_t)c.out + c.dx_slices - 1) / c.dx_slices + CX_BK - 1) / CX_BK * CX_BK;
}

template <int WM, int WN, int TN>
hipError_t launch_dw(const ck_call &c) {
    constexpr int CJ = WM * 128, CR = WN * TN * 16;
    constexpr int LDS = 2 * CW_BK * (CJ + CR) * 2;
    static_assert(LDS <= LDS_MAX, "LDS of a compute unit");
    const int64_t tiles_j = ((int64_t)c.in + CJ - 1) / CJ, tiles = tiles_j * (((int64_t)c.out + CR - 1) / CR);
    if (tiles * c.dw_slices > CK_GRID)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((qat_ckpt_dw_kernel<WM, WN, TN>), dim3((unsigned)(tiles * c.dw_slices)),
                       dim3(WM * WN * RBQ_WAVE), LDS, c.st, c.dY, c.codes, c.cscales, c.M, c.out, c.in,
                       f8_blocks(c.in), c.dW, c.planes, c.K, c.grads, c.parts, (int)tiles_j, (int)tiles, c.dw_slices);
    return hipGetLastError();
}

template <int WM, int TM>
hipError_t launch_dx(const ck_call &c) {
    constexpr int CM = 16 * WM * TM, LDS = 2 * (CM * CX_BK * 2 + 2 * CX_BK * CX_J * 2);
    static_assert(LDS <= LDS_MAX, "LDS of a compute unit");
    const int64_t tiles_j = ((int64_t)c.in + CX_J - 1) / CX_J, tiles_m = ((int64_t)c.M + CM - 1) / CM;
    const int64_t total = tiles_j * tiles_m * c.dx_slices;
    if (total > CK_GRID)
        return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)total), dim3(CX_THREADS), LDS, c.st, c.dY, c.planes, c.scales, c.M,
                           c.out, c.in, c.group_size, dx_rows(c), c.dX, c.status, (int)tiles_j, (int)tiles_m,
                           (int)total);
    };
    switch (c.K) {
    case 1: go(qat_ckpt_dx_kernel<WM, TM, 1>); break;
    case 2: go(qat_ckpt_dx_kernel<WM, TM, 2>); break;
    case 3: go(qat_ckpt_dx_kernel<WM, TM, 3>); break;
    default: go(qat_ckpt_dx_kernel<WM, TM, 4>); break;
    }
    return hipGetLastError();
}

template <int TM>
hipError_t launch_both(const ck_call &c) {
    constexpr int CM = 64 * TM, LDS = 2 * CW_BK * (256 + 256) * 2;
    static_assert(LDS >= 2 * (CM * CX_BK * 2 + 2 * CX_BK * CX_J * 2) && LDS <= LDS_MAX, "LDS of a compute unit");
    const int64_t x_tiles_j = ((int64_t)c.in + CX_J - 1) / CX_J, x_tiles_m = ((int64_t)c.M + CM - 1) / CM;
    const int64_t w_tiles_j = ((int64_t)c.in + 255) / 256, w_tiles = w_tiles_j * (((int64_t)c.out + 255) / 256);
    const int64_t x_total = x_tiles_j * x_tiles_m * c.dx_slices, total = x_total + w_tiles * c.dw_slices;
    if (total > CK_GRID)
        return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)total), dim3(CX_THREADS), LDS, c.st, c.dY, c.planes, c.scales, c.M,
                           c.out, c.in, c.group_size, dx_rows(c), c.dX, c.status, (int)x_tiles_j, (int)x_tiles_m,
                           (int)x_total, c.codes, c.cscales, f8_blocks(c.in), c.dW, c.grads, c.parts, (int)w_tiles_j,
                           (int)w_tiles, c.dw_slices);
    };
    switch (c.K) {
    case 1: go(qat_ckpt_both_kernel<TM, 1>); break;
    case 2: go(qat_ckpt_both_kernel<TM, 2>); break;
    case 3: go(qat_ckpt_both_kernel<TM, 3>); break;
    default: go(qat_ckpt_both_kernel<TM, 4>); break;
    }
    return hipGetLastError();
}

// Either of dX and dW may be null.
template <int TM>
hipError_t launch_few(const ck_call &c) {
    constexpr int LDS_X = 2 * (16 * TM * CX_BK * 2 + 2 * CX_BK * CX_J * 2), LDS_W = CW_BK * (128 + 256) * 2;
    constexpr int LDS = LDS_X > LDS_W ? LDS_X : LDS_W;
    static_assert(2 * LDS <= LDS_MAX, "LDS of a compute unit");
    const int64_t tiles_j = ((int64_t)c.in + 127) / 128;
    const int64_t x_total = c.dX != nullptr ? tiles_j * c.dx_slices : 0;
    const int64_t w_tiles = c.dW != nullptr ? tiles_j * (((int64_t)c.out + 255) / 256) : 0;
    if (x_total + w_tiles > CK_GRID)
        return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(x_total + w_tiles)), dim3(CX_THREADS), LDS, c.st, c.dY, c.planes,
                           c.scales, c.M, c.out, c.in, c.group_size, dx_rows(c), c.dX, c.status, (int)tiles_j,
                           (int)x_total, c.codes, c.cscales, f8_blocks(c.in), c.dW, c.grads, c.parts, (int)tiles_j,
                           (int)w_tiles);
    };
    switch (c.K) {
    case 1: go(qat_ckpt_few_kernel<TM, 1>); break;
    case 2: go(qat_ckpt_few_kernel<TM, 2>); break;
    case 3: go(qat_ckpt_few_kernel<TM, 3>); break;
    default: go(qat_ckpt_few_kernel<TM, 4>); break;
    }
    return hipGetLastError();
}

// Partial sums of dW's slices, the parts of the scales' gradients, and dX's
// slices, one after another.
size_t dw_slice_bytes(const ck_plan &p, int out, int in) {
    return p.dw_slices > 1 ? (size_t)p.dw_slices * (size_t)out * (size_t)in * sizeof(float) : 0;
}

size_t dw_part_bytes(const ck_plan &p, int out, int in, int K, int group_size) {
    return p.dw_slices == 1 && (group_size || in <= F8_BLOCK)
               ? 0 : (size_t)p.dw_slices * (size_t)K * (size_t)out * (size_t)f8_blocks(in) * sizeof(double);
}

size_t dx_slice_bytes(const ck_plan &p, int M, int in) {
    return p.dx_slices > 1 ? (size_t)p.dx_slices * (size_t)M * (size_t)in * sizeof(float) : 0;
}

ck_job sum_job(const void *from, float *to, int64_t n, int slices, int parts) {
    const int64_t blocks = parts <= 1 ? (n + CK_THREADS - 1) / CK_THREADS : (n + 3) / 4;
    return {from, to, n, slices, parts, (unsigned)std::min<int64_t>(blocks, 1 << 18)};
}

}  // namespace

hipError_t launch_qat_checkpoint(const uint16_t *X, int M, int in, int8_t *codes, uint16_t *scales,
                                 hipStream_t st) {
    // 16 x 4096: 2.1 us with one block a lane, 3.0 with four; 4096 x 11008: 22.1
    // and 24.3; 30000 x 1024 (8 blocks in a row): 19.7 and 16.7
    const int T = f8_blocks(in);
    if (f8_spread(M, T, INT64_MAX))
        hipLaunchKernelGGL(qat_checkpoint_kernel<1>, f8_token_grid(M, T, 1), dim3(CK_THREADS), 0, st, X, M, in, T,
                           codes, scales);
    else
        hipLaunchKernelGGL(qat_checkpoint_kernel<4>, f8_token_grid(M, T, 4), dim3(CK_THREADS), 0, st, X, M, in, T,
                           codes, scales);
    return hipGetLastError();
}

// Enough for any of the outputs.
size_t qat_backward_ckpt_workspace_bytes(int M, int out, int in, int K, int group_size) {
    size_t most = 0;
    for (int ask = 1; ask < 4; ++ask) {
        const ck_plan p = plan_backward(M, out, in, K, ask & 1, ask & 2);
        size_t n = ask & 1 ? dx_slice_bytes(p, M, in) : 0;
        if (ask & 2)
            n += dw_slice_bytes(p, out, in) + dw_part_bytes(p, out, in, K, group_size);
        most = std::max(most, n);
    }
    return most;
}

hipError_t launch_qat_backward_ckpt(const uint32_t *planes, const uint16_t *scales, int out, int in, int K,
                                    int group_size, const int8_t *x_codes, const uint16_t *x_scales,
                                    const uint16_t *dY, int M, float *dX, float *dW, float *dscales,
                                    void *workspace, size_t ws_bytes, int32_t *status, hipStream_t st) {
    // With less than the whole workspace nothing is sliced, and the scales'
    // gradients that would pass through it are taken from dW in a pass of
    // their own.
    const bool fits = ws_bytes >= qat_backward_ckpt_workspace_bytes(M, out, in, K, group_size);
    ck_plan p = plan_backward(M, out, in, K, dX != nullptr, dW != nullptr);
    const size_t part_bytes = dw_part_bytes(p, out, in, K, group_size);
    if (!fits)
        p.dx_slices = p.dw_slices = 1;
    float *ws = static_cast<float *>(workspace);
    ck_jobs left = {};
    int jobs = 0;
    ck_call c = {dY, planes, scales, x_codes, x_scales, M, out, in, K, group_size, dX, dW, nullptr, nullptr,
                 p.dx_slices, p.dw_slices, status, st};
    c.dx_slices = (int)((out + dx_rows(c) - 1) / dx_rows(c));        // (none of them empty)
    if (dW != nullptr && c.dw_slices > 1) {
        c.dW = ws;
        left.job[jobs++] = sum_job(ws, dW, (int64_t)out * in, c.dw_slices, 0);
        ws += (int64_t)c.dw_slices * out * in;
    }
    if (dscales != nullptr && part_bytes == 0) {
        c.grads = dscales;                  // a tile's columns are a whole group, and all its tokens
    } else if (dscales != nullptr && fits) {
        c.parts = reinterpret_cast<f64_a4 *>(ws);
        const int64_t rows = (int64_t)K * out;
        left.job[jobs++] = group_size ? sum_job(ws, dscales, rows * f8_blocks(in), c.dw_slices, 1)
                                      : sum_job(ws, dscales, rows, c.dw_slices, f8_blocks(in));
        ws += part_bytes / sizeof(float);
    }
    if (dX != nullptr && c.dx_slices > 1) {
        c.dX = ws;
        left.job[jobs++] = sum_job(ws, dX, (int64_t)M * in, c.dx_slices, 0);
    }
    hipError_t e = hipSuccess;
    switch (dx_tokens(M)) {
    case 16: e = launch_few<1>(c); break;
    case 32: e = launch_few<2>(c); break;
    case 64: e = launch_few<4>(c); break;
    default:
        if (p.both) {
            e = M > 128 ? launch_both<4>(c) : launch_both<2>(c);
            break;
        }
        if (dW != nullptr)
            e = p.dw_large ? launch_dw<2, 4, 4>(c) : launch_dw<1, 4, 2>(c);
        if (e == hipSuccess && dX != nullptr)
            e = M > 128 ? launch_dx<4, 4>(c) : launch_dx<4, 2>(c);
        break;
    }
    if (e == hipSuccess && dscales != nullptr && c.grads == nullptr && c.parts == nullptr)
        e = launch_qat_dscales(planes, out, in, K, group_size, dW, dscales, st);
    if (e != hipSuccess)
        return e;
    if (jobs) {
        const unsigned blocks = left.job[0].blocks + left.job[1].blocks + left.job[2].blocks;
        hipLaunchKernelGGL(qat_ckpt_join_kernel, dim3(blocks), dim3(CK_THREADS), 0, st, left);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace rbq
