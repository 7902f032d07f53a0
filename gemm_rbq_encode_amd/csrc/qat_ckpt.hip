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

#include "rbq.h"
#include "rbq_device.h"
#include "rbq_kernels.h"
#include "f8_device.h"

namespace rbq {

namespace {

constexpr int CK_THREADS = 256;
constexpr int CK_ROWS = CK_THREADS / 16;      // tokens of a workgroup: 16 lanes per block
constexpr int CK_BLOCKS = 4;                  // blocks per lane, loaded together

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

__global__ __launch_bounds__(CK_THREADS) void qat_checkpoint_kernel(const uint16_t *__restrict__ X, int M, int in,
                                                                    int T, int64_t units,
                                                                    int8_t *__restrict__ codes,
                                                                    uint16_t *__restrict__ scales) {
    const int li = threadIdx.x & 15;
    const int tg = (T + CK_BLOCKS - 1) / CK_BLOCKS;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t m = u / tg * CK_ROWS + (threadIdx.x >> 4);
        const int t0 = (int)(u % tg) * CK_BLOCKS;
        if (m >= M)
            continue;
        const uint16_t *row = X + m * in;
        uint4 v[CK_BLOCKS];
#pragma unroll
        for (int b = 0; b < CK_BLOCKS; ++b) {
            const int64_t c = (int64_t)(t0 + b) * F8_BLOCK + 8 * li;
            v[b] = c < in ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int b = 0; b < CK_BLOCKS; ++b) {
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
// stage t + 2 are issued, and the registers of stage t + 1 written to the
// other buffer, in pieces between the matrix instructions of stage t.  One
// barrier per stage.  Both operands of dW, and What of dX, lie with the
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
// The gradients of the scales are sums of +-dW over groups of columns: each
// wave adds its 128 columns from the registers it has just computed and
// writes one value per row and plane to parts [K][out][ceil(in / 128)], which
// are the group gradients themselves for groups of 128 and are added in order
// by qat_ckpt_sum_parts for scales per row.

constexpr int CW_BK = 64;
constexpr int CW_TM = 8;

template <int WM, int WN, int TN>
__global__ __launch_bounds__(WM *WN *RBQ_WAVE) void qat_ckpt_dw_kernel(
    const uint16_t *__restrict__ dY, const int8_t *__restrict__ codes, const uint16_t *__restrict__ cscales, int M,
    int out, int in, int T, float *__restrict__ dW, const uint32_t *__restrict__ planes, int K,
    float *__restrict__ parts, int tiles_j, int total) {
    constexpr int THREADS = WM * WN * RBQ_WAVE;
    constexpr int CJ = WM * 128, CR = WN * TN * 16;            // tile: columns x rows of dW
    constexpr int PJ = CJ / 8, PR = CR / 8;                    // pieces of an LDS row
    constexpr int XB = CW_BK * CJ * 2, STAGE = XB + CW_BK * CR * 2;
    constexpr int NX = CW_BK * CJ / 16 / THREADS;              // 16 codes each
    constexpr int NY = CW_BK * PR / THREADS;                   // 8 values of dY each
    static_assert(NX * THREADS * 16 == CW_BK * CJ && NY * THREADS == CW_BK * PR, "staging covers the tile");
    extern __shared__ __align__(16) unsigned char lds[];
    const int tid = threadIdx.x;
    const int lane = tid & (RBQ_WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / RBQ_WAVE);
    const int wj = wave % WM, wr = wave / WM;
    const int li = lane & 15, g = lane >> 4;
    const int id = xcd_run(blockIdx.x, total);
    const int64_t j0 = (int64_t)(id % tiles_j) * CJ, r0 = (int64_t)(id / tiles_j) * CR;

    v4f acc[CW_TM][TN];
#pragma unroll
    for (int i = 0; i < CW_TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

    v4u xr[NX], yr[NY];
    uint16_t xs[NX];
    auto load_x = [&](int64_t m0, int u) {
        const int c = u * THREADS + tid;
        const int64_t m = m0 + c / (CJ / 16), j = j0 + 16 * (c % (CJ / 16));
        const bool ok = m < M && j < in;
        xr[u] = ok ? *reinterpret_cast<const v4u *>(codes + m * in + j) : (v4u){0u, 0u, 0u, 0u};
        xs[u] = ok ? cscales[m * T + j / F8_BLOCK] : (uint16_t)0;
    };
    auto load_y = [&](int64_t m0, int u) {
        const int c = u * THREADS + tid;
        const int64_t m = m0 + c / PR;
        yr[u] = ck_piece(dY + m * out, r0 + 8 * (c % PR), out, m < M);
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

    const int64_t steps = ((int64_t)M + CW_BK - 1) / CW_BK;
#pragma unroll
    for (int u = 0; u < NX; ++u) {
        load_x(0, u);
        store_x(lds, u);
        load_x(CW_BK, u);
    }
#pragma unroll
    for (int u = 0; u < NY; ++u) {
        load_y(0, u);
        store_y(lds, u);
        load_y(CW_BK, u);
    }
    ck_barrier();
    for (int64_t t = 0; t < steps; ++t) {
        const unsigned char *cur = lds + (t & 1) * STAGE;
        unsigned char *nxt = lds + ((t + 1) & 1) * STAGE;
        const int64_t m2 = (t + 2) * CW_BK;
#pragma unroll
        for (int kk = 0; kk < CW_BK / 32; ++kk) {
            v8h b[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j)
                b[j] = ck_column(cur + yo[j] + kk * 32 * (CR * 2), CR * 2);
            v8h a = ck_column(cur + xo[0] + kk * 32 * (CJ * 2), CJ * 2);
#pragma unroll
            for (int i = 0; i < CW_TM; ++i) {
                v8h an = a;
                if (i + 1 < CW_TM)
                    an = ck_column(cur + xo[i + 1] + kk * 32 * (CJ * 2), CJ * 2);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[j], acc[i][j], 0, 0, 0);
                a = an;
                // one piece of the next stages' data after every second tile row
                const int u = (kk * CW_TM + i) / 2;
                if (i & 1) {
                    if (u < NX) {
                        store_x(nxt, u);
                        load_x(m2, u);
                    } else if (u - NX < NY) {
                        store_y(nxt, u - NX);
                        load_y(m2, u - NX);
                    }
                }
            }
        }
        static_assert(NX + NY <= CW_BK / 32 * CW_TM / 2, "every piece is staged within a stage");
        ck_barrier();
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
    if (parts == nullptr || j0 + wj * 128 >= in)
        return;
    const int64_t words = in >> 5;
    const int64_t w0 = (j0 + wj * 128) >> 5;
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t r = r0 + (wr * TN + j) * 16 + li;
            const uint32_t *pw = planes + ((int64_t)k * out + std::min<int64_t>(r, out - 1)) * words;
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (w0 + q >= words)
                    break;
                const uint32_t w = ~pw[w0 + q] >> (4 * g);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        s += __uint_as_float(__float_as_uint(acc[2 * q + h][j][v]) ^
                                             ((w << (31 - 16 * h - v)) & 0x80000000u));
            }
            s += __shfl_xor(s, 16, RBQ_WAVE);
            s += __shfl_xor(s, 32, RBQ_WAVE);
            if (g == 0 && r < out)
                parts[((int64_t)k * out + r) * T + (j0 >> 7) + wj] = s;
        }
    }
}

// dscales[n] = the sum of T parts in order, in fp64: one wave each.
__global__ __launch_bounds__(CK_THREADS) void qat_ckpt_sum_parts(const float *__restrict__ parts, int64_t n, int T,
                                                                 float *__restrict__ dscales) {
    const int lane = threadIdx.x & (RBQ_WAVE - 1);
    const int64_t i = (int64_t)blockIdx.x * (CK_THREADS / RBQ_WAVE) + threadIdx.x / RBQ_WAVE;
    if (i >= n)
        return;                                   // whole wave
    double s = 0.0;
    for (int t = lane; t < T; t += RBQ_WAVE)
        s += (double)parts[i * T + t];
    s = wave_sum_f64(s);
    if (lane == 0)
        dscales[i] = (float)s;
}

// ---------------------------------------------------------------------------
// dX[m][j] = sum_r dY[m][r] What[r][j], What = sum_k a_k B_k formed in fp32 and
// split into two fp16 parts hi = fp16(w), lo = fp16(w - hi), as in qat.hip.
// Tiles of 64 TM tokens x 128 columns, 64 rows r per stage; waves 4 x 2.  A
// thread forms 16 columns of one row.  With one or two planes a row has four
// values, which a byte permute looks up from two 8-byte tables (hi and lo)
// two columns at a time; with three and four the sums are formed one by one.

constexpr int CX_BK = 64;
constexpr int CX_J = 128;
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

template <int TM, int K>
__global__ __launch_bounds__(CX_THREADS) void qat_ckpt_dx_kernel(
    const uint16_t *__restrict__ dY, const uint32_t *__restrict__ planes, const uint16_t *__restrict__ scales, int M,
    int out, int in, int group_size, int64_t r_slice, float *__restrict__ dX, int32_t *__restrict__ status,
    int tiles_j, int tiles_m, int total) {
    constexpr int CM = 64 * TM;
    constexpr int YB = CM * CX_BK * 2, HB = CX_BK * CX_J * 2, STAGE = YB + 2 * HB;
    constexpr int NY = CM * (CX_BK / 8) / CX_THREADS;          // 8 values of dY each
    constexpr int PJ = CX_J / 8;
    extern __shared__ __align__(16) unsigned char lds[];
    const int tid = threadIdx.x;
    const int lane = tid & (RBQ_WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / RBQ_WAVE);
    const int wm = wave & 3, wj = wave >> 2;
    const int li = lane & 15, g = lane >> 4;
    const int id = xcd_run(blockIdx.x, total);
    const int z = id / (tiles_j * tiles_m);
    const int64_t j0 = (int64_t)(id % tiles_j) * CX_J, m0 = (int64_t)(id / tiles_j % tiles_m) * CM;
    const int64_t words = in >> 5;
    const int G = group_size ? in / group_size : 1;
    const int64_t r_lo = z * r_slice, r_hi = std::min<int64_t>(out, r_lo + r_slice);
    dX += (int64_t)z * M * in;

    v4f acc[4][TM];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

    // staging: 8 pieces per token row, piece p of token m at p ^ (m & 7)
    v4u yr[NY];
    auto load_y = [&](int64_t rb, int u) {
        const int c = u * CX_THREADS + tid;
        const int64_t m = m0 + (c >> 3);
        yr[u] = ck_piece(dY + m * out, rb + 8 * (c & 7), r_hi, m < M);
    };
    auto store_y = [&](unsigned char *at, int u) {
        const int c = u * CX_THREADS + tid;
        const int m = c >> 3, p = c & 7;
        *reinterpret_cast<v4u *>(at + m * (CX_BK * 2) + (p ^ (m & 7)) * 16) = yr[u];
    };
    const int fr = tid >> 3, fj = tid & 7;                     // this thread's row of What and 16 columns
    const int64_t fw = (j0 >> 5) + (fj >> 1);
    const int64_t fg = group_size ? j0 / group_size : 0;       // 128 columns lie in one group
    uint32_t bits[K];
    uint16_t sc[K];
    bool valid = false, ovf = false;
    auto load_w = [&](int64_t rb) {
        const int64_t r = rb + fr;
        valid = r < r_hi && fw < words;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            bits[k] = valid ? planes[((int64_t)k * out + r) * words + fw] : 0u;
            sc[k] = valid ? scales[((int64_t)k * out + r) * G + fg] : (uint16_t)0;
        }
    };
    uint32_t hv[8], lv[8];
    auto form = [&]() {
        const int sh = 16 * (fj & 1);
        if constexpr (K <= 2) {
            const uint32_t b0 = bits[0] >> sh, b1 = K > 1 ? bits[K - 1] >> sh : 0u;
            const float a0 = h2f(sc[0]), a1 = K > 1 ? h2f(sc[K - 1]) : 0.0f;
            // index b0 + 2 b1: -a0 - a1, a0 - a1, a1 - a0, a0 + a1 (K = 1: only the first two, b1 = 0)
            const float w0 = -a0 - a1, w1 = a0 - a1;
            const uint32_t diff = (b0 ^ b1) & 0xFFFFu;
            ovf = ovf || (valid && ((diff != 0xFFFFu && !(__builtin_fabsf(w0) < 65520.0f)) ||
                                    (diff != 0u && !(__builtin_fabsf(w1) < 65520.0f))));
            const _Float16 h0 = (_Float16)w0, h1 = (_Float16)w1;
            uint32_t hl, hh, ll, lh;
            ck_table(h0, h1, hl, hh);
            ck_table((_Float16)(w0 - (float)h0), (_Float16)(w1 - (float)h1), ll, lh);
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const uint32_t e = ((b0 >> (2 * p)) & 1u) | (((b1 >> (2 * p)) & 1u) << 1);
                const uint32_t o = ((b0 >> (2 * p + 1)) & 1u) | (((b1 >> (2 * p + 1)) & 1u) << 1);
                const uint32_t sel = (e | o << 16) * 0x101u + 0x04000400u;
                hv[p] = __builtin_amdgcn_perm(hh, hl, sel);
                lv[p] = __builtin_amdgcn_perm(lh, ll, sel);
            }
        } else {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                _Float16 h[2], l[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float w = 0.0f;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        w += __uint_as_float(__float_as_uint(h2f(sc[k])) ^
                                             ((~(bits[k] >> sh) << (31 - 2 * p - e)) & 0x80000000u));
                    ovf = ovf || (valid && !(__builtin_fabsf(w) < 65520.0f));
                    h[e] = (_Float16)w;
                    l[e] = (_Float16)(w - (float)h[e]);
                }
                hv[p] = ck_pack(h[0], h[1]);
                lv[p] = ck_pack(l[0], l[1]);
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
    uint32_t wo[4], yo[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        wo[i] = YB + k0 * (CX_J * 2) + (((wj * 4 + i) * 2) ^ ck_swizzle(k0, PJ)) * 16 + 8 * (li & 3);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
        yo[kk] = (wm * TM * 16 + li) * (CX_BK * 2) + ((4 * kk + g) ^ (li & 7)) * 16;

    const int64_t steps = (r_hi - r_lo + CX_BK - 1) / CX_BK;
    load_w(r_lo);
    form();
    store_w(lds);
    load_w(r_lo + CX_BK);
#pragma unroll
    for (int u = 0; u < NY; ++u) {
        load_y(r_lo, u);
        store_y(lds, u);
        load_y(r_lo + CX_BK, u);
    }
    ck_barrier();
    for (int64_t t = 0; t < steps; ++t) {
        const unsigned char *cur = lds + (t & 1) * STAGE;
        unsigned char *nxt = lds + ((t + 1) & 1) * STAGE;
        const int64_t r2 = r_lo + (t + 2) * CX_BK;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            v8h b[TM];
#pragma unroll
            for (int j = 0; j < TM; ++j)
                b[j] = *reinterpret_cast<const v8h *>(cur + yo[kk] + j * 16 * (CX_BK * 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const v8h al = ck_column(cur + wo[i] + HB + kk * 32 * (CX_J * 2), CX_J * 2);
                const v8h ah = ck_column(cur + wo[i] + kk * 32 * (CX_J * 2), CX_J * 2);
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(al, b[j], acc[i][j], 0, 0, 0);
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ah, b[j], acc[i][j], 0, 0, 0);
                const int u = kk * 4 + i;
                if (u == 0)
                    form();
                else if (u == 1) {
                    store_w(nxt);
                    load_w(r2);
                } else if (u - 2 < NY) {
                    store_y(nxt, u - 2);
                    load_y(r2, u - 2);
                }
            }
        }
        static_assert(NY <= 6, "every piece is staged within a stage");
        ck_barrier();
    }

    const bool vec = ((uintptr_t)dX & 15) == 0;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int64_t m = m0 + (wm * TM + j) * 16 + li;
        if (m >= M)
            continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = j0 + (wj * 4 + i) * 16 + 4 * g;
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

// dX = the sum of the S partial slices, in slice order.
__global__ __launch_bounds__(CK_THREADS) void qat_ckpt_sum_slices(const float *__restrict__ parts, int S, int64_t n,
                                                                  float *__restrict__ dX) {
    const int64_t i = (int64_t)blockIdx.x * CK_THREADS + threadIdx.x;
    if (i >= n)
        return;
    float v = parts[i];
    for (int z = 1; z < S; ++z)
        v += parts[z * n + i];
    dX[i] = v;
}

constexpr int LDS_MAX = 160 * 1024;

template <int WM, int WN, int TN>
hipError_t launch_dw(const uint16_t *dY, const int8_t *codes, const uint16_t *cscales, int M, int out, int in,
                     float *dW, const uint32_t *planes, int K, float *parts, hipStream_t st) {
    constexpr int CJ = WM * 128, CR = WN * TN * 16;
    constexpr int LDS = 2 * CW_BK * (CJ + CR) * 2;
    static_assert(LDS <= LDS_MAX, "LDS of a compute unit");
    const int64_t tiles_j = ((int64_t)in + CJ - 1) / CJ, total = tiles_j * (((int64_t)out + CR - 1) / CR);
    if (total > 0x7FFFFFFF / (WM * WN * RBQ_WAVE))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((qat_ckpt_dw_kernel<WM, WN, TN>), dim3((unsigned)total), dim3(WM * WN * RBQ_WAVE), LDS, st, dY,
                       codes, cscales, M, out, in, f8_blocks(in), dW, planes, K, parts, (int)tiles_j, (int)total);
    return hipGetLastError();
}

template <int TM>
hipError_t launch_dx(const uint16_t *dY, const uint32_t *planes, const uint16_t *scales, int M, int out, int in,
                     int K, int group_size, int S, int64_t r_slice, float *dX, int32_t *status, hipStream_t st) {
    constexpr int LDS = 2 * (64 * TM * CX_BK * 2 + 2 * CX_BK * CX_J * 2);
    static_assert(LDS <= LDS_MAX, "LDS of a compute unit");
    const int64_t tiles_j = ((int64_t)in + CX_J - 1) / CX_J, tiles_m = ((int64_t)M + 64 * TM - 1) / (64 * TM);
    const int64_t total = tiles_j * tiles_m * S;
    if (total > 0x7FFFFFFF / CX_THREADS)
        return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)total), dim3(CX_THREADS), LDS, st, dY, planes, scales, M, out, in,
                           group_size, r_slice, dX, status, (int)tiles_j, (int)tiles_m, (int)total);
    };
    switch (K) {
    case 1: go(qat_ckpt_dx_kernel<TM, 1>); break;
    case 2: go(qat_ckpt_dx_kernel<TM, 2>); break;
    case 3: go(qat_ckpt_dx_kernel<TM, 3>); break;
    default: go(qat_ckpt_dx_kernel<TM, 4>); break;
    }
    return hipGetLastError();
}

// Tokens per dX tile in units of 64, and slices of its contraction: enough
// workgroups for one per compute unit, at most 16 slices of at least 256 rows.
int dx_tokens(int M) { return M > 64 ? 4 : 1; }

int dx_slices(int M, int out, int in) {
    const int cm = 64 * dx_tokens(M);
    const int64_t tiles = ((int64_t)in + CX_J - 1) / CX_J * (((int64_t)M + cm - 1) / cm);
    const int64_t S = std::min<int64_t>({(256 + tiles - 1) / tiles, 16, std::max(1, out / 256)});
    return (int)std::max<int64_t>(S, 1);
}

size_t dx_slice_bytes(int M, int out, int in) {
    const int S = dx_slices(M, out, in);
    return S > 1 ? (size_t)S * (size_t)M * (size_t)in * sizeof(float) : 0;
}

size_t dw_part_bytes(int out, int in, int K, int group_size) {
    return group_size || in <= F8_BLOCK ? 0 : (size_t)K * (size_t)out * (size_t)f8_blocks(in) * sizeof(float);
}

}  // namespace

hipError_t launch_qat_checkpoint(const uint16_t *X, int M, int in, int8_t *codes, uint16_t *scales,
                                 hipStream_t st) {
    const int T = f8_blocks(in);
    const int64_t units = ((int64_t)M + CK_ROWS - 1) / CK_ROWS * ((T + CK_BLOCKS - 1) / CK_BLOCKS);
    hipLaunchKernelGGL(qat_checkpoint_kernel, dim3((unsigned)std::min<int64_t>(units, 1 << 22)), dim3(CK_THREADS),
                       0, st, X, M, in, T, units, codes, scales);
    return hipGetLastError();
}

// dW and its parts come first on the stream, the slices of dX after their sum:
// both may use the same memory.
size_t qat_backward_ckpt_workspace_bytes(int M, int out, int in, int K, int group_size) {
    return std::max(dx_slice_bytes(M, out, in), dw_part_bytes(out, in, K, group_size));
}

hipError_t launch_qat_backward_ckpt(const uint32_t *planes, const uint16_t *scales, int out, int in, int K,
                                    int group_size, const int8_t *x_codes, const uint16_t *x_scales,
                                    const uint16_t *dY, int M, float *dX, float *dW, float *dscales,
                                    void *workspace, size_t ws_bytes, int32_t *status, hipStream_t st) {
    hipError_t e = hipSuccess;
    if (dW != nullptr) {
        // the sums of a tile go straight to dscales where a tile's columns
        // are a whole group, else through the workspace; without one the
        // scales' gradients are taken from dW in a pass of its own
        const size_t need = dw_part_bytes(out, in, K, group_size);
        const bool fused = dscales != nullptr && ws_bytes >= need;
        float *parts = !fused ? nullptr : need ? static_cast<float *>(workspace) : dscales;
        const int64_t large = ((int64_t)in + 255) / 256 * (((int64_t)out + 255) / 256);
        e = large >= 200 ? launch_dw<2, 4, 4>(dY, x_codes, x_scales, M, out, in, dW, planes, K, parts, st)
                         : launch_dw<1, 4, 2>(dY, x_codes, x_scales, M, out, in, dW, planes, K, parts, st);
        if (e != hipSuccess)
            return e;
        if (fused && need) {
            const int64_t n = (int64_t)K * out;
            hipLaunchKernelGGL(qat_ckpt_sum_parts, dim3((unsigned)((n + 3) / 4)), dim3(CK_THREADS), 0, st, parts, n,
                               f8_blocks(in), dscales);
            e = hipGetLastError();
        } else if (dscales != nullptr && !fused) {
            e = launch_qat_dscales(planes, out, in, K, group_size, dW, dscales, st);
        }
        if (e != hipSuccess)
            return e;
    }
    if (dX != nullptr) {
        int S = dx_slices(M, out, in);
        if (ws_bytes < dx_slice_bytes(M, out, in))
            S = 1;
        const int64_t r_slice = (((int64_t)out + S - 1) / S + CX_BK - 1) / CX_BK * CX_BK;
        S = (int)(((int64_t)out + r_slice - 1) / r_slice);
        float *dst = S > 1 ? static_cast<float *>(workspace) : dX;
        e = dx_tokens(M) == 4
                ? launch_dx<4>(dY, planes, scales, M, out, in, K, group_size, S, r_slice, dst, status, st)
                : launch_dx<1>(dY, planes, scales, M, out, in, K, group_size, S, r_slice, dst, status, st);
        if (e != hipSuccess || S == 1)
            return e;
        const int64_t n = (int64_t)M * in;
        hipLaunchKernelGGL(qat_ckpt_sum_slices, dim3((unsigned)((n + CK_THREADS - 1) / CK_THREADS)),
                           dim3(CK_THREADS), 0, st, static_cast<const float *>(workspace), S, n, dX);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace rbq
