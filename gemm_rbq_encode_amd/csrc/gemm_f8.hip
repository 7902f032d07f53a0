// gemm_f8.hip -- the many-token product of a layer in 8-bit floating point
// blocks of 128:
//   Y[m][r] = sum_t xs[t][m] ws[r/128][t] sum_{j in block t} x[m][j] w[r][j]
//
// A workgroup computes a tile of W's rows by tokens.  Both operands pass
// through LDS by direct global-to-LDS loads of 16 bytes a lane: in tiles of up
// to 128 x 256 as a ring of three or four stages of one block of 128 columns
// each, one barrier per stage; in the large ones as pieces of a block that are
// freed and requested on their own.  The loads are inline assembly without
// register results and their waits are explicit (the compiler would wait for
// them before every LDS read); no other vector memory access is in flight in
// the main loops, so that the counts are exact.
//
// Where the tiles do not fill the compute units, or leave a part of a round
// over, tiles are cut into slices of columns whose fp32 sums a second kernel
// adds (in slice order: the same bits in every run).
//
// LDS holds rows of 128 bytes without padding (a load instruction fills 1 KB
// in lane order); the 16-byte piece q of row r lies at position q ^ (r & 7),
// so that the fragment reads of 8 rows of one piece hit all banks once.  The
// swizzle is applied to the addresses that are loaded from.
//
// Rows and tokens past the end repeat the last one (every element of the
// result depends on its own row and token only) and are not written.  A short
// last block is loaded through registers, zero past the end on both sides.
//
// Two kinds of sums inside a block:
//  * fp16 outputs: v_mfma_f32_16x16x128_f8f6f4, one instruction per 16 x 16
//    x 128 products.  Measured here: of the 8 products of 8 consecutive
//    columns the instruction keeps what is at least 2^-13 of the power of two
//    below the largest (each of the others is cut towards zero there), and
//    adds the groups in fp32.  A group is off by less than 7 * 2^-13 of its
//    largest product, about a seventieth of the 2^-4 that an e4m3 operand is
//    off itself; it buys twice the rate of the fp16 instruction.
//  * fp32 outputs, and fp16 ones of which the caller asks it: the codes
//    converted to fp16 (exact) in registers and v_mfma_f32_16x16x32_f16: exact
//    products, fp32 sums.
// Either way the block's sums are scaled by xs ws in one fp32 fma each.
//
// Large tiles are bound by the matrix instructions at the clock that their
// power leaves: 2048 tokens, 14336 x 4096: 124 to 128 us, 1.9 PFLOP/s (a library
// product of this size with one scale for the whole matrix: 103 us); 4096
// tokens, 8192 x 8192: 254 us, 2.2 PFLOP/s.  Exact products run at the fp16
// rate: 777 tokens, 5003 x 4128: 56 us, 570 TFLOP/s; 2048 tokens, 14336 x 4096:
// 230 us, 1.05 PFLOP/s, which is the fp16 instruction's under its power.
#include <algorithm>
#include <type_traits>

#include "rbq.h"
#include "rbq_device.h"
#include "rbq_kernels.h"
#include "f8_device.h"
#include "f8_plan.h"

namespace rbq {

namespace {

__device__ __forceinline__ uint32_t f8_lds_addr(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// 16 bytes from base + voff to LDS [m0 + 16 lane].  M0 is set here; nothing
// else in this kernel reads it.  A load to LDS may read M0 one wait state after
// a scalar write at the earliest, and the compiler places such waits around
// inline assembly, not inside it: hence the s_nop.
__device__ __forceinline__ void f8_load_lds(const void *base, uint32_t voff, uint32_t m0) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(m0) : "memory");
}

// 4 bytes from base + voff to LDS [m0 + 4 lane].
__device__ __forceinline__ void f8_load_lds4(const void *base, uint32_t voff, uint32_t m0) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(m0) : "memory");
}

// All but the N youngest loads have landed, in every wave.
template <int N>
__device__ __forceinline__ void f8_landed() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Rows r .. r + 3 of one token, at p; `vec`: rows come in whole fours and p is
// aligned to four outputs.
template <typename Y>
__device__ __forceinline__ void f8_write4(const v4f &v, int64_t r, int out, bool vec, Y *p) {
    if (vec && r < out) {
        if constexpr (sizeof(Y) == 2)
            *reinterpret_cast<uint2 *>(p) = make_uint2((uint32_t)f2h(v[0]) | (uint32_t)f2h(v[1]) << 16,
                                                       (uint32_t)f2h(v[2]) | (uint32_t)f2h(v[3]) << 16);
        else
            *reinterpret_cast<v4f *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r + i < out)
                p[i] = to_y<Y>(v[i]);
    }
}

template <typename Y>
__device__ __forceinline__ bool f8_fours(int out, const Y *y) {
    return (out & 3) == 0 && ((uintptr_t)y & (4 * sizeof(Y) - 1)) == 0;
}

// A wave's sums from row r0 and token m0 on: lane (li, g) holds rows 4 g + v of
// a row tile and token li of a token tile.
template <int TM, int TN, typename Y>
__device__ __forceinline__ void f8_write_tile(const v4f (&acc)[TM][TN], int64_t r0, int64_t m0, int li, int g, int out,
                                              int M, Y *__restrict__ y) {
    const bool vec = f8_fours(out, y);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int64_t m = m0 + j * 16 + li;
        if (m >= M)
            continue;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t r = r0 + i * 16 + 4 * g;
            f8_write4(acc[i][j], r, out, vec, y + m * out + r);
        }
    }
}

// Tiles of RT = 16 WM TM rows by CT = 16 WN TN tokens, a ring of NB stages of
// one block each.  The first `whole` tiles are computed by one workgroup each;
// every other one by `slices` workgroups, which take a share of its blocks
// each, and where these are several, leave their sums in fp32 in `parts`
// [slice][tile], F8_PART<RT, CT> apart.  (At least two waves per SIMD: with
// more registers the products are placed in accumulation registers, and every
// fma waits for a copy.)
template <int RT, int CT>
constexpr int F8_PART = RT * CT + 320;       // (a power of two apart, all would be written to the same channels at once)

template <int WM, int WN, int TM, int TN, int NB, bool EXACT, typename Y>
__global__ __launch_bounds__(WM *WN *RBQ_WAVE, 2) void gemm_f8_tile_kernel(
    const uint8_t *__restrict__ W, const float *__restrict__ ws, int out, int in, int T,
    const uint8_t *__restrict__ X, const float *__restrict__ xs, int M, Y *__restrict__ y,
    float *__restrict__ parts, int tiles_m, int tiles, int whole, int slices) {
    constexpr int WAVES = WM * WN;
    constexpr int RT = WM * TM * 16, CT = WN * TN * 16;
    constexpr int SX = RT * F8_BLOCK, SS = SX + CT * F8_BLOCK, SLOT = SS + CT * 4;   // rows, tokens, scales
    constexpr int LW = RT / 8 / WAVES, LX = CT / 8 / WAVES;      // 1 KB loads of a wave and stage
    constexpr int PER = LW + LX + 1;
    static_assert(LW * 8 * WAVES == RT && LX * 8 * WAVES == CT && CT % 64 == 0, "tile rows per wave load");
    static_assert(WAVES >= CT / 64 && TM * 16 <= F8_BLOCK, "scales of a stage");
    static_assert(NB >= 2 && NB <= 4 && PER * (NB - 2) < 64, "ring depth");
    extern __shared__ __align__(16) unsigned char lds[];
    const int lane = threadIdx.x & (RBQ_WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / RBQ_WAVE));
    const int wr = wave % WM, wc = wave / WM;
    const int li = lane & 15, g = lane >> 4;
    // tokens fastest, then rows, then (behind the whole tiles) slices
    const bool cut = (int)blockIdx.x >= whole;
    const int id = cut ? xcd_run(blockIdx.x - whole, (tiles - whole) * slices) : xcd_run(blockIdx.x, whole);
    const int tile = cut ? whole + id % (tiles - whole) : id, slice = cut ? id / (tiles - whole) : 0;
    const int shares = cut ? slices : 1;
    const int64_t r0 = (int64_t)(tile / tiles_m) * RT, m0 = (int64_t)(tile % tiles_m) * CT;

    parts += (int64_t)id * F8_PART<RT, CT>;
    asm volatile("" : "+s"(parts), "+s"(y));       // (here, not once the sums wait for them)
    const uint8_t *wbase = W + r0 * in, *xbase = X + m0 * in;
    const float *sbase = xs + m0;
    const int rlast = (int)std::min<int64_t>(out - 1 - r0, RT - 1), mlast = (int)std::min<int64_t>(M - 1 - m0, CT - 1);
    const uint32_t piece = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);   // the piece stored at this lane's place
    uint32_t woff[LW], xoff[LX];
#pragma unroll
    for (int i = 0; i < LW; ++i)
        woff[i] = (uint32_t)std::min((wave * LW + i) * 8 + (lane >> 3), rlast) * (uint32_t)in + piece;
#pragma unroll
    for (int i = 0; i < LX; ++i)
        xoff[i] = (uint32_t)std::min((wave * LX + i) * 8 + (lane >> 3), mlast) * (uint32_t)in + piece;
    constexpr int SW = CT / 64;                                   // (the other waves repeat these loads)
    const uint32_t soff = (uint32_t)std::min((wave % SW) * 64 + lane, mlast) * 4u;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(f8_lds_addr(lds));

    // this slice's blocks: t0 .. t0 + n - 1 whole ones, and the short last block in the last slice
    const int full = in / F8_BLOCK;
    const int t0 = (int)((int64_t)full * slice / shares), n = (int)((int64_t)full * (slice + 1) / shares) - t0;
    // load q = 0 .. PER - 1 of stage i
    auto issue = [&](int i, int q) {
        const int64_t t = t0 + i;
        const uint32_t at = lds0 + (uint32_t)(i % NB) * SLOT;
        if (q < LW)
            f8_load_lds(wbase + t * F8_BLOCK, woff[q < LW ? q : 0], at + (uint32_t)(wave * LW + q) * 1024u);
        else if (q < LW + LX)
            f8_load_lds(xbase + t * F8_BLOCK, xoff[q < LW + LX ? q - LW : 0],
                        at + (uint32_t)SX + (uint32_t)(wave * LX + q - LW) * 1024u);
        else
            f8_load_lds4(sbase + t * M, soff, at + (uint32_t)SS + (uint32_t)(wave % SW) * 256u);
    };

    const float *wsp = ws + std::min<int64_t>(r0 + wr * TM * 16, out - 1) / F8_BLOCK * T;   // (a wave's rows share a block)
    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

    // fragment of 16 rows starting at row `row` of an operand: pieces g and
    // g + 4 of the lane's row (the same ones on both sides)
    const uint32_t rd_lo = (uint32_t)(li * F8_BLOCK + ((g ^ (li & 7)) * 16));
    const uint32_t rd_hi = (uint32_t)(li * F8_BLOCK + (((g + 4) ^ (li & 7)) * 16));
    auto fragment = [&](const unsigned char *at, int row) {
        const uint4 lo = *reinterpret_cast<const uint4 *>(at + row * F8_BLOCK + rd_lo);
        const uint4 hi = *reinterpret_cast<const uint4 *>(at + row * F8_BLOCK + rd_hi);
        return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };

    // The products of one stage; with `request`, the loads of stage `next` go
    // out between them, a few after each row tile (issued together they would
    // hold the wave back from its products).
    auto compute = [&](const unsigned char *slot, float sw, int next, auto request) {
        auto between = [&](int i) {
            if constexpr (decltype(request)::value)
#pragma unroll
                for (int q = PER * i / TM; q < PER * (i + 1) / TM; ++q)
                    issue(next, q);
        };
        const unsigned char *wa = slot + wr * TM * 16 * F8_BLOCK;
        const unsigned char *xa = slot + SX + wc * TN * 16 * F8_BLOCK;
        const float *sl = reinterpret_cast<const float *>(slot + SS) + wc * TN * 16 + li;
        float s[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j)
            s[j] = sl[16 * j] * sw;
        if constexpr (!EXACT) {
            v8i a[3], b[TN];
            a[0] = fragment(wa, 0);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                b[j] = fragment(xa, 16 * j);
            if (TM > 1)
                a[1] = fragment(wa, 16);
            v4f p[2][TN];
            // The sums of row tile i - 1 are scaled between the products of
            // row tile i, and its fragment is read two tiles ahead; the
            // scheduling barriers keep this order (left alone, each product
            // is waited for before its fmas).
#pragma unroll
            for (int i = 0; i <= TM; ++i) {
                if (i + 2 < TM)
                    a[(i + 2) % 3] = fragment(wa, 16 * (i + 2));
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    if (i < TM) {
                        const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
                        p[i & 1][j] =
                            __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[i % 3], b[j], z, 0, 0, 0, 0, 0, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    if (i > 0)
                        acc[i - 1][j] = f8_fma(p[(i - 1) & 1][j], s[j], acc[i - 1][j]);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (i < TM)
                    between(i);
            }
        } else {
            // A product of fp16 takes as long as four vector instructions: one
            // issues it, and the conversions of what comes next (of the other
            // tokens beside row tile 0, of the next rows) and the fmas of the
            // row tile before go between, held there by the scheduling barriers.
            static_assert(TN == 4, "the places between the products");
            v8h a[2][4], b[TN][4];
            v8i ra[2], rb[2] = {fragment(xa, 0), fragment(xa, 16)};
            v4f p[2][TN];
            // pair k = 0 .. 15 of a fragment
            auto pair = [&](v8h (&h)[4], const v8i &u, int k) {
                const v2h c = k & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u[k >> 1], 1.0f, true)
                                    : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u[k >> 1], 1.0f, false);
                h[k >> 2][2 * (k & 3)] = c.x;
                h[k >> 2][2 * (k & 3) + 1] = c.y;
            };
            ra[0] = fragment(wa, 0);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                pair(b[0], rb[0], k);
            rb[0] = fragment(xa, 32);
            if (TM > 1)
                ra[1] = fragment(wa, 16);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                pair(a[0], ra[0], k);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if (i + 2 < TM)
                    ra[i & 1] = fragment(wa, 16 * (i + 2));
                auto step = [&](int j, int q, int n) {             // the n-th of the 4 TN products of this row tile
                    const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
                    p[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i & 1][q], b[j][q], q ? p[i & 1][j] : z, 0,
                                                                         0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (i == 0 && j + 1 < TN)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            pair(b[j + 1 < TN ? j + 1 : 0], rb[(j + 1) & 1], 4 * q + e);
                    if (i == 0 && q == 3 && j + 3 < TN)
                        rb[(j + 1) & 1] = fragment(xa, 16 * (j + 3));
                    if (i + 1 < TM && n < 16)
                        pair(a[(i + 1) & 1], ra[(i + 1) & 1], n);
                    if (i > 0) {
                        v4f &o = acc[i > 0 ? i - 1 : 0][n >> 2];
                        o[n & 3] = __builtin_fmaf(p[(i - 1) & 1][n >> 2][n & 3], s[n >> 2], o[n & 3]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                };
                if (i == 0) {
#pragma unroll
                    for (int n = 0; n < 4 * TN; ++n)
                        step(n >> 2, n & 3, n);
                } else {
#pragma unroll
                    for (int n = 0; n < 4 * TN; ++n)
                        step(n % TN, n / TN, n);
                }
                between(i);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[TM - 1][j] = f8_fma(p[(TM - 1) & 1][j], s[j], acc[TM - 1][j]);
        }
    };

#pragma unroll
    for (int k = 0; k < NB - 1; ++k)
        if (k < n)
#pragma unroll
            for (int q = 0; q < PER; ++q)
                issue(k, q);
    float sw = n > 0 ? wsp[t0] : 0.0f;
    auto step = [&](int i, auto request) {
        float w = sw;
        asm volatile("" : "+s"(w));                     // (the compiler's wait for it goes here)
        sw = wsp[t0 + std::min(i + 1, n - 1)];
        compute(lds + (i % NB) * SLOT, w, i + NB - 1, request);
    };
    // before stage i: it has landed (younger: the NB - 2 stages behind it),
    // and stage i - 1 is no longer read, in every wave
    int i = 0;
    for (; i + NB - 1 < n; ++i) {
        f8_landed<(NB - 2) * PER>();
        step(i, std::true_type());
    }
    for (; i < n; ++i) {
        const int younger = n - 1 - i;                  // at most NB - 2
        if (NB >= 4 && younger == 2)
            f8_landed<2 * PER>();
        else if (NB >= 3 && younger == 1)
            f8_landed<PER>();
        else
            f8_landed<0>();
        step(i, std::false_type());
    }
    if (full < T && slice == shares - 1) {
        // the short last block, through registers, zero past the end on both
        // sides (a piece past the end is read from the row's first bytes)
        __syncthreads();
        const bool ok = (int)piece < in - full * F8_BLOCK;
        const int64_t step = ok ? (int64_t)full * F8_BLOCK : -(int64_t)piece;
        auto zero_past = [&](const uint4 &v) {
            return make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
        };
#pragma unroll
        for (int i = 0; i < LW; ++i)
            *reinterpret_cast<uint4 *>(lds + (wave * LW + i) * 1024 + lane * 16) =
                zero_past(*reinterpret_cast<const uint4 *>(wbase + step + woff[i]));
#pragma unroll
        for (int i = 0; i < LX; ++i)
            *reinterpret_cast<uint4 *>(lds + SX + (wave * LX + i) * 1024 + lane * 16) =
                zero_past(*reinterpret_cast<const uint4 *>(xbase + step + xoff[i]));
        if (wave < SW)
            reinterpret_cast<float *>(lds + SS)[wave * 64 + lane] =
                sbase[(int64_t)full * M + std::min(wave * 64 + lane, mlast)];
        __syncthreads();
        compute(lds, wsp[full], 0, std::false_type());
    }
    if (shares == 1)
        f8_write_tile<TM, TN>(acc, r0 + wr * TM * 16, m0 + wc * TN * 16, li, g, out, M, y);
    else
        f8_write_tile<TM, TN>(acc, wr * TM * 16, wc * TN * 16, li, g, RT, mlast + 1, parts);
}

// The tiles from `whole` on: y = the sum of a tile's slices, in slice order.
// A thread adds 4 rows of a token; four slices' loads go out together.
template <int RT, int CT, typename Y>
__global__ __launch_bounds__(256) void gemm_f8_sum_kernel(const float *__restrict__ parts, int whole, int tiles,
                                                          int tiles_m, int slices, int out, int M,
                                                          Y *__restrict__ y) {
    constexpr int PIECES = RT / 4 * CT;
    const int cut = tiles - whole;
    const bool vec = ((uintptr_t)parts & 15) == 0, fours = f8_fours(out, y);
    for (int q = blockIdx.x / (PIECES / 256); q < cut; q += gridDim.x / (PIECES / 256)) {
        const int p = (int)(blockIdx.x % (PIECES / 256)) * 256 + threadIdx.x;
        const int tile = whole + q;
        const int64_t r = (int64_t)(tile / tiles_m) * RT + p % (RT / 4) * 4;
        const int64_t m = (int64_t)(tile % tiles_m) * CT + p / (RT / 4);
        if (r >= out || m >= M)
            continue;
        const float *from = parts + (int64_t)q * F8_PART<RT, CT> + 4 * p;
        const int64_t step = (int64_t)cut * F8_PART<RT, CT>;
        v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int z = 0; z < slices; z += 4) {
            v4f v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float *f = from + std::min(z + k, slices - 1) * step;
                if (vec)
                    v[k] = *reinterpret_cast<const v4f *>(f);
                else
                    v[k] = (v4f){f[0], f[1], f[2], f[3]};
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (z + k < slices)
                    s += v[k];
        }
        f8_write4(s, r, out, fours, y + m * out + r);
    }
}

// ---------------------------------------------------------------------------
// fp16 outputs, tiles of 32 TM rows (256, 224 or 192) by 256 tokens.  Two
// whole stages (64 KB each) leave the loads in bursts that are waited for;
// what the tile needs is a steady flow.  So a block is cut into pieces that are
// freed and requested on their own: the tokens of a block (32 KB, two slots:
// they are read into registers once, at the end of the block before), and half
// its rows (16 KB or less, five slots: row tiles 0 .. 3 of each row of waves,
// and the others).  Every half block has one barrier; the wait before it is
// for the pieces that the end of this half reads ahead, with the younger loads
// (a known number, as loads return in order) left in flight, so that a piece
// has three halves' time to arrive.  Fragments are read one row tile ahead,
// the next block's token fragments into the registers of the current ones as
// their last products are issued: after a barrier the products go on without a
// read in between.
//
// The smaller tiles fill rounds that tiles of 256 rows would leave part empty.
// A wave's 96 or 112 rows may lie in two of the weights' scale blocks, so the
// scales are chosen by row tile (four products more per row tile).

constexpr int GL_X = 256 * F8_BLOCK;              // a slot of tokens
constexpr int GL_W = 128 * F8_BLOCK;              // a slot of half the rows
constexpr int GL_S = 1024;                        // a slot of the tokens' scales
constexpr int GL_NW = 5;                          // slots of rows
constexpr int GL_W0 = 2 * GL_X, GL_S0 = GL_W0 + GL_NW * GL_W;
constexpr int GL_LDS = GL_S0 + 3 * GL_S;
constexpr int GL_THREADS = 512;

template <int TM>
__global__ __launch_bounds__(GL_THREADS) void gemm_f8_large_kernel(
    const uint8_t *__restrict__ W, const float *__restrict__ ws, int out, int in, int T,
    const uint8_t *__restrict__ X, const float *__restrict__ xs, int M, uint16_t *__restrict__ y, int tiles_m,
    int tiles_r) {
    constexpr int TN = 4, RT = 32 * TM, WR = 16 * TM;   // rows of the tile, of a wave
    constexpr bool SPLIT = WR != F8_BLOCK;              // a wave's rows may lie in two scale blocks
    constexpr int LO = TM > 6 ? 2 : 1;                  // loads of a wave for the second half's rows
    constexpr int PO = 32 * LO;                         // its rows per row of waves in a slot
    static_assert(TM >= 6 && TM <= 8 && PO >= WR - 64, "row tiles");
    extern __shared__ __align__(16) unsigned char lds[];
    const int lane = threadIdx.x & (RBQ_WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / RBQ_WAVE));
    const int wr = wave & 1, wc = wave >> 1;
    const int li = lane & 15, g = lane >> 4;

    // tiles go in bands of 8 token tiles, tokens fastest: the 32 workgroups of
    // an XCD share 8 token tiles and 4 row tiles
    int id = xcd_run(blockIdx.x, tiles_m * tiles_r);
    const int band = id / (8 * tiles_r), bw = std::min(8, tiles_m - 8 * band);
    id -= band * 8 * tiles_r;
    const int64_t r0 = (int64_t)(id / bw) * RT, m0 = (int64_t)(8 * band + id % bw) * 256;

    const uint8_t *wbase = W + r0 * in, *xbase = X + m0 * in;
    const float *sbase = xs + m0;
    const int rlast = (int)std::min<int64_t>(out - 1 - r0, RT - 1), mlast = (int)std::min<int64_t>(M - 1 - m0, 255);
    const uint32_t piece = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
    // row of the tile that lane l loads with load i of half h (with 224 rows, a
    // quarter of the second half's places repeat a row and are not read)
    auto slot_row = [&](int h, int i, int l) {
        if (h == 0) {
            const int q = (wave * 2 + i) * 8 + (l >> 3);
            return (q >> 6) * WR + (q & 63);
        }
        const int q = (wave * LO + i) * 8 + (l >> 3);
        return q / PO * WR + 64 + std::min(q % PO, WR - 65);
    };
    uint32_t woff[2][2], xoff[4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < (h == 0 ? 2 : LO); ++i)
            woff[h][i] = (uint32_t)std::min(slot_row(h, i, lane), rlast) * (uint32_t)in + piece;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        xoff[i] = (uint32_t)std::min((wave * 4 + i) * 8 + (lane >> 3), mlast) * (uint32_t)in + piece;
    const uint32_t soff = (uint32_t)std::min((wave & 3) * 64 + lane, mlast) * 4u;   // (two waves load the same)
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(f8_lds_addr(lds));

    const int full = in / F8_BLOCK;
    // load q = 0..3 of the tokens of block t, 4 of their scales; load i of half h = 2 t + (0, 1) of the rows
    auto issue_x = [&](int t, int q) {
        if (q < 4)
            f8_load_lds(xbase + (int64_t)t * F8_BLOCK, xoff[q],
                        lds0 + (uint32_t)(t & 1) * GL_X + (uint32_t)(wave * 4 + q) * 1024u);
        else
            f8_load_lds4(sbase + (int64_t)t * M, soff,
                         lds0 + GL_S0 + (uint32_t)(t % 3) * GL_S + (uint32_t)(wave & 3) * 256u);
    };
    auto row_slot = [&](int h) { return GL_W0 + (h % GL_NW) * GL_W; };
    auto issue_w = [&](int h, int odd, int i) {
        f8_load_lds(wbase + (int64_t)(h >> 1) * F8_BLOCK, woff[odd][i],
                    lds0 + (uint32_t)row_slot(h) + (uint32_t)(wave * (odd ? LO : 2) + i) * 1024u);
    };

    const uint32_t rd_lo = (uint32_t)(li * F8_BLOCK + ((g ^ (li & 7)) * 16));
    const uint32_t rd_hi = (uint32_t)(li * F8_BLOCK + (((g + 4) ^ (li & 7)) * 16));
    auto fragment = [&](const unsigned char *at, int row) {
        const uint4 lo = *reinterpret_cast<const uint4 *>(at + row * F8_BLOCK + rd_lo);
        const uint4 hi = *reinterpret_cast<const uint4 *>(at + row * F8_BLOCK + rd_hi);
        return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    auto token_slot = [&](int t) { return lds + (t & 1) * GL_X + wc * TN * 16 * F8_BLOCK; };
    auto rows_of = [&](int h, int odd) { return lds + row_slot(h) + wr * (odd ? PO : 64) * F8_BLOCK; };
    // scale blocks of the wave's first and last row tile, and the first row tile of the second
    const int64_t rw = std::min<int64_t>(r0 + wr * WR, out - 1), rb = rw / F8_BLOCK;
    const float *wsp = ws + rb * T;
    const int second = SPLIT ? (int)((rb + 1) * F8_BLOCK - rw) / 16 : TM;
    const int64_t next_block = SPLIT && second < TM && (rb + 1) * F8_BLOCK < out ? T : 0;

    v4f acc[TM][TN], p[2][TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        p[0][j] = p[1][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    }
    // Row tile i's products are in p[i & 1] and its sums taken beside those of
    // row tile i + 1; the last one of an odd number takes its own at once, and
    // has a fragment of its own, so that the next block finds the turns as
    // this one did.
    constexpr bool ODD = TM & 1;
    v8i a[2 + ODD], b[TN];
    auto at = [](int i) { return ODD && i == TM - 1 ? 2 : i & 1; };
    // scales of the tokens in this block (times the row's, where a wave has
    // one), of the last row tile in the block before, and of the rows
    float s[TN] = {}, last[TN], sw[2];
    auto row_scale = [&](int i) { return i < second ? sw[0] : sw[1]; };

    // The products of one half of a block, beside each the fmas of the row
    // tile before (of the block before, at its first).  wa: this half's rows,
    // wn: the next half's; bn: the next block's tokens; between(i): the loads
    // to issue behind row tile i.
    auto half = [&](const unsigned char *wa, const unsigned char *wn, const unsigned char *bn, auto odd,
                    auto between) {
        constexpr int I0 = 4 * decltype(odd)::value, N = decltype(odd)::value ? TM - 4 : 4;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int I = I0 + i;
            a[I + 1 < TM ? at(I + 1) : 0] = i + 1 < N ? fragment(wa, 16 * (i + 1)) : fragment(wn, 0);
            float f[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j)
                f[j] = I == 0 ? last[j] : SPLIT ? s[j] * row_scale(I - 1) : s[j];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const v4f z = {0.0f, 0.0f, 0.0f, 0.0f};
                p[I & 1][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[at(I)], b[j], z, 0, 0, 0, 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (I == TM - 1)
                    b[j] = fragment(bn, 16 * j);
                if (I > 0)
                    acc[I - 1][j] = f8_fma(p[(I - 1) & 1][j], f[j], acc[I - 1][j]);
                else if (!ODD)
                    acc[TM - 1][j] = f8_fma(p[1][j], f[j], acc[TM - 1][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
            between(i);
        }
        if (ODD && decltype(odd)::value)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[TM - 1][j] = f8_fma(p[0][j], s[j] * row_scale(TM - 1), acc[TM - 1][j]);
    };
    auto first_fragments = [&](const unsigned char *wa, const unsigned char *ba) {
        a[0] = fragment(wa, 0);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            b[j] = fragment(ba, 16 * j);
    };
    // the scales of a block: those of the tokens from sl, of the rows in sw
    auto take_scales = [&](auto scale) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            last[j] = s[j];
            s[j] = SPLIT ? scale(j) : scale(j) * sw[0];
        }
    };
    auto keep_last = [&]() {                     // (before the rows' scales of the next block are taken)
        if (SPLIT && !ODD)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                s[j] *= row_scale(TM - 1);
    };

    // requests go out in the order W 2t, X t, S t, W 2t + 1
    if (full > 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t >= full)
                break;
            issue_w(2 * t, 0, 0);
            issue_w(2 * t, 0, 1);
#pragma unroll
            for (int q = 0; q < 5; ++q)
                issue_x(t, q);
#pragma unroll
            for (int i = 0; i < LO; ++i)
                issue_w(2 * t + 1, 1, i);
        }
        if (full > 1)
            f8_landed<7 + 2 * LO>();
        else
            f8_landed<LO>();
        first_fragments(rows_of(0, 0), token_slot(0));
    }
    sw[0] = full > 0 ? wsp[0] : 0.0f;
    sw[1] = SPLIT && full > 0 ? wsp[next_block] : sw[0];
    constexpr std::integral_constant<int, 0> c0;
    constexpr std::integral_constant<int, 1> c1;
    constexpr std::integral_constant<int, 2> c2;
    // Block t, with `more` full blocks (two: two or more) behind it.  Past the
    // last one old bytes of the slots are read, for fragments that no one uses.
    auto stage = [&](int t, auto more) {
        constexpr int MORE = decltype(more)::value;
        // second half of t; younger: W 2t + 2, X and S t + 1, W 2t + 3
        f8_landed<(MORE > 0 ? 7 + LO : 0)>();
        asm volatile("" : "+s"(sw[0]), "+s"(sw[1]));       // (the compiler's wait for them goes here)
        const float *sl = reinterpret_cast<const float *>(lds + GL_S0 + (t % 3) * GL_S) + wc * TN * 16 + li;
        take_scales([&](int j) { return sl[16 * j]; });
        half(rows_of(2 * t, 0), rows_of(2 * t + 1, 1), lds, c0, [&](int i) {
            if (MORE > 1) {
                if (i == 0) {
                    issue_w(2 * t + 4, 0, 0);
                    issue_w(2 * t + 4, 0, 1);
                } else {
                    issue_x(t + 2, 2 * i - 2);
                    if (i < 3)
                        issue_x(t + 2, 2 * i - 1);
                }
            }
        });
        // W 2t + 2 and X t + 1; younger: W 2t + 3, W 2t + 4, X and S t + 2
        f8_landed<(MORE > 1 ? 7 + LO : MORE > 0 ? LO : 0)>();
        float sn[2] = {sw[0], sw[1]};
        if (MORE > 0) {
            sn[0] = wsp[t + 1];
            if (SPLIT)
                sn[1] = wsp[next_block + t + 1];
        }
        half(rows_of(2 * t + 1, 1), rows_of(2 * t + 2, 0), token_slot(t + 1), c1, [&](int i) {
            if (MORE > 1 && i < LO)
                issue_w(2 * t + 5, 1, i);
        });
        keep_last();
        sw[0] = sn[0];
        sw[1] = sn[1];
    };
    int t = 0;
    for (; t + 2 < full; ++t)
        stage(t, c2);
    if (t + 1 < full)
        stage(t++, c1);
    if (t < full)
        stage(t, c0);
    if (full < T) {
        // the short last block, through registers, zero past the end on both
        // sides (a piece past the end is read from the row's first bytes)
        __syncthreads();
        int l = lane;
        asm volatile("" : "+v"(l));                        // (the places are worked out anew, not kept)
        const int c = ((l & 7) ^ (l >> 3)) * 16;
        const bool ok = c < in - full * F8_BLOCK;
        const int64_t at = ok ? (int64_t)full * F8_BLOCK + c : 0;
        auto zero_past = [&](const uint4 &v) {
            return make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = std::min((wave * 4 + i) * 8 + (l >> 3), mlast);
            const uint4 v = *reinterpret_cast<const uint4 *>(xbase + m * in + at);
            *reinterpret_cast<uint4 *>(lds + (wave * 4 + i) * 1024 + l * 16) = zero_past(v);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < (h == 0 ? 2 : LO); ++i) {
                const int64_t r = std::min(slot_row(h, i, l), rlast);
                const uint4 v = *reinterpret_cast<const uint4 *>(wbase + r * in + at);
                *reinterpret_cast<uint4 *>(lds + row_slot(h) + (wave * (h == 0 ? 2 : LO) + i) * 1024 + l * 16) =
                    zero_past(v);
            }
        __syncthreads();
        first_fragments(rows_of(0, 0), token_slot(0));
        sw[0] = wsp[full];
        sw[1] = wsp[next_block + full];
        take_scales([&](int j) { return sbase[(int64_t)full * M + std::min((wc * TN + j) * 16 + li, mlast)]; });
        half(rows_of(0, 0), rows_of(1, 1), lds, c0, [](int) {});
        half(rows_of(1, 1), rows_of(0, 0), lds, c1, [](int) {});
        keep_last();
    }
    if (!ODD)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[TM - 1][j] = f8_fma(p[1][j], s[j], acc[TM - 1][j]);
    f8_write_tile<TM, TN>(acc, r0 + wr * WR, m0 + wc * TN * 16, li, g, out, M, y);
}

template <int WM, int WN, int TM, int TN, int NB, bool EXACT, typename Y>
hipError_t launch_tile(const uint8_t *W, const float *ws, int out, int in, const uint8_t *X, const float *xs, int M,
                       Y *y, float *parts, f8_plan p, hipStream_t st) {
    constexpr int RT = WM * TM * 16, CT = WN * TN * 16;
    constexpr int LDS = NB * ((RT + CT) * F8_BLOCK + CT * 4);
    static_assert(LDS <= 160 * 1024, "LDS of a compute unit");
    const int tiles_m = (int)(((int64_t)M + CT - 1) / CT), tiles = tiles_m * (int)(((int64_t)out + RT - 1) / RT);
    const int64_t groups = p.whole + (int64_t)(tiles - p.whole) * p.slices;
    hipLaunchKernelGGL((gemm_f8_tile_kernel<WM, WN, TM, TN, NB, EXACT, Y>), dim3((unsigned)groups), dim3(WM * WN * RBQ_WAVE),
                       LDS, st, W, ws, out, in, f8_blocks(in), X, xs, M, y, parts, tiles_m, tiles, p.whole, p.slices);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.slices == 1)
        return e;
    constexpr int PER_TILE = RT / 4 * CT / 256;
    hipLaunchKernelGGL((gemm_f8_sum_kernel<RT, CT, Y>), dim3((unsigned)std::min(tiles - p.whole, 4096) * PER_TILE),
                       dim3(256), 0, st, parts, p.whole, tiles, tiles_m, p.slices, out, M, y);
    return hipGetLastError();
}

template <int TM>
hipError_t launch_large(const uint8_t *W, const float *ws, int out, int in, const uint8_t *X, const float *xs, int M,
                        uint16_t *y, hipStream_t st) {
    const int tiles_m = (int)(((int64_t)M + 255) / 256), tiles_r = (int)(((int64_t)out + 32 * TM - 1) / (32 * TM));
    hipLaunchKernelGGL((gemm_f8_large_kernel<TM>), dim3((unsigned)(tiles_m * tiles_r)), dim3(GL_THREADS), GL_LDS, st,
                       W, ws, out, in, f8_blocks(in), X, xs, M, y, tiles_m, tiles_r);
    return hipGetLastError();
}

template <bool EXACT, typename Y>
hipError_t launch_tiles(const uint8_t *W, const float *ws, int out, int in, const uint8_t *X, const float *xs, int M,
                        Y *y, float *parts, f8_plan p, hipStream_t st) {
    switch (p.kind) {
    case F8_LARGE: return launch_tile<2, 4, 4, 4, 3, EXACT>(W, ws, out, in, X, xs, M, y, parts, p, st);
    case F8_LARGE + 1: return launch_tile<2, 2, 4, 4, 4, EXACT>(W, ws, out, in, X, xs, M, y, parts, p, st);
    default: return launch_tile<2, 2, 2, 4, 4, EXACT>(W, ws, out, in, X, xs, M, y, parts, p, st);
    }
}

}  // namespace

size_t gemm_f8_workspace_bytes(int out, int in, int M, int exact) {
    if (M <= F8_FEW || !gemm_f8_tile_supports(out, in, M))
        return 0;
    const f8_plan p = plan_tiles(out, in, M, exact);
    const int64_t rows = F8_ROWS[p.kind], tokens = F8_TOKENS[p.kind];
    const int64_t tiles = (out + rows - 1) / rows * ((M + tokens - 1) / tokens);
    return p.slices > 1 ? (size_t)((tiles - p.whole) * p.slices * (rows * tokens + F8_PART<0, 0>)) * sizeof(float) : 0;
}

hipError_t launch_gemm_f8_tile(const uint8_t *W, const float *ws, int out, int in, const uint8_t *X, const float *xs,
                               int M, void *y, int y_f32, int exact, void *workspace, size_t ws_bytes, hipStream_t st) {
    f8_plan p = plan_tiles(out, in, M, exact);
    if (ws_bytes < gemm_f8_workspace_bytes(out, in, M, exact))
        p.slices = 1;
    float *parts = static_cast<float *>(workspace);
    if (y_f32)
        return launch_tiles<true>(W, ws, out, in, X, xs, M, static_cast<float *>(y), parts, p, st);
    uint16_t *o = static_cast<uint16_t *>(y);
    if (exact)
        return launch_tiles<true>(W, ws, out, in, X, xs, M, o, parts, p, st);
    switch (p.kind) {
    case 0: return launch_large<8>(W, ws, out, in, X, xs, M, o, st);
    case 1: return launch_large<7>(W, ws, out, in, X, xs, M, o, st);
    case 2: return launch_large<6>(W, ws, out, in, X, xs, M, o, st);
    default: return launch_tiles<false>(W, ws, out, in, X, xs, M, o, parts, p, st);
    }
}

}  // namespace rbq
