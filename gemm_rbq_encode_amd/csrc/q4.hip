// q4.hip -- linears in 4 bits with a scale per row and group of 128 columns: the
// encoder and the products for few tokens.
//
// A weight is (c - z) s with a code c in 0..15, the group's zero point z (8
// where a layer has none) and binary16 scale s.
#include <hip/hip_runtime.h>

#include "rbq.h"
#include "rbq_device.h"
#include "rbq_kernels.h"
#include "q4_device.h"
#include "q4_plan.h"

namespace rbq {

namespace {

constexpr int Q4E_THREADS = 256, Q4E_AHEAD = 4;

// Maximum over the 16 lanes of a row, by rotations.
__device__ __forceinline__ float row_max(float v) {
#define RBQ_ROR(n) \
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + (n), 0xF, 0xF, true)))
    RBQ_ROR(8);
    RBQ_ROR(4);
    RBQ_ROR(2);
    RBQ_ROR(1);
#undef RBQ_ROR
    return v;
}

// ---------------------------------------------------------------------------
// encoder: 16 lanes hold a group (8 consecutive weights each) between its maximum and
// its codes, four groups a lane at a time so that four loads are on their way.  W is
// read once; bound by that read: 4096 x 11008 with zero points 44.9 us, 4.5 TB/s of
// reads and writes (a copy: 5.2).
template <bool ZEROS>
__global__ __launch_bounds__(Q4E_THREADS) void encode_q4_kernel(const float *__restrict__ W, int out, int in, int T,
                                                                uint8_t *__restrict__ codes,
                                                                uint16_t *__restrict__ scales,
                                                                uint8_t *__restrict__ zeros, int32_t *status) {
    const int lane16 = threadIdx.x & 15;
    const uint32_t groups = (uint32_t)out * (uint32_t)T;
    const uint32_t per_pass = gridDim.x * (Q4E_THREADS / 16);
    const uint32_t first = blockIdx.x * (Q4E_THREADS / 16) + (threadIdx.x >> 4);
    bool broken = false;
    // (every lane takes the same turns: the rows of 16 lanes exchange values)
    for (uint32_t g0 = 0; g0 < groups; g0 += per_pass * Q4E_AHEAD) {
        float4 v[Q4E_AHEAD][2];
        uint32_t row[Q4E_AHEAD], t[Q4E_AHEAD];
        bool here[Q4E_AHEAD];
#pragma unroll
        for (int i = 0; i < Q4E_AHEAD; ++i) {
            const uint64_t g = (uint64_t)g0 + (uint64_t)i * per_pass + first;
            row[i] = g < groups ? (uint32_t)g / (uint32_t)T : 0;
            t[i] = (uint32_t)g - row[i] * (uint32_t)T;
            here[i] = g < groups && (int64_t)t[i] * 128 + lane16 * 8 < in;
            v[i][0] = v[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (here[i]) {
                const float4 *p = (const float4 *)(W + (int64_t)row[i] * in + (int64_t)t[i] * 128 + lane16 * 8);
                v[i][0] = p[0];
                v[i][1] = p[1];
            }
        }
#pragma unroll
        for (int i = 0; i < Q4E_AHEAD; ++i) {
            const float w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
            float hi = 0.0f, lo = 0.0f;     // lo: of -w
            bool odd = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                hi = fmaxf(hi, ZEROS ? w[j] : __builtin_fabsf(w[j]));
                lo = fmaxf(lo, -w[j]);
                odd |= !(__builtin_fabsf(w[j]) < __builtin_inff());
            }
            hi = row_max(hi);
            if (ZEROS)
                lo = row_max(lo);
            const bool bad = (__ballot(odd) >> (threadIdx.x & 48) & 0xFFFF) != 0;
            float want = ZEROS ? (hi + lo) / 15.0f : hi / 7.0f;
            want = fminf(fmaxf(want, 5.9604644775390625e-8f), 65504.0f);
            const uint16_t s16 = bad ? 0x7E00 : f2h(want);
            const float s = h2f(bad ? 0x3C00 : s16);
            const float z = ZEROS ? fminf(__builtin_rintf(lo / s), 15.0f) : 8.0f;
            uint32_t packed = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c = fminf(fmaxf(__builtin_rintf(w[j] / s) + z, 0.0f), 15.0f);
                packed |= (uint32_t)c << (4 * j);
            }
            if (here[i]) {
                const int64_t at = (int64_t)row[i] * (in / 2) + (int64_t)t[i] * 64 + lane16 * 4;
                *(uint32_t *)(codes + at) = bad ? 0u : packed;
                if (lane16 == 0) {
                    scales[(int64_t)row[i] * T + t[i]] = s16;
                    if (ZEROS)
                        zeros[(int64_t)row[i] * T + t[i]] = bad ? 0 : (uint8_t)z;
                    broken |= bad;
                }
            }
        }
    }
    if (broken && status != nullptr)
        atomicOr(status, RBQ_STATUS_NONFINITE_W);
}

// ---------------------------------------------------------------------------
// few tokens: a workgroup takes 16 NT rows and 16 tokens; each of its waves takes
// one group at a time, the next two on their way, and goes through the row tiles
// with the tokens' operands of that group.  A lane holds one row's 32 columns of a
// group in one 16-byte load, which four matrix instructions take apart; a group's
// sums are scaled and added in fp32, the waves' sums in their order.  The rows'
// scales and zero points pass through LDS (STAGED) where they fit: read by the lanes
// that use them, 2 bytes of 16 lines each, they took as long as half of the codes
// (11008 x 4096, one token: 9.9 us with, 7.7 without their loads).
//
// Up to 4 tokens (FEW) a group of them is one load, and the four operands of 8
// columns that a lane would hold for its token are held by four lanes: row 4 m + q of
// the matrix instruction is part q of token m.  Of its product with part q' of the
// codes row 4 m + q' counts, which is result q' of lanes 16 m .. 16 m + 15, so the
// sum over q' needs four instructions, as before, and three additions.
//
// More tokens go to the operands' order through a wave's own 4 KB of LDS: loaded in
// that order, 16 bytes of 64 places each, they bounded the kernel (16 tokens: 11008 x
// 4096 10.6 us so, 9.8 side by side; 4096 x 11008 15.9 and 12.4).  Eight waves: 16 are
// faster on long rows (4096 x 11008, one token: 7.1 us against 8.4) and slower on many
// (11008 x 4096: 8.0 and 7.3; 128256 x 4096: 70 and 53), 4 slower everywhere but there.
// From HBM, device time, one token: 4096 x 4096 4.6 us, 11008 x 4096 7.3 (3.1 TB/s),
// 28672 x 8192 26.0 (4.5 TB/s), 128256 x 4096 54 (4.9 TB/s): bytes, and on the smaller
// layers the start and end of one round of workgroups.
constexpr int Q4_WAVES = 8;

typedef uint32_t q4_bytes16 __attribute__((ext_vector_type(4), aligned(1)));

// n bytes to LDS (any alignment in memory, 16 bytes' in LDS).
__device__ __forceinline__ void q4_stage(const void *from, uint8_t *to, int n) {
    const uint8_t *p = (const uint8_t *)from;
    for (int i = threadIdx.x * 16; i + 16 <= n; i += Q4_WAVES * 64 * 16)
        *(uint4 *)(to + i) = __builtin_bit_cast(uint4, *(const q4_bytes16 *)(p + i));
    const int rest = n & 15;
    if ((int)threadIdx.x < rest)
        to[n - rest + threadIdx.x] = p[n - rest + threadIdx.x];
}

template <int NT, bool FEW, bool STAGED, bool ZEROS, bool WIDE>
__global__ __launch_bounds__(Q4_WAVES * 64) void gemm_q4_few_kernel(const uint8_t *__restrict__ codes,
                                                                    const uint16_t *__restrict__ scales,
                                                                    const uint8_t *__restrict__ zeros, int out, int in,
                                                                    int T, const uint16_t *__restrict__ X, int M,
                                                                    void *__restrict__ Y) {
    constexpr int W = Q4_WAVES, PARTS = FEW ? 1 : 4;
    // (the waves' tokens, then their sums)
    constexpr int SUMS = W * NT * PARTS * 64 * (int)sizeof(float), TOKENS = FEW ? 0 : W * 4096;
    __shared__ __align__(16) uint8_t shared[SUMS > TOKENS ? SUMS : TOKENS];
    auto part = (float(*)[NT][PARTS][64])shared;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, kb = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.x * (16 * NT), m0 = (int64_t)blockIdx.y * 16;
    const int tokens = (int)min((int64_t)16, M - m0);
    X += m0 * in;
    // (rows past the end repeat the last one; 32-bit offsets from the first row)
    const int last = (int)min((int64_t)16 * NT - 1, (int64_t)out - 1 - r0);
    const uint16_t *ls = STAGED ? (const uint16_t *)lds : scales + r0 * T;
    const uint8_t *lz = STAGED ? lds + q4_staged_scales(16 * NT, T) : zeros + (ZEROS ? r0 * T : 0);
    const uint8_t *wbase = codes + r0 * (in / 2);
    uint32_t woff[NT], at_scale[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int row = min(16 * i + li, last);
        woff[i] = (uint32_t)row * (uint32_t)(in / 2);
        at_scale[i] = (uint32_t)row * (uint32_t)T;
    }
    constexpr int XL = FEW ? 1 : 4;
    // 16 lanes load a token's 128 columns: FEW, in the operand's order already; else
    // tokens 4 q + kb, side by side, and through LDS to the order
    const int xm = FEW ? li >> 2 : kb, xc = FEW ? kb * 32 + (li & 3) * 8 : li * 8;
    // groups in flight; two take turns
    struct {
        uint4 w[NT], x[XL];
    } load[2];
    auto request = [&](int t, int b) __attribute__((always_inline)) {
        if (t >= T)
            return;
        // (past a row's end: any codes, the tokens are 0 there)
        const uint32_t at = (uint32_t)min(t * 64 + kb * 16, in / 2 - 16);
#pragma unroll
        for (int i = 0; i < NT; ++i)
            load[b].w[i] = *(const uint4 *)(wbase + (woff[i] + at));
        const int column = t * 128 + xc;
#pragma unroll
        for (int q = 0; q < XL; ++q) {
            load[b].x[q] = make_uint4(0, 0, 0, 0);
            if (xm + 4 * q < tokens && column < in)
                load[b].x[q] = *(const uint4 *)(X + (int64_t)(xm + 4 * q) * in + column);
        }
    };
    const q4_bits bits;
    float acc[NT][PARTS] = {};
    auto compute = [&](int t, int b) __attribute__((always_inline)) {
        if (t >= T)
            return;
        q4_f16x8 a[4];
        if constexpr (FEW) {
            a[0] = q4_order(load[b].x[0]);
        } else {
            // (a wave's own 4 KB, in its order: no barrier; the 16-byte pieces of a
            // token change places by its number, which spreads them over the banks)
            uint4 *mine = (uint4 *)(shared + wave * 4096);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                mine[(4 * q + kb) * 16 + (li ^ (4 * q + kb))] = load[b].x[q];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                a[q] = q4_order(mine[li * 16 + ((kb * 4 + q) ^ li)]);
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            q4_f16x8 w[4];
            q4_unpack(bits, load[b].w[i], ZEROS ? lz[at_scale[i] + t] : 8, w);
            const float by = h2f(ls[at_scale[i] + t]);
            const q4_f32x4 none = {};
            if constexpr (FEW) {
                float g = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const q4_f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[0], w[q], none, 0, 0, 0);
                    g = q == 0 ? d[0] : g + d[q];
                }
                acc[i][0] = __builtin_fmaf(g, by, acc[i][0]);
            } else {
                q4_f32x4 g = none;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    g = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[q], w[q], g, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[i][k] = __builtin_fmaf(g[k], by, acc[i][k]);
            }
        }
    };
    int t = wave;
    request(t, 0);
    if (STAGED) {
        q4_stage(scales + r0 * T, lds, (last + 1) * T * 2);
        if (ZEROS)
            q4_stage(zeros + r0 * T, lds + q4_staged_scales(16 * NT, T), (last + 1) * T);
    }
    request(t + W, 1);
    if (STAGED)
        __syncthreads();
    for (; t < T; t += 2 * W) {
        compute(t, 0);
        request(t + 2 * W, 0);
        compute(t + W, 1);
        request(t + 3 * W, 1);
    }
    if (!FEW)
        __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int k = 0; k < PARTS; ++k)
            part[wave][i][k][lane] = acc[i][k];
    __syncthreads();
    for (int q = threadIdx.x; q < tokens * 16 * NT; q += W * 64) {
        // (16 NT rows of a token side by side)
        const int r = q % (16 * NT), token = q / (16 * NT);
        const int l = (FEW ? token : token >> 2) * 16 + (r & 15), k = FEW ? 0 : token & 3;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i)
            y += part[i][r >> 4][k][l];
        if (r0 + r < out) {
            const int64_t at = (m0 + token) * out + r0 + r;
            if (WIDE)
                ((float *)Y)[at] = y;
            else
                ((uint16_t *)Y)[at] = f2h(y);
        }
    }
}

}  // namespace

hipError_t launch_encode_q4(const float *W, int out, int in, uint8_t *codes, uint16_t *scales, uint8_t *zeros,
                            int32_t *status, hipStream_t st) {
    const int T = (in + 127) / 128;
    const int64_t groups = (int64_t)out * T;
    const int64_t want = (groups + Q4E_THREADS / 16 * Q4E_AHEAD - 1) / (Q4E_THREADS / 16 * Q4E_AHEAD);
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : (1 << 20));
    if (zeros != nullptr)
        encode_q4_kernel<true><<<grid, Q4E_THREADS, 0, st>>>(W, out, in, T, codes, scales, zeros, status);
    else
        encode_q4_kernel<false><<<grid, Q4E_THREADS, 0, st>>>(W, out, in, T, codes, scales, nullptr, status);
    return hipGetLastError();
}

hipError_t launch_gemm_q4(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int out, int in,
                          const uint16_t *X, int M, void *Y, int y_f32, void *workspace, size_t ws_bytes,
                          hipStream_t st) {
    if (q4_tiled(out, in, M))
        return launch_gemm_q4_tile(codes, scales, zeros, out, in, X, M, Y, y_f32, workspace, ws_bytes, st);
    const int T = (in + 127) / 128;
    using std::bool_constant;
    auto run = [&](auto nt, auto few, auto staged, auto zero, auto wide) {
        constexpr int NT = decltype(nt)::value;
        constexpr bool STAGED = decltype(staged)::value, ZEROS = decltype(zero)::value;
        const int64_t across = ((int64_t)out + 16 * NT - 1) / (16 * NT);
        const size_t lds = STAGED ? q4_staged_scales(16 * NT, T) + (ZEROS ? (size_t)(16 * NT) * T : 0) : 0;
        // (a grid's second axis ends at 65535)
        constexpr int64_t TOKENS = 65535 * 16;
        for (int64_t m = 0; m < M; m += TOKENS) {
            const int n = (int)std::min<int64_t>(M - m, TOKENS);
            const dim3 grid((unsigned)across, (unsigned)((n + 15) / 16));
            gemm_q4_few_kernel<NT, decltype(few)::value, STAGED, ZEROS, decltype(wide)::value>
                <<<grid, Q4_WAVES * 64, lds, st>>>(codes, scales, zeros, out, in, T, X + m * in, n,
                                                   (uint8_t *)Y + m * out * (decltype(wide)::value ? 4 : 2));
        }
    };
    auto typed = [&](auto nt, auto few, auto staged) {
        auto zeroed = [&](auto zero) {
            y_f32 ? run(nt, few, staged, zero, bool_constant<true>{}) : run(nt, few, staged, zero, bool_constant<false>{});
        };
        zeros != nullptr ? zeroed(bool_constant<true>{}) : zeroed(bool_constant<false>{});
    };
    constexpr std::integral_constant<int, 1> one;
    constexpr std::integral_constant<int, 2> two;
    constexpr std::integral_constant<int, 3> three;
    constexpr bool_constant<true> yes;
    constexpr bool_constant<false> no;
    const q4_few_plan p = plan_q4_few(out, in, M);
    if (p.four)
        p.staged ? typed(one, yes, yes) : typed(one, yes, no);
    else if (!p.staged)
        typed(one, no, no);
    else
        p.row_tiles == 1 ? typed(one, no, yes) : p.row_tiles == 2 ? typed(two, no, yes) : typed(three, no, yes);
    return hipGetLastError();
}

}  // namespace rbq
