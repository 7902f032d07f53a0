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
// encoder: 16 lanes hold a group (8 consecutive weights each), four groups a
// lane at a time.  W is read once; bound by that read.
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
// few tokens: a workgroup takes 16 rows and up to 16 MT tokens, its waves split
// the columns in chunks of 512.  A lane holds one row's 32 columns of a group in
// one 16-byte load, which four matrix instructions take apart; a group's sums
// are scaled and added in fp32.

constexpr int Q4_WAVES = 8, Q4_AHEAD = 4;

template <int MT, bool ZEROS, bool WIDE>
__global__ __launch_bounds__(Q4_WAVES * 64) void gemm_q4_few_kernel(const uint8_t *__restrict__ codes,
                                                                    const uint16_t *__restrict__ scales,
                                                                    const uint8_t *__restrict__ zeros, int out, int in,
                                                                    int T, const uint16_t *__restrict__ X, int M,
                                                                    void *__restrict__ Y) {
    __shared__ q4_f32x4 part[Q4_WAVES][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r0 = blockIdx.x * 16, m0 = blockIdx.y * (16 * MT);
    const int row = min(r0 + (lane & 15), out - 1), kb = lane >> 4;
    const uint8_t *w = codes + (int64_t)row * (in / 2) + kb * 16;
    const uint16_t *s = scales + (int64_t)row * T;
    const uint8_t *z = ZEROS ? zeros + (int64_t)row * T : nullptr;
    const uint16_t *x[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        x[i] = X + (int64_t)min(m0 + 16 * i + (lane & 15), M - 1) * in + kb * 32;
    const q4_bits bits;
    q4_f32x4 acc[MT] = {};
    for (int t0 = wave * Q4_AHEAD; t0 < T; t0 += Q4_WAVES * Q4_AHEAD) {
        uint4 raw[Q4_AHEAD];
        float sc[Q4_AHEAD];
        int zp[Q4_AHEAD];
#pragma unroll
        for (int i = 0; i < Q4_AHEAD; ++i) {
            const int t = t0 + i;
            const bool here = t < T && t * 128 + kb * 32 < in;
            raw[i] = here ? *(const uint4 *)(w + (int64_t)t * 64) : make_uint4(0, 0, 0, 0);
            sc[i] = t < T ? h2f(s[t]) : 0.0f;
            zp[i] = ZEROS ? (t < T ? z[t] : 0) : 8;
        }
#pragma unroll
        for (int i = 0; i < Q4_AHEAD; ++i) {
            const int t = t0 + i;
            if (t >= T)
                break;
            const bool here = t * 128 + kb * 32 < in;
            q4_f16x8 b[4];
            q4_unpack(bits, raw[i], zp[i], b);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                q4_f32x4 g = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 v = here ? *(const uint4 *)(x[mt] + (int64_t)t * 128 + j * 8) : make_uint4(0, 0, 0, 0);
                    g = __builtin_amdgcn_mfma_f32_16x16x32_f16(q4_order(v), b[j], g, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[mt][k] = __builtin_fmaf(g[k], sc[i], acc[mt][k]);
            }
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        part[wave][mt][lane] = acc[mt];
    __syncthreads();
    for (int q = threadIdx.x; q < MT * 256; q += Q4_WAVES * 64) {
        const int mt = q >> 8, k = q >> 6 & 3, l = q & 63;
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < Q4_WAVES; ++i)
            y += part[i][mt][l][k];
        const int m = m0 + 16 * mt + (l >> 4) * 4 + k, r = r0 + (l & 15);
        if (m < M && r < out) {
            if (WIDE)
                ((float *)Y)[(int64_t)m * out + r] = y;
            else
                ((uint16_t *)Y)[(int64_t)m * out + r] = f2h(y);
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
    auto run = [&](auto mt, auto wide, auto zero) {
        constexpr int MT = decltype(mt)::value;
        const dim3 grid((unsigned)((out + 15) / 16), (unsigned)((M + 16 * MT - 1) / (16 * MT)));
        gemm_q4_few_kernel<MT, decltype(zero)::value, decltype(wide)::value>
            <<<grid, Q4_WAVES * 64, 0, st>>>(codes, scales, zeros, out, in, T, X, M, Y);
    };
    auto typed = [&](auto mt) {
        using std::bool_constant;
        if (y_f32)
            zeros != nullptr ? run(mt, bool_constant<true>{}, bool_constant<true>{})
                             : run(mt, bool_constant<true>{}, bool_constant<false>{});
        else
            zeros != nullptr ? run(mt, bool_constant<false>{}, bool_constant<true>{})
                             : run(mt, bool_constant<false>{}, bool_constant<false>{});
    };
    if (M <= 16)
        typed(std::integral_constant<int, 1>{});
    else
        typed(std::integral_constant<int, 4>{});
    return hipGetLastError();
}

}  // namespace rbq
