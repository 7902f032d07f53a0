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
// dW[r][j] = sum_m dY[m][r] x^[m][j] on v_mfma_f32_16x16x32_f16: 128 x 128
// tiles, 32 tokens per step staged through LDS transposed.

constexpr int CW_THREADS = 256;
constexpr int CW_TILE = 128;
constexpr int CW_BK = 32;
constexpr int CW_LDP = CW_BK + 8;

__global__ __launch_bounds__(CW_THREADS) void qat_ckpt_dw_kernel(const uint16_t *__restrict__ dY,
                                                                 const int8_t *__restrict__ codes,
                                                                 const uint16_t *__restrict__ cscales, int M,
                                                                 int out, int in, int T, float *__restrict__ dW) {
    __shared__ __align__(16) _Float16 As[CW_TILE * CW_LDP];   // [dW row][token]
    __shared__ __align__(16) _Float16 Bs[CW_TILE * CW_LDP];   // [column][token]
    const int tid = threadIdx.x;
    const int lane = tid & (RBQ_WAVE - 1);
    const int wave = tid / RBQ_WAVE;
    const int wr = wave & 1, wc = wave >> 1;
    const int li = lane & 15, lg = lane >> 4;
    const int64_t r0 = (int64_t)blockIdx.y * CW_TILE, j0 = (int64_t)blockIdx.x * CW_TILE;
    const int mm = tid & 31, q = tid >> 5;    // staging: 16 values of token mm

    v4f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

    for (int64_t m0 = 0; m0 < M; m0 += CW_BK) {
        const int64_t m = m0 + mm;
        uint16_t a[16];
        v2h b[8];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            a[i] = m < M && r0 + 16 * q + i < out ? dY[m * out + r0 + 16 * q + i] : (uint16_t)0;
        const int64_t c = j0 + 16 * q;
        if (m < M && c < in) {
            const uint4 u = *reinterpret_cast<const uint4 *>(codes + m * in + c);
            const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
            const _Float16 s1 = __builtin_bit_cast(_Float16, cscales[m * T + c / F8_BLOCK]);
            const v2h s = {s1, s1};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b[2 * i] = ckpt_pair<0>(w[i], s);
                b[2 * i + 1] = ckpt_pair<1>(w[i], s);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                b[i] = (v2h){(_Float16)0.0f, (_Float16)0.0f};
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            As[(16 * q + i) * CW_LDP + mm] = __builtin_bit_cast(_Float16, a[i]);
            Bs[(16 * q + i) * CW_LDP + mm] = b[i / 2][i & 1];
        }
        __syncthreads();
        v8h af[4], bf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            af[i] = *reinterpret_cast<const v8h *>(&As[(64 * wr + i * 16 + li) * CW_LDP + 8 * lg]);
            bf[i] = *reinterpret_cast<const v8h *>(&Bs[(64 * wc + i * 16 + li) * CW_LDP + 8 * lg]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af[i], bf[j], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = j0 + 64 * wc + 16 * j + li;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t r = r0 + 64 * wr + 16 * i + 4 * lg + v;
                if (r < out && c < in)
                    dW[r * in + c] = acc[i][j][v];
            }
        }
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

hipError_t launch_qat_backward_ckpt(const uint32_t *planes, const uint16_t *scales, int out, int in, int K,
                                    int group_size, const int8_t *x_codes, const uint16_t *x_scales,
                                    const uint16_t *dY, int M, float *dX, float *dW, float *dscales,
                                    void *workspace, size_t ws_bytes, int32_t *status, hipStream_t st) {
    hipError_t e = hipSuccess;
    if (dW != nullptr) {
        const dim3 grid((unsigned)((in + CW_TILE - 1) / CW_TILE), (unsigned)(((int64_t)out + CW_TILE - 1) / CW_TILE));
        hipLaunchKernelGGL(qat_ckpt_dw_kernel, grid, dim3(CW_THREADS), 0, st, dY, x_codes, x_scales, M, out, in,
                           f8_blocks(in), dW);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    if (dscales != nullptr && (e = launch_qat_dscales(planes, out, in, K, group_size, dW, dscales, st)) != hipSuccess)
        return e;
    if (dX != nullptr)
        e = launch_qat_backward(planes, scales, out, in, K, group_size, nullptr, dY, M, dX, nullptr, nullptr,
                                workspace, ws_bytes, status, st);
    return e;
}

}  // namespace rbq
