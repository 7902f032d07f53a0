// f8.hip -- 8-bit floating point blocks of 128: the weight encoder, the token
// quantiser and the products for one and few tokens.
//
// A value is code * scale with an OCP e4m3 code (4 significant bits, at most
// 448) and one fp32 scale per block of 128 x 128 weights, or per block of 128
// columns of one token.  For a block with A = max |v| (at least 2^-100, so
// that 448 / A is finite and an all-zero block needs no case of its own):
//   scale = fl32(A / 448),  code = e4m3(fl32(v * fl32(448 / A)))
// each rounded to nearest even.  The largest entry takes code +-448; a block
// with a NaN or infinite entry has scale NaN and codes 0.
#include <algorithm>

#include "rbq.h"
#include "rbq_device.h"
#include "rbq_kernels.h"
#include "f8_device.h"
#include "f8_plan.h"

namespace rbq {

namespace {

constexpr int FQ_THREADS = 256;

// ---------------------------------------------------------------------------
// tokens: 16 lanes hold one block (8 consecutive fp16 each, one 16-byte load),
// so the maximum is four DPP rotations inside a row of 16 lanes and needs no
// LDS.  A workgroup takes 16 tokens x 4 blocks, the four loads of a lane issued
// together, or 1 x 16, one block a lane, which takes less time from the load to
// the codes.  Bound by the read of X and the write of the codes: 2048 x 14336
// takes 15.4 us, 5.8 TB/s, over three inputs in turn, which the 256 MB cache
// holds in part; 18.3 us, 4.8 TB/s, over eight (705 MB), and 26 us where X has
// to come past another kernel's unwritten lines.

template <int B>
__global__ __launch_bounds__(FQ_THREADS) void quantize_f8_kernel(const uint16_t *__restrict__ X, int M, int in,
                                                                 int T, uint8_t *__restrict__ codes,
                                                                 float *__restrict__ scales) {
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
            const uint32_t top = row16_max_u32(absmax8_f16(v[b]));
            float scale, inv;
            f8_scale_f16(top, scale, inv);
            if (c < in)
                *reinterpret_cast<uint2 *>(codes + m * in + c) = f8_codes8(v[b], inv);
            if (li == 0 && t0 + b < T)
                scales[(int64_t)(t0 + b) * M + m] = scale;
        }
    }
}

// ---------------------------------------------------------------------------
// weights: one workgroup per 128 x 128 block, held in 64 registers per thread
// between the maximum and the codes, so W is read once.  Bound by that read:
// 14336 x 4096 takes 53.5 us, 5.5 TB/s of W and codes (three inputs in turn are
// 880 MB: from HBM).

__global__ __launch_bounds__(FQ_THREADS) void encode_f8_kernel(const float *__restrict__ W, int out, int in, int T,
                                                               uint8_t *__restrict__ codes,
                                                               float *__restrict__ scales,
                                                               int32_t *__restrict__ status) {
    __shared__ uint32_t part[FQ_THREADS / RBQ_WAVE];
    const int t = blockIdx.x % T, rb = blockIdx.x / T;
    const int64_t c = (int64_t)t * F8_BLOCK + 4 * (threadIdx.x & 31);
    const int64_t r0 = (int64_t)rb * F8_BLOCK + (threadIdx.x >> 5);
    uint4 v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t r = r0 + 8 * i;
        v[i] = r < out && c < in ? *reinterpret_cast<const uint4 *>(W + r * in + c) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t a = max(v[i].x & 0x7FFFFFFFu, v[i].y & 0x7FFFFFFFu);
        const uint32_t b = max(v[i].z & 0x7FFFFFFFu, v[i].w & 0x7FFFFFFFu);
        top = max(top, max(a, b));
    }
    top = wave_max_u32_dpp(top);
    if ((threadIdx.x & (RBQ_WAVE - 1)) == 0)
        part[threadIdx.x / RBQ_WAVE] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    float scale, inv;
    f8_scale_f32(top, scale, inv);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t r = r0 + 8 * i;
        if (r < out && c < in) {
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(__uint_as_float(v[i].x) * inv, __uint_as_float(v[i].y) * inv,
                                                    0, false);
            p = __builtin_amdgcn_cvt_pk_fp8_f32(__uint_as_float(v[i].z) * inv, __uint_as_float(v[i].w) * inv, p,
                                                true);
            *reinterpret_cast<uint32_t *>(codes + r * in + c) = inv == 0.0f ? 0u : (uint32_t)p;
        }
    }
    if (threadIdx.x == 0) {
        scales[(int64_t)rb * T + t] = scale;
        if (status != nullptr && inv == 0.0f)
            atomicOr(status, (int)RBQ_STATUS_NONFINITE_W);
    }
}

// ---------------------------------------------------------------------------
// one and few tokens: 16 rows of W on one side of the matrix instruction, 16
// tokens on the other.  The codes are converted to fp16 (exact) after the
// load and the sums of a block are fp32: here the read of W is what bounds,
// and the conversions and the slower instruction hide behind it.  The four
// sums of a lane take their two scales in four fmas per block.  The waves of
// a workgroup split the blocks of 16 rows and add their partial sums through
// LDS in wave order (the same order in every run).  Lane (i, g) holds bytes
// 16g.. and 64 + 16g.. of row i of both operands: any assignment of columns
// gives the same sum as long as both sides share it, and this one makes a
// load 64 contiguous bytes per row.
//
// Over 640 MB of layers in turn, so that W comes from HBM: one token, 11008 x
// 4096: 11.1 us, 4.1 TB/s of W; 32000 x 4096: 26.2 us, 5.0 TB/s; 16 tokens, 4096 x
// 11008: 15.1 us, 3.0 TB/s (the tokens' 176 KB are read by each of the 256
// workgroups).  Three layers in turn, which stay in the 256 MB cache: 9.9 and
// 13.3 us for the first and the last.

// Every wave keeps U blocks in flight: the loads of block u + U of its own are
// issued as soon as block u's registers are free.

// The 32 bytes of lane group g of block t of a row.  Pieces past its end are
// read from its first bytes, so that every load is unconditional, and are
// taken as zero by f8_cut once they are used.
struct f8_bytes {
    uint4 lo, hi;
};

__device__ __forceinline__ f8_bytes f8_load(const uint8_t *__restrict__ row, int t, int g, int in) {
    const int64_t c = (int64_t)t * F8_BLOCK + 16 * g;
    return {*reinterpret_cast<const uint4 *>(row + (c < in ? c : 0)),
            *reinterpret_cast<const uint4 *>(row + (c + 64 < in ? c + 64 : 0))};
}

__device__ __forceinline__ void f8_cut(f8_bytes &f, int t, int g, int in) {
    const int64_t c = (int64_t)t * F8_BLOCK + 16 * g;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    if (c >= in)
        f.lo = z;
    if (c + 64 >= in)
        f.hi = z;
}

__device__ __forceinline__ void f8_halves(const f8_bytes &f, v8h (&h)[4]) {
    h[0] = f8_to_f16((int)f.lo.x, (int)f.lo.y);
    h[1] = f8_to_f16((int)f.lo.z, (int)f.lo.w);
    h[2] = f8_to_f16((int)f.hi.x, (int)f.hi.y);
    h[3] = f8_to_f16((int)f.hi.z, (int)f.hi.w);
}

// Every workgroup begins at another block of its rows (the XCD's neighbours
// one block further each): in step, they would all read the same few blocks of
// the tokens, and rows whose length is a multiple of 4096 bytes, from the same
// channels of the L2.
__device__ __forceinline__ int f8_turn(int t, int turn, int T) { return t + turn < T ? t + turn : t + turn - T; }

// The RT x NT tiles of every wave, added in wave order and written: row tile
// i, token tile j of lane (li, g) are rows 16 i + 4 g + v and token 16 j + li.
template <int RT, int NT, int WAVES, typename Y>
__device__ __forceinline__ void f8_join(float *part, const v4f (&acc)[RT][NT], int wave, int lane, int64_t r0,
                                        int out, int64_t m0, int M, Y *__restrict__ y) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<v4f *>(&part[(((i * NT + j) * WAVES + wave) * RBQ_WAVE + lane) * 4]) = acc[i][j];
    __syncthreads();
    for (int q = wave; q < RT * NT; q += WAVES) {
        v4f s = *reinterpret_cast<const v4f *>(&part[(q * WAVES * RBQ_WAVE + lane) * 4]);
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            s += *reinterpret_cast<const v4f *>(&part[((q * WAVES + w) * RBQ_WAVE + lane) * 4]);
        const int64_t m = m0 + 16 * (q % NT) + (lane & 15);
        const int64_t r = r0 + 16 * (q / NT) + 4 * (lane >> 4);
        if (m < M)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (r + v < out)
                    y[m * out + r + v] = to_y<Y>(s[v]);
    }
}

template <int RT, int NT, int WAVES, int U, typename Y>
__global__ __launch_bounds__(WAVES *RBQ_WAVE) void gemm_f8_few_kernel(
    const uint8_t *__restrict__ W, const float *__restrict__ ws, int out, int in, int T,
    const uint8_t *__restrict__ X, const float *__restrict__ xs, int M, int64_t groups, Y *__restrict__ y) {
    __shared__ __align__(16) float part[RT * NT * WAVES * RBQ_WAVE * 4];
    const int lane = threadIdx.x & (RBQ_WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / RBQ_WAVE));
    const int li = lane & 15, g = lane >> 4;
    const int full = in / F8_BLOCK;
    const int64_t r0 = (int64_t)blockIdx.x * (16 * RT);
    const uint8_t *wrow[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)                                          // rows past the last: not written
        wrow[i] = W + std::min(r0 + 16 * i + li, (int64_t)out - 1) * in;
    const float *wsr = ws + r0 / F8_BLOCK * T;
    const int n = wave < T ? (T - wave + WAVES - 1) / WAVES : 0;          // blocks of this wave
    const int turn = (int)((blockIdx.x >> 3) % (unsigned)T);
    for (int64_t gr = blockIdx.y; gr < groups; gr += gridDim.y) {
        const int64_t m0 = gr * (16 * NT);
        const uint8_t *xrow[NT];
        int64_t mi[NT];
        v4f acc[RT][NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            mi[j] = std::min(m0 + 16 * j + li, (int64_t)M - 1);
            xrow[j] = X + mi[j] * in;
#pragma unroll
            for (int i = 0; i < RT; ++i)
                acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        }
        f8_bytes wb[U][RT], xb[U][NT];
        float sw[U], sx[U][NT];
        auto load = [&](int u, int q) {
            const int t = f8_turn(std::min(wave + q * WAVES, T - 1), turn, T);
#pragma unroll
            for (int i = 0; i < RT; ++i)
                wb[u][i] = f8_load(wrow[i], t, g, in);
            sw[u] = wsr[t];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                xb[u][j] = f8_load(xrow[j], t, g, in);
                sx[u][j] = xs[(int64_t)t * M + mi[j]];
            }
        };
        auto add = [&](int u, int q) {
            if (full < T && f8_turn(wave + q * WAVES, turn, T) == full) {   // the block that the row's end cuts
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    f8_cut(wb[u][i], full, g, in);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    f8_cut(xb[u][j], full, g, in);
            }
            v8h a[RT][4], b[4];
#pragma unroll
            for (int i = 0; i < RT; ++i)
                f8_halves(wb[u][i], a[i]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                f8_halves(xb[u][j], b);
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    acc[i][j] = f8_fma(f8_mma(a[i], b), sw[u] * sx[u][j], acc[i][j]);
            }
        };
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < n)
                load(u, u);
        int q = 0;
        for (; q + U < n; q += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                add(u, q + u);
                load(u, q + U + u);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (q + u >= n)
                break;
            add(u, q + u);
        }
        f8_join<RT, NT, WAVES, Y>(part, acc, wave, lane, r0, out, m0, M, y);
        __syncthreads();                     // the partial sums are read before the next group's
    }
}

// One fp16 token, quantised by the wave that needs the block: lane l holds
// columns 2l and 2l + 1, the maximum is a DPP reduction over the wave, and
// the 128 codes pass through 128 bytes of LDS of the wave's own.  Only token
// column 0 of the product is written; the other 15 repeat it.
template <int WAVES, int U>
__global__ __launch_bounds__(WAVES *RBQ_WAVE) void gemv_f8_kernel(const uint8_t *__restrict__ W,
                                                                  const float *__restrict__ ws, int out, int in,
                                                                  int T, const uint16_t *__restrict__ x,
                                                                  uint16_t *__restrict__ y) {
    __shared__ __align__(16) float part[WAVES * RBQ_WAVE * 4];
    __shared__ __align__(16) uint16_t xq[WAVES][U][F8_BLOCK / 2];
    const int lane = threadIdx.x & (RBQ_WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / RBQ_WAVE));
    const int li = lane & 15, g = lane >> 4;
    const int full = in / F8_BLOCK;
    const int64_t r0 = (int64_t)blockIdx.x * 16;
    const uint8_t *wrow = W + std::min(r0 + li, (int64_t)out - 1) * in;
    const float *wsr = ws + r0 / F8_BLOCK * T;
    v4f acc[1][1] = {{(v4f){0.0f, 0.0f, 0.0f, 0.0f}}};
    f8_bytes wb[U];
    uint32_t xv[U];
    float sw[U];
    const int n = wave < T ? (T - wave + WAVES - 1) / WAVES : 0;
    const int turn = (int)((blockIdx.x >> 3) % (unsigned)T);
    auto load = [&](int u, int i) {
        const int t = f8_turn(std::min(wave + i * WAVES, T - 1), turn, T);
        const int64_t c = (int64_t)t * F8_BLOCK + 2 * lane;
        xv[u] = *reinterpret_cast<const uint32_t *>(x + (c < in ? c : 0));
        sw[u] = wsr[t];
        wb[u] = f8_load(wrow, t, g, in);
    };
    auto add = [&](int u, int i) {
        if (full < T && f8_turn(wave + i * WAVES, turn, T) == full) {
            f8_cut(wb[u], full, g, in);
            if ((int64_t)full * F8_BLOCK + 2 * lane >= in)
                xv[u] = 0u;
        }
        const uint32_t v = xv[u];
        const uint32_t top = wave_max_u32_dpp(max(v & 0x7FFFu, (v >> 16) & 0x7FFFu));
        float sx, inv;
        f8_scale_f16(top, sx, inv);
        const int p = __builtin_amdgcn_cvt_pk_fp8_f32(h2f((uint16_t)v) * inv, h2f((uint16_t)(v >> 16)) * inv, 0,
                                                      false);
        // each wave writes and reads 128 bytes of its own, in order
        xq[wave][u][lane] = inv == 0.0f ? (uint16_t)0 : (uint16_t)p;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const f8_bytes xb = {*reinterpret_cast<const uint4 *>(&xq[wave][u][8 * g]),
                             *reinterpret_cast<const uint4 *>(&xq[wave][u][32 + 8 * g])};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        v8h a[4], b[4];
        f8_halves(wb[u], a);
        f8_halves(xb, b);
        acc[0][0] = f8_fma(f8_mma(a, b), sw[u] * sx, acc[0][0]);
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
        load(u, u);                       // (past this wave's last block: the row's last one again)
    int i = 0;
    for (; i + U < n; i += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            add(u, i + u);
            load(u, i + U + u);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (i + u >= n)
            break;
        add(u, i + u);
    }
    f8_join<1, 1, WAVES, uint16_t>(part, acc, wave, lane, r0, out, 0, 1, y);
}

template <int RT, int NT, int WAVES, int U, typename Y>
hipError_t launch_few(const uint8_t *W, const float *ws, int out, int in, const uint8_t *X, const float *xs, int M,
                      Y *y, hipStream_t st) {
    const int64_t groups = ((int64_t)M + 16 * NT - 1) / (16 * NT);
    const dim3 grid((unsigned)(((int64_t)out + 16 * RT - 1) / (16 * RT)), (unsigned)std::min<int64_t>(groups, 65535));
    hipLaunchKernelGGL((gemm_f8_few_kernel<RT, NT, WAVES, U, Y>), grid, dim3(WAVES * RBQ_WAVE), 0, st, W, ws, out, in,
                       f8_blocks(in), X, xs, M, groups, y);
    return hipGetLastError();
}

// Rows per workgroup and blocks in flight.  More rows read the tokens less
// often, fewer rows make more workgroups; us with 16 and with 32 rows, W from
// HBM, 4096 columns (1, 16 and 32 tokens):
//    1000 rows    5.8  7.5     7.0  8.9     8.9 11.1
//    4096         6.9  8.3     7.3  9.1     9.2 11.3
//    5003         8.7  9.0    11.5 10.2    15.5 12.6
//    8192         9.3  9.7    12.9 10.6    15.6 11.8
//   11008        13.1 15.1    16.1 16.8    21.7 21.3
//   14336        15.3 16.3    20.3 18.2    27.5 21.9
//   22016        22.2 23.7    28.5 26.3    39.4 31.9
// (4096 rows of 11008 and 14336 columns: 16 rows by 15 to 32 %.)  From 12288 rows
// on 32 are the better choice for all but one token; between 5000 and 8192, where
// they make one round of 16 rows' two, they would be from a few tokens on too, by
// 10 to 25 %.  Two blocks in flight and 8 waves: 3 or 4 blocks take 3 to 30 %
// longer, 16 waves between 3 % less and 16 % more.  More than F8_FEW tokens come
// here only where the tiled kernels' offsets do not reach.
template <typename Y>
hipError_t launch_few_tokens(const uint8_t *W, const float *ws, int out, int in, const uint8_t *X, const float *xs,
                             int M, Y *y, hipStream_t st) {
    if (M <= 16)
        return out >= 12288 ? launch_few<2, 1, 8, 2>(W, ws, out, in, X, xs, M, y, st)
                            : launch_few<1, 1, 8, 2>(W, ws, out, in, X, xs, M, y, st);
    return out >= 12288 ? launch_few<2, 2, 8, 2>(W, ws, out, in, X, xs, M, y, st)
                        : launch_few<1, 2, 8, 2>(W, ws, out, in, X, xs, M, y, st);
}

}  // namespace

hipError_t launch_quantize_f8(const uint16_t *X, int M, int in, uint8_t *codes, float *scales, hipStream_t st) {
    // 4 x 4096: 2.0 us with one block a lane, 2.6 with four; 2048 x 4096: 6.1 and
    // 6.5; 4096 x 4096: 10.5 and 9.9
    const int T = f8_blocks(in);
    if (f8_spread(M, T, 65536))
        hipLaunchKernelGGL(quantize_f8_kernel<1>, f8_token_grid(M, T, 1), dim3(FQ_THREADS), 0, st, X, M, in, T, codes,
                           scales);
    else
        hipLaunchKernelGGL(quantize_f8_kernel<4>, f8_token_grid(M, T, 4), dim3(FQ_THREADS), 0, st, X, M, in, T, codes,
                           scales);
    return hipGetLastError();
}

hipError_t launch_encode_f8(const float *W, int out, int in, uint8_t *codes, float *scales, int32_t *status,
                            hipStream_t st) {
    const int T = f8_blocks(in);
    const int64_t groups = (int64_t)T * f8_blocks(out);
    if (groups > 0x7FFFFFFF / FQ_THREADS)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(encode_f8_kernel, dim3((unsigned)groups), dim3(FQ_THREADS), 0, st, W,
                       out, in, T, codes, scales, status);
    return hipGetLastError();
}

hipError_t launch_gemm_f8(const uint8_t *W, const float *ws, int out, int in, const uint8_t *X, const float *xs,
                          int M, void *y, int y_f32, int exact, void *workspace, size_t ws_bytes, hipStream_t st) {
    if (M > F8_FEW && gemm_f8_tile_supports(out, in, M))
        return launch_gemm_f8_tile(W, ws, out, in, X, xs, M, y, y_f32, y_f32 || exact, workspace, ws_bytes, st);
    return y_f32 ? launch_few_tokens(W, ws, out, in, X, xs, M, static_cast<float *>(y), st)
                 : launch_few_tokens(W, ws, out, in, X, xs, M, static_cast<uint16_t *>(y), st);
}

hipError_t launch_gemv_f8(const uint8_t *W, const float *ws, int out, int in, const uint16_t *x, uint16_t *y,
                          hipStream_t st) {
    // blocks in flight per wave: no more than a wave has (512 rows, 512 columns:
    // 2.3 us with 1, 3.5 us with 4)
    constexpr int WAVES = 8;
    const int T = f8_blocks(in);
    const dim3 grid((unsigned)(((int64_t)out + 15) / 16)), block(WAVES * RBQ_WAVE);
    if (T <= WAVES)
        hipLaunchKernelGGL((gemv_f8_kernel<WAVES, 1>), grid, block, 0, st, W, ws, out, in, T, x, y);
    else if (T <= 2 * WAVES)
        hipLaunchKernelGGL((gemv_f8_kernel<WAVES, 2>), grid, block, 0, st, W, ws, out, in, T, x, y);
    else
        hipLaunchKernelGGL((gemv_f8_kernel<WAVES, 4>), grid, block, 0, st, W, ws, out, in, T, x, y);
    return hipGetLastError();
}

}  // namespace rbq
