// gemm_q4.hip -- the many-token product of a layer in 4 bits with group scales:
//   Y[m][r] = sum_t s[r][t] sum_{j in group t} (c[r][j] - z[r][t]) X[m][j]
#include <hip/hip_runtime.h>

#include "rbq.h"
#include "rbq_kernels.h"
#include "f8_device.h"
#include "q4_device.h"
#include "q4_plan.h"

namespace rbq {

namespace {

__device__ __forceinline__ auto q4_buffer(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x00027000);
}

// Where the 16-byte piece q of token m lies among its 16 in LDS.
__device__ __forceinline__ int q4_place(int q, int m) {
    return ((q & 3) * 4 + (q >> 2)) ^ m ^ (m & 1) << 1;
}

template <typename Y>
__device__ __forceinline__ Y q4_to(float v) {
    if constexpr (sizeof(Y) == 2)
        return (Y)f2h(v);
    else
        return (Y)v;
}

// Tiles of 256 rows by 64 tokens, a wave 64 rows of them; a group of 128 columns a
// stage.  The tokens of a stage go through registers, where they are put into the
// operands' order, to one of two buffers in LDS (256 bytes a token, placed so that 16
// tokens' reads of one piece and 16 pieces' writes of one token hit every bank once).
// The codes of a wave's rows go straight to its registers, 16 bytes a lane and row
// tile, and are unpacked there for 64 tokens each.  Both are requested a stage ahead.
// The scales and zero points of Q4_AHEAD groups at a time go through LDS, a row a
// thread: loaded where they are used, 2 bytes from each of 16 rows, they took 39 of
// 277 us (2048 tokens, 14336 x 4096).
//
// 2048 tokens of 14336 x 4096: 240 to 250 us by the card, 0.96 to 1.0 PFLOP/s (a library's
// fp16 product of that size: 211 us, 1.14).  8192 of 11008 x 4096: 717 to 740 us, 1.0 to
// 1.03.  Two workgroups a CU, at 41 cycles a product and SIMD where the instruction takes
// 16: bound by issue, 3.7 vector instructions beside a product (1 to scale its group's
// sum, 2.3 to unpack), of which four alone bring 16 to 26 or 28.  Tried, beside 254 then:
// 128 tokens a tile (unpacks half as often, but one wave a SIMD and 141 moves between
// register files: 290 us), 512 rows (292 us), two or four products before the other work
// (256, 278), no order given (255 to 262).
constexpr int Q4_AHEAD = 8;

typedef uint32_t q4_u32x4 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t q4_u32x2 __attribute__((ext_vector_type(2), aligned(1)));

template <bool ZEROS, typename Y>
__global__ __launch_bounds__(256, 2) void gemm_q4_tile_kernel(
    const uint8_t *__restrict__ codes, const uint16_t *__restrict__ scales, const uint8_t *__restrict__ zeros, int out,
    int in, int T, const uint16_t *__restrict__ X, int M, Y *__restrict__ y, float *__restrict__ parts, int tiles_m,
    int tiles_r, int slices) {
    constexpr int TM = 4, TN = 4, THREADS = 256, RT = Q4_ROWS, CT = Q4_TOKENS;
    static_assert(RT == THREADS && RT == TM * 64 && CT == TN * 16 && THREADS / 16 == 16);
    constexpr int PIECES = CT * 16 / THREADS;       // 16-byte pieces of X a thread stages
    __shared__ __align__(16) uint8_t lds[2][CT * 256];
    __shared__ __align__(16) uint16_t lscales[2][RT][Q4_AHEAD];
    __shared__ __align__(8) uint8_t lzeros[ZEROS ? 2 : 1][RT][Q4_AHEAD];
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g = lane >> 4;
    const int wr = __builtin_amdgcn_readfirstlane(tid >> 6);

    // tiles in bands of 8 token tiles, tokens fastest: the workgroups of an XCD
    // share tokens and rows
    int id = xcd_run(blockIdx.x, tiles_m * tiles_r * slices);
    const int slice = __builtin_amdgcn_readfirstlane(id % slices);
    id /= slices;
    const int band = id / (8 * tiles_r), bw = min(8, tiles_m - 8 * band);
    id -= band * 8 * tiles_r;
    const int64_t r0 = (int64_t)__builtin_amdgcn_readfirstlane(id / bw) * RT;
    const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane(8 * band + id % bw) * CT;
    const int t0 = __builtin_amdgcn_readfirstlane(T / slices * slice + min(slice, T % slices));
    const int t1 = t0 + __builtin_amdgcn_readfirstlane(T / slices + (slice < T % slices));

    // Loads through buffer descriptors of the tile's rows and tokens, so that the parts
    // of an address that all lanes share are scalar.  Every load is inside the tile
    // (q4_plan.h), with no help of the descriptors' ranges, which need not count the
    // scalar part; only the 0 of tokens that do not count is a range's, of an offset that
    // passes it by itself.
    const int rows = (int)min((int64_t)RT, (int64_t)out - r0), toks = (int)min((int64_t)CT, (int64_t)M - m0);
    const auto wbuf = q4_buffer(codes + r0 * (in / 2), (uint32_t)rows * (uint32_t)(in / 2));
    // (Sixteen tokens that are none of the tile's are not read again: an empty range, and
    // no scalar part that could be taken off it.  32 tokens, 28672 x 8192: 51.8 us so, 53.7
    // where they are.)
    const auto xbuf = q4_buffer(X + m0 * in, (uint32_t)toks * (uint32_t)in * 2u);
    const auto none = q4_buffer(X + m0 * in, 0);
    const decltype(q4_buffer(X, 0)) xbufs[PIECES] = {xbuf, toks > 16 ? xbuf : none, toks > 32 ? xbuf : none, toks > 48 ? xbuf : none};
    const uint32_t xkeep[PIECES] = {~0u, toks > 16 ? ~0u : 0u, toks > 32 ? ~0u : 0u, toks > 48 ? ~0u : 0u};
    static_assert(PIECES == 4);
    int rfirst[TM], mfirst[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
        rfirst[i] = q4_first(wr * 64 + i * 16, rows);
#pragma unroll
    for (int n = 0; n < TN; ++n)
        mfirst[n] = q4_first(n * 16, toks);
    const uint32_t woff = q4_lane_codes(rows, in, li, g), xoff = q4_lane_tokens(toks, in, tid >> 4, tid & 15);
    // (a thread's tokens are THREADS / 16 apart, a multiple of 16)
    const uint32_t xat = (uint32_t)((tid >> 4) * 256 + (q4_place(tid & 15, tid >> 4 & 15) * 16));

    // A group goes through the row tiles one by one: beside the 16 products of row
    // tile i stand the scaling of the sums of tile i - 1 and the unpacking of tile
    // i + 1, whose raw codes make room for the next group's.  The tokens' operands
    // of a group stay in registers and are replaced by the next group's as the last
    // row tile uses them.
    const q4_bits bits;
    uint4 wraw[TM], xraw[PIECES];
    uint32_t sraw, zraw;
    float s[2];
    q4_f16x8 a[TN][4], b[2][4];
    q4_f32x4 acc[TM][TN] = {}, p[2][TN] = {};
    auto request_w = [&](int t, int i) __attribute__((always_inline)) {
        const uint32_t at = (uint32_t)rfirst[i] * (uint32_t)(in / 2) + (uint32_t)q4_column(in, t) / 2;
        wraw[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(wbuf, woff, at, 0));
    };
    // Q4_AHEAD groups of the thread's row (past the row's end: anything, not used;
    // past the array's end none)
    const uint16_t *const sfirst = scales + r0 * T;
    const uint8_t *const zfirst = ZEROS ? zeros + r0 * T : nullptr;
    const uint32_t srow = (uint32_t)(q4_first(tid & ~15, rows) + min(tid & 15, rows - 1)) * (uint32_t)T;
    const uint32_t send = (uint32_t)min((int64_t)1 << 30, (out - r0) * T);
    auto stage_s = [&](int t, int buffer) __attribute__((always_inline)) {
        const uint32_t at = srow + (uint32_t)t;
        if (at + Q4_AHEAD <= send) {
            *(uint4 *)lscales[buffer][tid] = __builtin_bit_cast(uint4, *(const q4_u32x4 *)(sfirst + at));
            if (ZEROS)
                *(uint2 *)lzeros[buffer][tid] = __builtin_bit_cast(uint2, *(const q4_u32x2 *)(zfirst + at));
        } else {
            for (int e = 0; e < Q4_AHEAD; ++e)
                if (at + e < send) {
                    lscales[buffer][tid][e] = sfirst[at + e];
                    if (ZEROS)
                        lzeros[buffer][tid][e] = zfirst[at + e];
                }
        }
    };
    auto read_s = [&](int t, int i) __attribute__((always_inline)) {
        const int row = wr * 64 + i * 16 + li, at = (t - t0) % Q4_AHEAD, buffer = (t - t0) / Q4_AHEAD & 1;
        sraw = lscales[buffer][row][at];
        if (ZEROS)
            zraw = lzeros[buffer][row][at];
    };
    auto request_x = [&](int t) __attribute__((always_inline)) {
        const int column = q4_column(in, t);
        const uint32_t at = column + (tid & 15) * 8 >= t * 128 ? xoff : Q4_BEYOND;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            xraw[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(xbufs[i], at, ((uint32_t)mfirst[i] * (uint32_t)in * 2u + (uint32_t)column * 2u) & xkeep[i], 0));
    };
    auto stage_x = [&](int buffer) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            *(q4_f16x8 *)(lds[buffer] + xat + i * (THREADS / 16) * 256) = q4_order(xraw[i]);
    };
    auto read = [&](int buffer, int n, int j) __attribute__((always_inline)) {
        a[n][j] = *(const q4_f16x8 *)(lds[buffer] + li * 256 + n * 16 * 256 + q4_place(4 * g + j, li) * 16);
    };
    auto unpack = [&](int i) __attribute__((always_inline)) {
        s[i & 1] = h2f((uint16_t)sraw);
        asm("" : "+v"(s[i & 1]));       // (converted once, not in each fma)
        q4_unpack(bits, wraw[i], ZEROS ? zraw : 8, b[i & 1]);
    };
    auto scale = [&](int i, float by) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                acc[i][n][k] = __builtin_fmaf(p[i & 1][n][k], by, acc[i][n][k]);
    };

    const int last = t1 - 1;
    if (t0 < t1) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            request_w(t0, i);
        request_x(t0);
        stage_s(t0, 0);
        stage_x(0);
        request_x(min(t0 + 1, last));
        __syncthreads();
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                read(0, n, j);
        read_s(t0, 0);
        unpack(0);
        request_w(min(t0 + 1, last), 0);
        read_s(t0, 1);
    }
    float before = 0.0f;        // the scale of the last row tile of the group before
    for (int t = t0; t < t1; ++t) {
        const int next = min(t + 1, last), buffer = (t + 1 - t0) & 1;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            if (i == TM - 1)
                __syncthreads();
            const float by = i == 0 ? before : s[(i - 1) & 1];
            // (a group's tile 1 on; its tile 0 and the next tile's scale are of the next)
            unpack((i + 1) % TM);
            read_s(i + 2 < TM ? t : next, (i + 2) % TM);
            if (i == 0 && (t - t0) % Q4_AHEAD == 0)
                stage_s(t + Q4_AHEAD, ((t - t0) / Q4_AHEAD + 1) & 1);
            request_w(i + 1 < TM ? next : min(t + 2, last), (i + 1) % TM);
            if (i == TM - 2) {
                stage_x(buffer);
                request_x(min(t + 2, last));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    const q4_f32x4 none = {};
                    p[i & 1][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[n][j], b[i & 1][j], j == 0 ? none : p[i & 1][n], 0, 0, 0);
                    if (i == TM - 1)
                        read(buffer, n, j);
                }
            scale((i + TM - 1) % TM, by);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);        // a product,
                __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);        // other work
                if (i == TM - 1)
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // and a read
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        before = s[(TM - 1) & 1];
    }
    scale(TM - 1, before);
    const bool whole = slices == 1;
    float *part = parts + (int64_t)slice * M * out;
    // (rows and tokens that stand twice are written by their own sixteen)
    auto write = [&](auto full) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)::value;
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int m = (FULL ? n * 16 : mfirst[n]) + 4 * g + k;
                if (!FULL && (m >= toks || m < n * 16))
                    continue;
                const int64_t at = (m0 + m) * out + r0;
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int r = (FULL ? wr * 64 + i * 16 : rfirst[i]) + li;
                    if (FULL || (r < rows && r >= wr * 64 + i * 16)) {
                        if (whole)
                            y[at + r] = q4_to<Y>(acc[i][n][k]);
                        else
                            part[at + r] = acc[i][n][k];
                    }
                }
            }
    };
    if (rows == RT && toks == CT)
        write(std::true_type{});
    else
        write(std::false_type{});
}

// Y = the slices' sums, in their order, eight loads on their way at a time.
template <typename Y>
__global__ __launch_bounds__(256) void gemm_q4_sum_kernel(const float *__restrict__ parts, int64_t n, int slices,
                                                          Y *__restrict__ y) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float v = 0.0f;
        for (int s = 0; s < slices; s += 8) {
            float a[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                a[k] = s + k < slices ? parts[(s + k) * n + i] : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v += a[k];
        }
        y[i] = q4_to<Y>(v);
    }
}

template <bool ZEROS, typename Y>
hipError_t launch_tile(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int out, int in,
                       const uint16_t *X, int M, Y *y, float *parts, int slices, hipStream_t st) {
    const int tiles_m = (M + Q4_TOKENS - 1) / Q4_TOKENS, tiles_r = (out + Q4_ROWS - 1) / Q4_ROWS;
    gemm_q4_tile_kernel<ZEROS, Y><<<(unsigned)(tiles_m * tiles_r * slices), 256, 0, st>>>(
        codes, scales, zeros, out, in, (in + 127) / 128, X, M, y, parts, tiles_m, tiles_r, slices);
    if (slices > 1) {
        const int64_t n = (int64_t)M * out;
        gemm_q4_sum_kernel<Y><<<(unsigned)std::min<int64_t>((n + 255) / 256, 1 << 16), 256, 0, st>>>(parts, n, slices, y);
    }
    return hipGetLastError();
}

template <typename Y>
hipError_t launch_typed(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int out, int in,
                        const uint16_t *X, int M, Y *y, float *parts, int slices, hipStream_t st) {
    return zeros != nullptr ? launch_tile<true>(codes, scales, zeros, out, in, X, M, y, parts, slices, st)
                            : launch_tile<false>(codes, scales, zeros, out, in, X, M, y, parts, slices, st);
}

}  // namespace

size_t gemm_q4_workspace_bytes(int out, int in, int M) {
    if (!q4_tiled(out, in, M))
        return 0;
    const int slices = q4_slices(out, in, M);
    return slices > 1 ? (size_t)slices * (size_t)M * (size_t)out * sizeof(float) : 0;
}

hipError_t launch_gemm_q4_tile(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int out, int in,
                               const uint16_t *X, int M, void *y, int y_f32, void *workspace, size_t ws_bytes,
                               hipStream_t st) {
    const int slices = ws_bytes < gemm_q4_workspace_bytes(out, in, M) ? 1 : q4_slices(out, in, M);
    float *parts = static_cast<float *>(workspace);
    return y_f32 ? launch_typed(codes, scales, zeros, out, in, X, M, static_cast<float *>(y), parts, slices, st)
                 : launch_typed(codes, scales, zeros, out, in, X, M, static_cast<uint16_t *>(y), parts, slices, st);
}

}  // namespace rbq
