// f8_device.h -- device helpers of the 8-bit floating point block kernels:
// scales and e4m3 codes of a block of 128, and the matrix instructions over
// one block.
#pragma once

#include "rbq_device.h"

namespace rbq {

constexpr int F8_BLOCK = 128;
constexpr float F8_MAX = 448.0f;

inline __host__ __device__ int f8_blocks(int n) { return (n >> 7) + ((n & 127) != 0); }

// Kernels over tokens in blocks of 128: workgroups of 256 threads, 16 lanes to
// a block, take f8_rows(B) tokens x B blocks a lane; grid x the blocks, y the
// tokens (from 65535 on, in a loop).
constexpr __host__ __device__ int f8_rows(int B) { return B == 1 ? 1 : 16; }

inline dim3 f8_token_grid(int M, int T, int B) {
    const int cols = B == 1 ? 16 : B;
    const int64_t rows = ((int64_t)M + f8_rows(B) - 1) / f8_rows(B);
    return dim3((unsigned)((T + cols - 1) / cols), (unsigned)(rows < 65535 ? rows : 65535));
}

// One block a lane, for the least time from the load to the codes: up to `most`
// blocks, and with rows of fewer than 16, of which lanes are left over, few.
inline bool f8_spread(int M, int T, int64_t most) {
    return (int64_t)M * T <= (T < 16 ? 4096 : most);
}

// Tile of workgroup `id` of `total`: consecutive workgroups go to consecutive
// XCDs, so each of the 8 takes a run of consecutive tiles, which share
// operands in its L2.
__device__ __forceinline__ int xcd_run(int id, int total) {
    const int per = total >> 3;
    return id < per * 8 ? (id & 7) * per + (id >> 3) : id;
}

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));

// Largest |v| of eight fp16 values, as fp16 bits (magnitude bits order like
// unsigned integers; NaN and infinity above every finite value).
__device__ __forceinline__ uint32_t absmax8_f16(const uint4 &v) {
    const uint32_t m = 0x7FFF7FFFu;
    const v2u16 a = __builtin_elementwise_max(__builtin_bit_cast(v2u16, v.x & m), __builtin_bit_cast(v2u16, v.y & m));
    const v2u16 b = __builtin_elementwise_max(__builtin_bit_cast(v2u16, v.z & m), __builtin_bit_cast(v2u16, v.w & m));
    const v2u16 c = __builtin_elementwise_max(a, b);
    return max((uint32_t)c.x, (uint32_t)c.y);
}

// Maximum over each row of 16 lanes, in all of its lanes (DPP rotations).
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
    int x = (int)v;
    x = (int)max((uint32_t)x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x128, 0xF, 0xF, false));   // row_ror:8
    x = (int)max((uint32_t)x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x124, 0xF, 0xF, false));
    x = (int)max((uint32_t)x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x122, 0xF, 0xF, false));
    x = (int)max((uint32_t)x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x121, 0xF, 0xF, false));
    return (uint32_t)x;
}

// Scale and multiplier of a block from the fp32 bits of its largest |v|:
// two correctly rounded quotients; a non-finite maximum gives scale NaN and
// multiplier 0.
__device__ __forceinline__ void f8_scale_f32(uint32_t top, float &scale, float &inv) {
    const float A = fmaxf(__uint_as_float(top), 0x1p-100f);
    const bool bad = top >= 0x7F800000u;
    scale = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(A, F8_MAX);
    inv = bad ? 0.0f : __fdiv_rn(F8_MAX, A);
}

// ... from the fp16 bits.
__device__ __forceinline__ void f8_scale_f16(uint32_t top, float &scale, float &inv) {
    f8_scale_f32(top >= 0x7C00u ? 0x7F800000u : __float_as_uint(h2f((uint16_t)top)), scale, inv);
}

// e4m3 codes of eight fp16 values times `inv` (0: all codes 0).
__device__ __forceinline__ uint2 f8_codes8(const uint4 &v, float inv) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    int p[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        p[i] = __builtin_amdgcn_cvt_pk_fp8_f32(h2f((uint16_t)u[2 * i]) * inv, h2f((uint16_t)(u[2 * i] >> 16)) * inv,
                                               0, false);
        p[i] = __builtin_amdgcn_cvt_pk_fp8_f32(h2f((uint16_t)u[2 * i + 1]) * inv,
                                               h2f((uint16_t)(u[2 * i + 1] >> 16)) * inv, p[i], true);
    }
    return inv == 0.0f ? make_uint2(0u, 0u) : make_uint2((uint32_t)p[0], (uint32_t)p[1]);
}

// 16 x 16 sums over 128 e4m3 products: lane (i = l % 16, g = l / 16) gives 32
// bytes of row i of each side; element (4 g + v, i) comes back in register v.
//
// The fp16 form converts the codes (every e4m3 value is an fp16 number) and
// adds exact products in fp32.
__device__ __forceinline__ v4f f8_mma(const v8h (&a)[4], const v8h (&b)[4]) {
    v4f c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[q], b[q], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ v8h f8_to_f16(int lo, int hi) {
    const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return (v8h){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ void f8_to_f16(const v8i &u, v8h (&h)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        h[q] = f8_to_f16(u[2 * q], u[2 * q + 1]);
}

// acc + s * p, four fmas.
__device__ __forceinline__ v4f f8_fma(const v4f &p, float s, const v4f &acc) {
    v4f r;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        r[v] = __builtin_fmaf(p[v], s, acc[v]);
    return r;
}

// An output rounded once from its fp32 sum.
template <typename Y>
__device__ __forceinline__ Y to_y(float v);
template <>
__device__ __forceinline__ float to_y<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t to_y<uint16_t>(float v) { return f2h(v); }

}  // namespace rbq
