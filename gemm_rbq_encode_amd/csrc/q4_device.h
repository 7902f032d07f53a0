// q4_device.h -- 4-bit codes and fp16 tokens as operands of the fp16 matrix
// instruction.
//
// A 32-bit word holds the codes of 8 consecutive columns, the lowest bits first.
// A code in the low bits of a half with the exponent of 1024 (or four bits
// higher, with that of 64) is the number 1024 + c (64 + c), so one and-or makes
// two operands and one packed subtraction of 1024 + z (64 + z) leaves the exact
// c - z.  The operands come out in the order of columns 0 4 1 5 2 6 3 7, and the
// tokens are put into the same order.
#pragma once

#include "rbq_device.h"

namespace rbq {

typedef _Float16 q4_f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 q4_f16x2 __attribute__((ext_vector_type(2)));
typedef float q4_f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ q4_f16x2 q4_pair(uint32_t v) { return __builtin_bit_cast(q4_f16x2, v); }

// The bits and exponents in registers: as literals they would make two
// instructions of every and-or.
struct q4_bits {
    uint32_t low = 0x000F000Fu, high = 0x00F000F0u, e1024 = 0x64006400u, e64 = 0x54005400u;
    __device__ __forceinline__ q4_bits() { asm("" : "+s"(low), "+s"(high), "+v"(e1024), "+v"(e64)); }
};

// Codes of 32 columns with zero point z -> four operands of 8 columns.
__device__ __forceinline__ void q4_unpack(const q4_bits &k, uint4 raw, uint32_t z, q4_f16x8 (&b)[4]) {
    // -(1024 + z) and -(64 + z): their last places are 1 and 1/16
    const q4_f16x2 f = q4_pair(0xE400E400u + (z & 15) * 0x10001u), n = q4_pair(0xD400D400u + (z & 15) * 0x100010u);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = w[i] >> 8;
        const q4_f16x2 p0 = q4_pair((w[i] & k.low) | k.e1024) + f;
        const q4_f16x2 p1 = q4_pair((w[i] & k.high) | k.e64) + n;
        const q4_f16x2 p2 = q4_pair((u & k.low) | k.e1024) + f;
        const q4_f16x2 p3 = q4_pair((u & k.high) | k.e64) + n;
        b[i] = q4_f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
}

// 8 consecutive fp16 of a token in the order of the operands.
__device__ __forceinline__ q4_f16x8 q4_order(uint4 v) {
    uint4 o;
    o.x = __builtin_amdgcn_perm(v.z, v.x, 0x05040100);
    o.y = __builtin_amdgcn_perm(v.z, v.x, 0x07060302);
    o.z = __builtin_amdgcn_perm(v.w, v.y, 0x05040100);
    o.w = __builtin_amdgcn_perm(v.w, v.y, 0x07060302);
    return __builtin_bit_cast(q4_f16x8, o);
}

}  // namespace rbq
