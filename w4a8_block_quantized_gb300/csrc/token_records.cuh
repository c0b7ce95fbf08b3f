// token_records.cuh -- encoding of INT8 codes, shared by the kernels that produce them
// (prep.cu and row_quant.cu): the bytes of the API layout, and the nibble planes and row-sum
// entries of a token record (the layout in w4a8_internal.h).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "quant_math.cuh"
#include "w4a8_internal.h"

namespace w4a8 {

// Two e4m3 codes in one 16-bit word, v0 in the low byte: rounded to nearest even, 448 past the largest.  Of
// the planes' values (integers of at most 4 significant bits up to 128) the conversion is exact.
__device__ __forceinline__ uint32_t e4m3x2(float v0, float v1) {
    unsigned short d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(v1), "f"(v0));
    return d;
}

// Zero-point operand of one token and block: rs = 64*rh + rl as the exact fp16 pair
// {rh / 8, rl / 512} (see the rx layout in w4a8_internal.h), then 12 zero bytes.
__device__ __forceinline__ uint4 rx_entry(int rs) {
    const int rh = rs >> 6, rl = rs & 63;
    const __half2 p = __floats2half2_rn(static_cast<float>(rh) * 0.125f, static_cast<float>(rl) * (1.0f / 512.0f));
    return make_uint4(*reinterpret_cast<const uint32_t*>(&p), 0u, 0u, 0u);
}

// Token record of row m, block b, for records of 2^ts tokens (the layout in w4a8_internal.h).
__device__ __forceinline__ uint8_t* token_rec(uint8_t* trec, int64_t m, int64_t b, int64_t nb, int ts) {
    return trec + ((m >> ts) * nb + b) * (static_cast<int64_t>(144) << ts);
}

// Byte offset, inside a token record, of the 4 codes k = 4j .. 4j+3 of the block (j < 16) of
// row r in plane p (0 = high nibbles, 1 = low nibbles): 128-byte swizzle of 16-byte chunks.
__device__ __forceinline__ int plane_off(int r, int j, int p) {
    const int c = (j >> 2) + 4 * p;
    return r * 128 + ((c ^ (r & 7)) << 4) + ((j & 3) << 2);
}

// Section 3 eq. (3) planes of four float codes (exact integers in [-127, 127]): hi word holds
// e4m3(16 * floor(q / 16)) (the signed high nibble times 16), lo word e4m3(q - that) (the
// unsigned low nibble), element j in byte j.  Two elements per mul / sub .rn.f32x2; every
// product and difference here is exact (q is an integer in [-127, 127]).
__device__ __forceinline__ void planes4f(float4 q, uint32_t& hi, uint32_t& lo) {
    const uint64_t k16 = pk2(0.0625f, 0.0625f), k1 = pk2(16.0f, 16.0f);
    float a0, a1, a2, a3;
    upk2(mul2(pk2(q.x, q.y), k16), a0, a1);
    upk2(mul2(pk2(q.z, q.w), k16), a2, a3);
    const uint64_t h01 = mul2(pk2(floorf(a0), floorf(a1)), k1), h23 = mul2(pk2(floorf(a2), floorf(a3)), k1);
    float h0, h1, h2, h3, l0, l1, l2, l3;
    upk2(h01, h0, h1);
    upk2(h23, h2, h3);
    upk2(sub2(pk2(q.x, q.y), h01), l0, l1);
    upk2(sub2(pk2(q.z, q.w), h23), l2, l3);
    hi = e4m3x2(h0, h1) | (e4m3x2(h2, h3) << 16);
    lo = e4m3x2(l0, l1) | (e4m3x2(l2, l3) << 16);
}

// Four float codes as int8 bytes: adding 1.5 * 2^23 puts the integer, in two's complement,
// in the low mantissa bits, whose low byte is the code.
__device__ __forceinline__ uint32_t bytes4f(float4 q) {
    const uint32_t b0 = __float_as_uint(q.x + 12582912.0f), b1 = __float_as_uint(q.y + 12582912.0f);
    const uint32_t b2 = __float_as_uint(q.z + 12582912.0f), b3 = __float_as_uint(q.w + 12582912.0f);
    return __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
}

}  // namespace w4a8
