// kv_codes.cuh -- the cache's 8-bit codes as fp16 pairs, for the tensor cores.
//
// Both formats' codes are exact in fp16.
#pragma once

#include <cstdint>

#include "w4a8_internal.h"

namespace w4a8 {

// b byte permutation: result byte i is byte (sel >> 4 i) & 7 of {b, a}.
__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
    return __byte_perm(a, b, sel);
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four codes (one register) to two fp16 pairs.
//   INT8  code + 128 as an unsigned byte u under the byte 0x64 is the fp16 1024 + u; less 1152 it is the
//         code, exactly: a permute and half a packed subtraction a code, no conversion.
//   e4m3  one conversion a pair.  (By bits -- a permute, a shift and a mask a pair, all on the one pipe -- the
//         attention of 64 ragged sequences took 1.4 times as long.)  A NaN code stays NaN, so codes in places that
//         nobody sees are replaced before they meet a weight of 0.
template <int FMT>
struct Codes;

template <>
struct Codes<W4A8_KV_INT8> {
    // bytes made ready for pair(): done once per register
    static __device__ __forceinline__ uint32_t ready(uint32_t w) { return w ^ 0x80808080u; }
    // bytes I, J of a ready register, made ready for value()
    template <int I, int J>
    static __device__ __forceinline__ uint32_t raw(uint32_t w) {
        return byte_perm(w, 0x64646464u, I | (4 << 4) | (J << 8) | (4 << 12));
    }
    static __device__ __forceinline__ uint32_t value(uint32_t raw) { return hsub2(raw, 0x64806480u); }
};

template <>
struct Codes<W4A8_KV_E4M3> {
    static __device__ __forceinline__ uint32_t ready(uint32_t w) { return w; }
    template <int I, int J>
    static __device__ __forceinline__ uint32_t raw(uint32_t w) {
        uint32_t d;
        const uint32_t h = (I == 0 && J == 1) ? w : byte_perm(w, 0u, I | (J << 4));
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(h));
        return d;
    }
    static __device__ __forceinline__ uint32_t value(uint32_t raw) { return raw; }
};

}  // namespace w4a8
