// 8-bit floating point (OCP E4M3) with one fp32 scale per block of 128: the
// helpers that the quantising kernels and the products share.
#pragma once

#include "common.hpp"
#include "mxfp8.hpp"

namespace moe {

constexpr int kBlk = 128;  // values of a block along a row; a weight block is 128 x 128

__host__ __device__ __forceinline__ int blk_count(int n) { return (n + kBlk - 1) / kBlk; }

// Exponent of a block's scale: the smallest e with amax <= 448 * 2^e, within the
// normal fp32 powers of two; 0 for a block of zeros.  448 is 1.75 * 2^8, so e is
// amax's own exponent less 8, one more where its fraction passes 1.75.  (A power of
// two, as in the blocks of 32: x * 2^-e is exact, so a value's code does not depend
// on how a division was rounded.  With amax / 448 in its place one value in 700 of
// bf16 activations lay on a code's border and went the way of the rounding.)
// An infinity gives some e whose codes for it are NaN; a NaN is passed over by the
// maximum, its code is NaN as well.
__device__ __forceinline__ int blk_exp(float amax) {
    const uint32_t u = __builtin_bit_cast(uint32_t, amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return u == 0 ? 0 : e < -126 ? -126 : e;
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2f(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

__device__ __forceinline__ void unpack_bf16x8(intx4 raw, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = __builtin_bit_cast(float, (uint32_t)raw[q] << 16);
        v[2 * q + 1] = __builtin_bit_cast(float, (uint32_t)raw[q] & 0xffff0000u);
    }
}

// Two values rounded to nearest even by the conversion instruction, a NaN of any
// payload staying one.
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    typedef float floatx2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(floatx2{a, b}, bf16x2));
}

__device__ __forceinline__ intx4 pack_bf16x8(const float (&v)[8]) {
    intx4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = (int)pack_bf16x2(v[2 * q], v[2 * q + 1]);
    return o;
}

__device__ __forceinline__ float abs_max8(const float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) m = fmaxf(m, fabsf(v[c]));
    return m;
}

// eight values times 2^-e -> eight codes
__device__ __forceinline__ uint64_t blk_codes8(const float (&v)[8], int e) {
    const float inv = pow2f(-e);
    const uint32_t lo = fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    const uint32_t hi = fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    return (uint64_t)lo | ((uint64_t)hi << 32);
}

}  // namespace moe
