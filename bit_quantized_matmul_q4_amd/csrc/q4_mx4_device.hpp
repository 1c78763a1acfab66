// q4_mx4_device.hpp -- the microscaled 4-bit form on the device: element
// types, and a block's scale and codes.  Shared by q4_mx4.hip and q4_norm.hip.
//
// A block of 32 consecutive values has one power of two 2^E (a byte E + 127;
// 255: not a number) and codes of 4 bits: sign, 2 exponent bits, 1 mantissa
// bit, the values 0, 0.5, 1, 1.5, 2, 3, 4, 6.  With a the block's largest
// magnitude, E = max(floor(log2 a) - 2, -127) and a code is v / 2^E rounded to
// the nearest (ties to an even code), what is over 6 to 6: exact in every
// case, since the division is by a power of two and the conversion
// instruction rounds once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_mx4_plan.hpp"

namespace q4 {
namespace mx4 {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Element types: 0 binary16, 1 bfloat16, 2 binary32.  Eight values lie in
// kVecs<KIND> vectors of 16 bytes.
template <int KIND>
constexpr int kVecs = KIND == 2 ? 2 : 1;

// Binary32 bits of the magnitude of the largest of eight values; infinities
// and NaN stand above every finite value.
template <int KIND>
__device__ __forceinline__ uint32_t top8(const u32x4 (&v)[kVecs<KIND>])
{
    uint32_t top = 0;
    if constexpr (KIND == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = max(top, v[i][j] & 0x7FFFFFFFu);
        return top;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            top = max(top, max(v[0][j] & 0x7FFFu, (v[0][j] >> 16) & 0x7FFFu));
        if constexpr (KIND == 1)
            return top << 16;
        else
            return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)top));
    }
}

// The largest over the four lanes of a quad, which hold a block of 32 values.
__device__ __forceinline__ uint32_t top_of_quad(uint32_t top)
{
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
    return max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top)
{
    const uint32_t e = top >> 23;
    return e == 255 ? 255 : e > 2 ? e - 2 : 0;
}

// 2^(byte - 127); for byte 0 the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

// The codes of eight values, the first in the lowest bits; 0 for a block that
// holds an infinity or NaN.
template <int KIND>
__device__ __forceinline__ uint32_t codes8(const u32x4 (&v)[kVecs<KIND>], uint32_t byte)
{
    const float s = scale_value(byte);
    uint32_t w = 0;
    if constexpr (KIND == 2) {
        const auto f = [&](int i) { return __builtin_bit_cast(float, (uint32_t)v[i / 4][i % 4]); };
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(0), f(1), s, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(2), f(3), s, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(4), f(5), s, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(6), f(7), s, 3);
    } else if constexpr (KIND == 1) {
        const auto p = [&](int i) { return __builtin_bit_cast(bf16x2, (uint32_t)v[0][i]); };
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p(0), s, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p(1), s, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p(2), s, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p(3), s, 3);
    } else {
        const auto p = [&](int i) { return __builtin_bit_cast(f16x2, (uint32_t)v[0][i]); };
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, p(0), s, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, p(1), s, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, p(2), s, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, p(3), s, 3);
    }
    return byte == 255 ? 0 : w;
}

}  // namespace mx4
}  // namespace q4
