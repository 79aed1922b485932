// fourbit.cuh -- the 4-bit cached row: layout, quantization and the way back.
//
// A cached key or value row of one KV head (H elements) is cut into groups of
// 32 consecutive elements.  Each group has a scale s and 4-bit codes c:
//     a = max|x|,  s = ue5m3(a / 7),  c = clamp(rn(x / s), -7, 7),  value = c * s
// (symmetric absolute-maximum quantization, "جعل inference رخيصًا: KV cache
// وbatching والتكميم"; a scale per group because four bits leave a whole row of
// H elements too few steps).  ue5m3 keeps four significant bits of a / 7 in one
// byte: the f16 number with bits (byte << 7), no sign.  Four bits suffice: the
// nearest such s is at most 1/16 off, so the group's largest element has
// |x / s| <= 7 * 16 / 15 < 7.5 and its code's error stays below the half step
// that rounding costs anyway.  And they make the way back exact: c (3 bits) times s (4 bits)
// has at most 7 significant bits, so every value is exactly an f16 (and a bf16)
// number and the attention kernel adds no rounding of its own to K or V.
// s is at most 9216 (7 * 9216 = 64512, the largest multiple of 7 below f16's
// range whose scale has four bits); larger elements saturate.  Groups with
// a / 7 below 2^-18 get s = 0 and read as zeros.
//
// Layout: codes [num_blocks][K][16][H/2] bytes -- the tile of a block and KV
// head is contiguous, H/2 bytes a row, element 2i in the low half of byte i,
// stored as c + 8 -- and scales [num_blocks][K][16][H/32] bytes.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace gqa {

constexpr int kQ4Group = 32;            // elements per scale
constexpr uint32_t kQ4MaxScale = 225u;  // ue5m3 code of 9216

// a / 7 rounded to ue5m3, nearest even, saturating.  a is max|x|, not NaN.
__device__ __forceinline__ uint32_t q4_scale_code(float a) {
    const float y = __fdiv_rn(a, 7.f);
    if (y >= 9216.f) return kQ4MaxScale;
    if (y < 6.103515625e-05f) return (uint32_t)__float2int_rn(y * 131072.f);  // steps of 2^-17
    const uint32_t u = __float_as_uint(y);
    // keep three mantissa bits of 23, then rebias the exponent from 127 to 15
    return ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
}
__device__ __forceinline__ float q4_scale_value(uint32_t code) {
    return __half2float(__ushort_as_half((unsigned short)(code << 7)));
}
// The 4-bit code of x under scale value s, as stored (c + 8).  NaN: zero.
__device__ __forceinline__ uint32_t q4_code(float x, float s) {
    if (s == 0.f) return 8u;
    const float y = __fdiv_rn(x, s);
    const int r = (y != y) ? 0 : __float2int_rn(fminf(fmaxf(y, -7.f), 7.f));
    return (uint32_t)(r + 8);
}

}  // namespace gqa
