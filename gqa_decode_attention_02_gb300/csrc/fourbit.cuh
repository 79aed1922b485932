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
// a / 7 of 2^-18 or less get s = 0 and read as zeros.
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

// a / 7 rounded to ue5m3, nearest even, saturating.  a is the magnitude of an f16
// or bf16 element (at most 11 significant bits), so a / 7 either is a midpoint of
// the grid exactly or is at least 2^-12 of itself away from one: the product with
// 1 / 7 (2^-23 off), rounded to 17 bits first, decides as the quotient does.
__device__ __forceinline__ uint32_t q4_scale_code(float a) {
    const uint32_t u = (__float_as_uint(a * 0.14285714924335480f) + 0x40u) & 0xffffff80u;
    const float y = __uint_as_float(u);
    if (y >= 9216.f) return kQ4MaxScale;
    if (y < 6.103515625e-05f) return (uint32_t)__float2int_rn(y * 131072.f);  // steps of 2^-17
    // keep three mantissa bits of 23, then rebias the exponent from 127 to 15
    return ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
}
// Scale codes whose elements may lie beyond 7.5 scales: the last one (saturation)
// and those below 2^-14 (a coarser grid).
__device__ __forceinline__ bool q4_scale_clips(uint32_t code) {
    return code - 8u >= kQ4MaxScale - 8u;
}
__device__ __forceinline__ float q4_scale_value(uint32_t code) {
    return __half2float(__ushort_as_half((unsigned short)(code << 7)));
}
// Reciprocal of a scale value for q4_word, at most 2^-23 of itself off; 0 for 0.
__device__ __forceinline__ float q4_scale_inverse(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return s == 0.f ? 0.f : r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t q4_pair(float lo, float hi) {
    return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t q4_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t q4_add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float q4_lo(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float q4_hi(uint64_t a) {
    return __uint_as_float((uint32_t)(a >> 32));
}
// The 4-bit codes of eight elements under a scale of inverse r, as stored (c + 8,
// element e in bits 4e..).  x / s is a midpoint between codes exactly or at least
// 2^-14 away from one (x has 11 significant bits, s four).  x * r + 384, rounded to
// the 2^-15 that numbers near 384 have, is at most 2^-16 + 2^-20 off and meets the
// midpoints exactly, so it falls as x / s does; adding 1.5 * 2^23 then rounds to the
// integer, nearest even.  That leaves 0x4b400000 + c + 8 as the number's bits: the
// words add up as they are, and what their upper parts sum to comes off once.
// CLIP: keep within [-7, 7].
template <bool CLIP>
__device__ __forceinline__ uint32_t q4_word(const float (&x)[8], float r) {
    uint32_t word = 0;
    const uint64_t rr = q4_pair(r, r);
#pragma unroll
    for (int e = 6; e >= 0; e -= 2) {
        uint64_t z = q4_fma2(q4_pair(x[e], x[e + 1]), rr, q4_pair(384.f, 384.f));
        if (CLIP)
            z = q4_pair(fminf(fmaxf(q4_lo(z), 377.f), 391.f),
                        fminf(fmaxf(q4_hi(z), 377.f), 391.f));
        // 1.5 * 2^23 - 384 + 8
        z = q4_add2(z, q4_pair(12582536.f, 12582536.f));
        word = word * 256u + (uint32_t)(z >> 32) * 16u + (uint32_t)z;
    }
    return word - 0x4b400000u * 0x11111111u;
}

}  // namespace gqa
