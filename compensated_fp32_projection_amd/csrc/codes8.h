// 8-bit codes: quantising, rescaling and reading (device code; the formulas are
// in include/cfp32.h).
#pragma once

#include "device_common.h"

namespace cfp32 {

constexpr float kLeastScale = 0x1p-126f;

// The value of byte SEL of `codes`.  Floats: the byte's exponent and mantissa,
// put where FP16's are, are the value times 2^-8 (also below the normal ones),
// with no code that is not finite.
template <bool E4M3, int SEL>
__device__ __forceinline__ float code_value(uint32_t codes)
{
    if constexpr (E4M3) {
        const uint32_t x = codes >> (8 * SEL);
        const uint16_t h = (uint16_t)((x & 0x80) << 8 | (x & 0x7F) << 7);
        return (float)__builtin_bit_cast(_Float16, h) * 256.0f;
    } else {
        return (float)(int8_t)(codes >> (8 * SEL));
    }
}

// The scale of a block whose largest magnitude is `most` (its bits).
template <bool E4M3>
__device__ __forceinline__ float fresh_scale(uint32_t most)
{
    if constexpr (E4M3) {
        // most = m 2^e: 2^(e - 8) while m is at most 1.75 = 448 / 2^8.
        const int x = (int)(most >> 23) - 8 + ((most & 0x7FFFFF) > 0x600000);
        return __builtin_bit_cast(float, (uint32_t)max(x, 1) << 23);
    } else {
        return fmaxf(__builtin_bit_cast(float, most) * (1.0f / 127.0f), kLeastScale);
    }
}

// The least k for which `s` 2^k is `least` or more (bits of both, normal).
__device__ __forceinline__ int doublings(uint32_t s, uint32_t least)
{
    return least <= s ? 0 : (int)(least >> 23) - (int)(s >> 23) + ((least & 0x7FFFFF) > (s & 0x7FFFFF));
}

// The least k >= 0 for which a block of scale s x 2^k holds `most` (its bits, finite): the largest code x the scale is
// `most` or more, or (integers, where that is rounded) the scale is one that `most` would be given itself.  With the
// first alone, every 20th `most` did not fit the scale that it had been given.
template <bool E4M3>
__device__ __forceinline__ int growth(float s, uint32_t most)
{
    const int k = doublings(__builtin_bit_cast(uint32_t, s * (E4M3 ? 448.0f : 127.0f)), most);
    if constexpr (E4M3) return k;
    else return min(k, doublings(__builtin_bit_cast(uint32_t, s), __builtin_bit_cast(uint32_t, fresh_scale<false>(most))));
}

// x / s to the nearest integer, ties to even, of the exact quotient (|x| is at
// most 127 s but for two roundings, s normal).  x * inv is off by 2^-16 at most,
// so t is the nearest integer or, next to a tie, its neighbour; what x leaves
// beside t s needs no more than FP32's bits, and decides.
__device__ __forceinline__ int quotient(float x, float s, float inv)
{
    int t = (int)rintf(x * inv);
    const float r = 2.0f * fmaf(-(float)t, s, x);
    const bool odd = t & 1;
    t += r > s || (r == s && odd);
    t -= r < -s || (r == -s && odd);
    return t;
}

// Four values as codes of scale s.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode(const float (&x)[4], float s, float inv)
{
    if constexpr (E4M3) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, w, true);
    } else {
        // x inv is as good as the quotient but next to a tie, where few waves are (8190 tokens of 8 x 128 24 -> 21 us).
        float t[4], far = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float y = x[e] * inv;
            t[e] = rintf(y);
            far = fmaxf(far, fabsf(y - t[e]));
        }
        if (__any(far > 0.4999f))
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = (float)quotient(x[e], s, inv);
        uint32_t w = 0;  // bytes of t + 128, signs turned
#pragma unroll
        for (int e = 0; e < 4; ++e) w = __builtin_amdgcn_cvt_pk_u8_f32(t[e] + 128.0f, e, w);
        return w ^ 0x80808080u;
    }
}

// Four codes divided by 2^k.
template <bool E4M3>
__device__ __forceinline__ uint32_t shifted(uint32_t codes, int k)
{
    const float x[4] = {__builtin_amdgcn_ldexpf(code_value<E4M3, 0>(codes), -k), __builtin_amdgcn_ldexpf(code_value<E4M3, 1>(codes), -k),
                        __builtin_amdgcn_ldexpf(code_value<E4M3, 2>(codes), -k), __builtin_amdgcn_ldexpf(code_value<E4M3, 3>(codes), -k)};
    return encode<E4M3>(x, 1.0f, 1.0f);
}

}  // namespace cfp32
