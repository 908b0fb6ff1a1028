// MXFP4 arithmetic shared by the quantisers and the grouped GEMMs' epilogues:
// E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; no infinity,
// no NaN) with one E8M0 scale 2^e per 32 elements.  Element 2i of a row is the
// low nibble of its byte i, element 2i + 1 the high one.
#pragma once

#include "moe_internal.h"

namespace moe {
namespace mx4 {

typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

// largest magnitude of 8 bf16, as its 15 bits.  Magnitudes order as integers,
// an infinity (0x7f80) above every number and a NaN above that.
__device__ __forceinline__ uint32_t amax8(uint4 v)
{
    auto mx = [](uint32_t a, uint32_t b) __attribute__((always_inline)) {
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                      __builtin_bit_cast(u16x2, b)));
    };
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t m = mx(mx(v.x & kAbs, v.y & kAbs), mx(v.z & kAbs, v.w & kAbs));
    return max(m & 0xffffu, m >> 16);
}

// Scale byte (e + 127) of a block whose largest magnitude is amax: e is the
// smallest integer in [-127, 127] with amax <= 6 * 2^e = 1.5 * 2^(e+2).  With
// amax = m * 2^E, m in [1, 2), that is E - 2, or E - 1 when m > 1.5; a
// subnormal or zero amax is below 6 * 2^-127.  (The OCP conversion takes E - 2
// and saturates; where m > 1.5 this one keeps the maximum instead.)  The elements have neither
// infinity nor NaN, so either takes the scale's NaN (255).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    if (amax >= 0x7f80u) return 255u;
    const int s = (int)(amax >> 7) - 2 + ((amax & 0x7fu) > 0x40u ? 1 : 0);
    return (uint32_t)max(s, 0);
}

// 2^(s - 127) for the packed conversions, which take the scale's exponent
__device__ __forceinline__ float scale_f32(uint32_t s) { return __uint_as_float(s == 0 ? 0x00400000u : s << 23); }

// The codes of 8 bf16 under scale byte s, element i in bits 4i .. 4i+3: the
// hardware conversion divides by the scale and rounds to nearest even (it
// agrees with that definition for every bf16 value and every scale under
// which the value lies within 6: 8.45 million pairs).  Zero codes under the
// NaN scale.
__device__ __forceinline__ uint32_t encode8(uint4 v, uint32_t s)
{
    const float sc = scale_f32(s);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w[0]), sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w[1]), sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w[2]), sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w[3]), sc, 3);
    return s == 255u ? 0u : c;
}

// One block of 32 bf16 held as 8 by each of four consecutive lanes (4j ..
// 4j+3, in element order; all four must execute it): the block's maximum
// goes round the quad by two lane permutations.  Returns the scale byte.
__device__ __forceinline__ uint32_t quant8_quad(uint4 v, uint32_t& codes)
{
    uint32_t a = amax8(v);
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xF, 0xF, false));
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xF, 0xF, false));
    const uint32_t s = scale_byte(a);
    codes = encode8(v, s);
    return s;
}

// the 8 values of a word of codes as bf16, which holds them all (2^-128, the
// smallest, is a subnormal bf16); what passes its range is infinite and the
// NaN scale gives NaN (checked for all 256 x 256 scale and code bytes)
__device__ __forceinline__ uint4 decode8(uint32_t c, uint32_t s)
{
    const float sc = scale_f32(s);
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 3)));
}

}  // namespace mx4
}  // namespace moe
