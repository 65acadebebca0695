// The 8-bit float format on the device: e4m3 codes with a power-of-two scale for each block.
#pragma once

#include "common.h"

namespace qlora {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
constexpr uint32_t kFp8Nan = 255u;   // scale byte of a block that is not finite (its codes are 0)

template <int DT>
constexpr uint32_t kInf16 = DT == kDtF16 ? 0x7C00u : 0x7F80u;

// The larger magnitude bits of two packed pairs (as integers: NaN above infinity above finite).
__device__ __forceinline__ uint32_t max_mag2(uint32_t m, uint32_t w) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                  __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}

// The largest 16-bit pattern in m's halves over the 16 lanes of a DPP row (rotations within the
// row: a VALU instruction each, where a shuffle goes through LDS).
__device__ __forceinline__ uint32_t max_row16(uint32_t m) {
    uint32_t t = max(m & 0xFFFFu, m >> 16);
    t = max(t, (uint32_t)__builtin_amdgcn_mov_dpp((int)t, 0x128, 0xF, 0xF, true));
    t = max(t, (uint32_t)__builtin_amdgcn_mov_dpp((int)t, 0x124, 0xF, 0xF, true));
    t = max(t, (uint32_t)__builtin_amdgcn_mov_dpp((int)t, 0x122, 0xF, 0xF, true));
    return max(t, (uint32_t)__builtin_amdgcn_mov_dpp((int)t, 0x121, 0xF, 0xF, true));
}

// Scale byte of a block whose largest magnitude has the 16-bit pattern a: the least e >= 0 with
// value <= 448 2^(e - 127).  448 = 1.75 * 2^8, so e is the exponent field less 8, one more where
// the fraction is above 0.75; what is subnormal in fp32 is far below 448 * 2^-127.
template <int DT>
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t a) {
    const uint32_t f = __float_as_uint(h16_to_f32<DT>(a));
    const int e = (int)(f >> 23) - 8 + ((f & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return a >= kInf16<DT> ? kFp8Nan : (uint32_t)max(e, 0);
}
// 2^(byte - 127) as fp32 (byte 0 is subnormal).
__device__ __forceinline__ float fp8_scale_value(uint32_t byte) {
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Codes of 8 values: x / scale in e4m3, ties to even (v_cvt_scalef32_pk_fp8_*, two at a time).
template <int DT>
__device__ __forceinline__ u32x2_t fp8_codes8(u32x4_t v, uint32_t byte) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float scale = fp8_scale_value(byte);
    u32x2_t o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s16x2 c = {0, 0};
        const uint32_t lo = v[2 * i], hi = v[2 * i + 1];   // (a bit cast of an element itself takes element 0)
        if (DT == kDtF16) {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c, __builtin_bit_cast(f16x2_t, lo), scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(c, __builtin_bit_cast(f16x2_t, hi), scale, true);
        } else {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2_t, lo), scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2_t, hi), scale, true);
        }
        o[i] = byte == kFp8Nan ? 0u : __builtin_bit_cast(uint32_t, c);
    }
    return o;
}

}  // namespace qlora
