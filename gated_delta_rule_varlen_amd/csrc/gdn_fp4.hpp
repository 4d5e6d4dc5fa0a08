// gdn_fp4.hpp -- the 4-bit cache's codes and scales on the device.
//
// A block of 32 elements shares 2^e, held as the byte e + 127: shifted by 23 it is that number in fp32, which is what the
// chip's conversions between 4-bit codes and floats take as their scale.  They round to the nearest code, a tie to the
// even one, and widen exactly.
#pragma once

#include "gdn_device.hpp"

namespace gdn {
namespace fp4 {

constexpr uint32_t kNotANumber = 255;  // the scale byte of a block with an infinity or NaN

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight elements' values, from their 32 bits of codes.
__device__ __forceinline__ void values(uint32_t codes, uint32_t scale_byte, float* y) {
    const float s = scale_of(scale_byte);
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 1);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 3);
    y[0] = a[0], y[1] = a[1], y[2] = b[0], y[3] = b[1], y[4] = c[0], y[5] = c[1], y[6] = d[0], y[7] = d[1];
}

}  // namespace fp4
}  // namespace gdn
