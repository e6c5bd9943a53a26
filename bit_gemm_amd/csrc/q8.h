// Rows in 8 bits: e4m3 codes with a power-of-two scale (e8m0) for each block
// of 128. Shared by the norm that makes such rows and by the head's kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace mq {

constexpr int kQ8Block = 128;

// Bits of |v|. As whole numbers they order as magnitudes do, with Inf above
// every finite value and NaN above Inf, so a maximum of them loses neither.
__device__ __forceinline__ uint32_t q8_magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

// The scale byte e + 127 of a block whose largest magnitude has these bits: the
// smallest e >= -127 with top <= 448 2^e. 448 = 1.75 2^8, so e is top's
// exponent less 8, one more where its fraction passes 1.75.
__device__ __forceinline__ uint32_t q8_scale(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  if (top == 0u) return 127u;
  const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 0);
}

// Eight values of a block as codes. x 2^-e is exact (or, where it is too small
// for a code, rounds to the same code), so each value is rounded once, to e4m3.
__device__ __forceinline__ uint2 q8_codes(const float* v, uint32_t scale) {
  if (scale == 255u) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float m = __builtin_bit_cast(float, (254u - scale) << 23);
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * m, v[1] * m, 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * m, v[3] * m, a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * m, v[5] * m, 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * m, v[7] * m, b, true);
  return make_uint2((uint32_t)a, (uint32_t)b);
}

// The largest of 16 lanes that share a block (lanes 16 i .. 16 i + 15 of a wave).
__device__ __forceinline__ uint32_t q8_top16(uint32_t top) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  return top;
}

}  // namespace mq
