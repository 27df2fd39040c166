// Block-scaled 8-bit codes of kept activations: 32 consecutive columns of a row share a
// power-of-two scale 2^e (one byte, e + 127) and each holds an e4m3fn code of value / 2^e.
//
// e is the smallest with amax <= 448 2^e, so nothing saturates (the exponent of amax alone would
// clip block maxima above 1.75 of their power of two), and at least -117, so every code's value
// (the smallest 2^-9 2^e) is a normal number of bf16 and fp32: decoding is exact in both.  A
// block with a NaN or an infinity gets the scale byte 255 and reads back as NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_common.h"

namespace moe {

constexpr int kMxMinExp = -117;
constexpr uint32_t kMxNan = 255;

// the scale byte of a block whose largest |value| has these fp32 bits (NaN above infinity)
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return kMxNan;
  // amax = m 2^x (m in [1, 2)): 448 = 1.75 2^8
  int e = static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < kMxMinExp ? kMxMinExp : e;
  return static_cast<uint32_t>(e + 127);
}
// 2^-e for the codes (0 for the NaN byte: its codes are 0)
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == kMxNan ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 2^e for the values
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  const uint32_t bits = byte == kMxNan ? 0x7FC00000u : byte << 23;
  return __uint_as_float(byte == 0 ? 0x00400000u : bits);
}
// Four codes of v[i] * inv.  The product is exact above the smallest normal code, and the
// hardware conversion rounds to nearest even.  (A NaN block has inv = 0: NaN and infinity times 0
// are NaN, whose code is NaN too.)
__device__ __forceinline__ uint32_t mx_encode4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  return static_cast<uint32_t>(w);
}
// the values of the 8 codes of two words
__device__ __forceinline__ void mx_decode8(uint2 q, float s, float (&v)[8]) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q.x), false);
  const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q.x), true);
  const f32x2_t c = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q.y), false);
  const f32x2_t d = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q.y), true);
  v[0] = a.x * s; v[1] = a.y * s; v[2] = b.x * s; v[3] = b.y * s;
  v[4] = c.x * s; v[5] = c.y * s; v[6] = d.x * s; v[7] = d.y * s;
}

}  // namespace moe
