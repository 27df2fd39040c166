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

#include "gemm_device.h"
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
// The 8-bit codes of one 32-column block of an output row, whose 16 values in lane l are
// columns 8 q + 0..3 (l < 32) or 8 q + 4..7 in register group q, and the other 16 in lane l ^ 32:
// of the values rounded to bf16, as the quantizer of bf16 rows would read them.  Returns 16 codes
// in column order, columns 0..15 in lane l < 32 and 16..31 in lane l + 32; byte: the block's scale.
// Every lane must take part.
__device__ __forceinline__ uint4 block_codes(const f32x16_t& v, uint32_t& byte) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  uint32_t w[8], m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    const uint32_t lo = (w[i] << 16) & 0x7FFFFFFFu, hi = w[i] & 0x7FFF0000u;
    m = m > lo ? m : lo;
    m = m > hi ? m : hi;
  }
  const u32x2_t mm = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  byte = mx_scale_byte(mm[0] > mm[1] ? mm[0] : mm[1]);
  const float inv = mx_inverse(byte);
  uint32_t c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    c[q] = mx_encode4(__uint_as_float(w[2 * q] << 16), __uint_as_float(w[2 * q] & 0xFFFF0000u),
                      __uint_as_float(w[2 * q + 1] << 16), __uint_as_float(w[2 * q + 1] & 0xFFFF0000u), inv);
  // (each swap exchanges its second operand in lanes l < 32 with its first in lanes l + 32)
  const u32x2_t a = __builtin_amdgcn_permlane32_swap(c[0], c[1], false, false);   // columns 0..7 | 8..15
  const u32x2_t b = __builtin_amdgcn_permlane32_swap(c[2], c[3], false, false);   // 16..23 | 24..31
  const u32x2_t x = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const u32x2_t y = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  return make_uint4(x[0], y[0], x[1], y[1]);
}
// the values of the 4 codes of a word
__device__ __forceinline__ void mx_decode4(uint32_t q, float s, float& v0, float& v1, float& v2, float& v3) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q), false);
  const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q), true);
  v0 = a.x * s; v1 = a.y * s; v2 = b.x * s; v3 = b.y * s;
}
// the values of the 8 codes of two words
__device__ __forceinline__ void mx_decode8(uint2 q, float s, float (&v)[8]) {
  mx_decode4(q.x, s, v[0], v[1], v[2], v[3]);
  mx_decode4(q.y, s, v[4], v[5], v[6], v[7]);
}

}  // namespace moe
