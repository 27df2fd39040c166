// Loads and stores of 8 adjacent columns of a row of fp32 or bf16, shared by the kernels that move rows.
#pragma once

#include "moe_common.h"

namespace moe {

template <bool kEoF32>
__device__ __forceinline__ void load8(const void* base, size_t row, int H, int c, float (&v)[8]) {
  if (kEoF32) {
    const float4* p = reinterpret_cast<const float4*>(base) + (row * H) / 4 + 2 * c;
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(base)[(row * H) / 8 + c];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(static_cast<uint16_t>(w[i] & 0xFFFFu));
      v[2 * i + 1] = bf16_to_f32(static_cast<uint16_t>(w[i] >> 16));
    }
  }
}

// 8 columns of one row as loaded: one 16-byte word (bf16) or two (fp32)
template <bool kEoF32>
struct Raw8 {
  uint4 w[kEoF32 ? 2 : 1];
};

// streaming 16-byte load: every expert row and shared row is read exactly once, so the
// loads carry the non-temporal hint (measured: a 9-rows-read-per-row-written stream moves
// ~10% more bytes per second with it)
typedef uint32_t stream_word_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  const stream_word_t v = __builtin_nontemporal_load(reinterpret_cast<const stream_word_t*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}

// NT: the non-temporal hint (rows read once); otherwise plain loads (rows read by many
// tokens, such as the router weight's rows in the router's input gradient)
template <bool NT>
__device__ __forceinline__ uint4 load_row16(const uint4* p) {
  if (NT) return load_stream(p);
  return *p;
}

template <bool kEoF32, bool NT>
__device__ __forceinline__ void raw_load(const void* base, size_t row, int H, int c, Raw8<kEoF32>& r) {
  if (kEoF32) {
    const uint4* p = reinterpret_cast<const uint4*>(base) + (row * H) / 4 + 2 * c;
    r.w[0] = load_row16<NT>(p);
    r.w[kEoF32 ? 1 : 0] = load_row16<NT>(p + 1);
  } else {
    r.w[0] = load_row16<NT>(reinterpret_cast<const uint4*>(base) + (row * H) / 8 + c);
  }
}

template <bool kEoF32>
__device__ __forceinline__ void raw_values(const Raw8<kEoF32>& r, float (&v)[8]) {
  if (kEoF32) {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w,
                           r.w[kEoF32 ? 1 : 0].x, r.w[kEoF32 ? 1 : 0].y, r.w[kEoF32 ? 1 : 0].z, r.w[kEoF32 ? 1 : 0].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(static_cast<uint16_t>(w[i] & 0xFFFFu));
      v[2 * i + 1] = bf16_to_f32(static_cast<uint16_t>(w[i] >> 16));
    }
  }
}

// the loaded columns whose mask is 0 (keep8 of philox.h) become 0, whatever they held
template <bool F32>
__device__ __forceinline__ void mask_raw(Raw8<F32>& r, const uint32_t (&m)[F32 ? 8 : 4]) {
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    r.w[i].x &= m[4 * i];
    r.w[i].y &= m[4 * i + 1];
    r.w[i].z &= m[4 * i + 2];
    r.w[i].w &= m[4 * i + 3];
  }
}

// 8 values (8 adjacent elements) to group i of a matrix of fp32 or bf16; NT: with the non-temporal hint (a
// constant: of two branches that differ in the hint alone the compiler makes one, without it)
template <bool F32, bool NT = false>
__device__ __forceinline__ void store_group(void* p, size_t i, const float (&v)[8]) {
  typedef float f32x4s_t __attribute__((ext_vector_type(4)));
  if (F32) {
    f32x4s_t* q = reinterpret_cast<f32x4s_t*>(p) + 2 * i;
    const f32x4s_t a{v[0], v[1], v[2], v[3]}, b{v[4], v[5], v[6], v[7]};
    if constexpr (NT) {
      __builtin_nontemporal_store(a, q);
      __builtin_nontemporal_store(b, q + 1);
    } else {
      q[0] = a;
      q[1] = b;
    }
  } else {
    const stream_word_t w{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7])};
    stream_word_t* q = reinterpret_cast<stream_word_t*>(p) + i;
    if constexpr (NT) __builtin_nontemporal_store(w, q);
    else *q = w;
  }
}
// whether an output of this many bytes is written past the caches: from the 256 MB that the last-level
// cache holds on, what is written first is gone before the next kernel reads it
__host__ inline bool stream_stores(size_t bytes) { return bytes >= (size_t{256} << 20); }

template <bool F32>
__device__ __forceinline__ Raw8<F32> load_group(const void* p, size_t i) {   // 8 values of group i, read once
  Raw8<F32> r;
  if (F32) {
    r.w[0] = load_stream(reinterpret_cast<const uint4*>(p) + 2 * i);
    r.w[F32 ? 1 : 0] = load_stream(reinterpret_cast<const uint4*>(p) + 2 * i + 1);
  } else {
    r.w[0] = load_stream(reinterpret_cast<const uint4*>(p) + i);
  }
  return r;
}

}  // namespace moe
