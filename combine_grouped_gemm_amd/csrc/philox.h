// Counter-based random numbers for dropout: Philox 4x32 with ten rounds (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  A number depends on its key and its
// counter alone, so a mask is computed wherever it is used and never stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// What of an element stays: the eight elements 8 i .. 8 i + 7 take the eight 16-bit halves (low first)
// of the four words of counter (i, offset) under the key seed; an element whose number is below cut is
// dropped, the others are multiplied by scale = 65536 / (65536 - cut).  16 bits an element instead of
// 32: the ten rounds are the operators' largest arithmetic, and a p rounded to 2^-16 (with the scale
// of the rounded p) costs no bias.
struct DropArgs {
  const uint64_t* rng;   // [2] seed, offset (device memory: a captured call reads what is there then)
  uint32_t cut;          // 0 .. 65536
  float scale;
};

__host__ inline DropArgs drop_args(double p, const uint64_t* rng) {
  DropArgs d;
  d.rng = rng;
  d.cut = static_cast<uint32_t>(p * 65536.0 + 0.5);
  d.scale = d.cut < 65536u ? 65536.0f / static_cast<float>(65536u - d.cut) : 0.0f;
  return d;
}

struct DropState {
  uint32_t k0, k1, o0, o1, cut;
  float scale;
};

__device__ __forceinline__ DropState drop_state(const DropArgs& d) {
  const uint64_t seed = d.rng[0], off = d.rng[1];
  return DropState{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(off),
                   static_cast<uint32_t>(off >> 32), d.cut, d.scale};
}

__device__ __forceinline__ uint4 philox(const DropState& d, uint64_t i) {
  uint32_t c0 = static_cast<uint32_t>(i), c1 = static_cast<uint32_t>(i >> 32), c2 = d.o0, c3 = d.o1;
  uint32_t k0 = d.k0, k1 = d.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t m0 = static_cast<uint64_t>(c0) * 0xD2511F53u, m2 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(m2 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(m2);
    c2 = static_cast<uint32_t>(m0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(m0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// v: elements 8 i .. 8 i + 7, dropped (0, whatever they held) or scaled; w: philox(d, i)
__device__ __forceinline__ void drop8(const DropState& d, uint4 w, float (&v)[8]) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t n = (j & 1) ? q[j / 2] >> 16 : q[j / 2] & 0xFFFFu;
    v[j] = n >= d.cut ? v[j] * d.scale : 0.0f;
  }
}

// masks over 8 loaded elements (4 words of two bf16 each, or 8 of fp32): all ones where drop8 keeps one
template <bool F32>
__device__ __forceinline__ void keep8(const DropState& d, uint4 w, uint32_t (&m)[F32 ? 8 : 4]) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool lo = (q[j] & 0xFFFFu) >= d.cut, hi = (q[j] >> 16) >= d.cut;
    if constexpr (F32) {
      m[2 * j] = lo ? ~0u : 0u;
      m[2 * j + 1] = hi ? ~0u : 0u;
    } else {
      m[j] = (lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
    }
  }
}

}  // namespace moe
