// Activations kept in 8 bits between forward and backward (mxfp8.h has the format), and the
// SwiGLU backward that reads them.
//
//   quantize     codes and scale bytes of rows of bf16 or fp32 values
//   dequantize   the values, as they lie or scattered to a token's k expert-ordered rows
//   SwiGLU       s = 1 / (1 + e^-a), h = a s u of the kept pre-activations (a, u); with dh = dy W_down
//                of the UNGATED upstream gradient and the row's gate g
//                  d_gate = <dh, h>,  da = g dh u s (1 + a (1 - s)),  du = g dh a s,  h_out = g h
//
// The gates' gradient needs no expert outputs: <dy, W_down h> = <W_down^T dy, h>.  With g folded
// into h_out the weight gradient is dW_down = dy^T (g h) over the plain permuted dy.
//
// All three move each byte once and are bound by memory; a lane takes 8 adjacent columns (8 bytes of
// codes, 16 of bf16), four lanes a block, so that a wave's accesses are contiguous, and every stream
// is touched once (non-temporal).  Measured, bf16: 8191 x 7168 quantized in 31 us (5.8 TB/s) and
// written to 8 expert-ordered rows each in 178 us (5.6 TB/s); SwiGLU backward of 65536 slots of I
// 2048 with gates in 266 us (5.06 TB/s; a 1 GiB copy on the card: 5.15).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_common.h"
#include "moe_launch.h"
#include "mxfp8.h"

namespace moe {
namespace {

constexpr int kCkThreads = 256;

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

// 8 adjacent values at 8-column group i
template <bool F32>
__device__ __forceinline__ void load8(const void* p, size_t i, float (&v)[8]) {
  if constexpr (F32) {
    const u32x4v a = __builtin_nontemporal_load(reinterpret_cast<const u32x4v*>(p) + 2 * i);
    const u32x4v b = __builtin_nontemporal_load(reinterpret_cast<const u32x4v*>(p) + 2 * i + 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(a[j]);
      v[4 + j] = __uint_as_float(b[j]);
    }
  } else {
    const u32x4v a = __builtin_nontemporal_load(reinterpret_cast<const u32x4v*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(a[j] << 16);
      v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, size_t i, const float (&v)[8]) {
  if constexpr (F32) {
    u32x4v a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __float_as_uint(v[j]);
      b[j] = __float_as_uint(v[4 + j]);
    }
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4v*>(p) + 2 * i);
    __builtin_nontemporal_store(b, reinterpret_cast<u32x4v*>(p) + 2 * i + 1);
  } else {
    const u32x4v a = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7])};
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4v*>(p) + i);
  }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* q, size_t i) {
  const u32x2v w = __builtin_nontemporal_load(reinterpret_cast<const u32x2v*>(q) + i);
  return make_uint2(w[0], w[1]);
}

// Rows of cols % 32 == 0 columns lie one after the other, so blocks never straddle rows and the
// tensor is a flat run of n8 groups of 8 columns (4 groups a block).
template <bool F32>
__global__ __launch_bounds__(kCkThreads) void quantize_mx_kernel(const void* __restrict__ x, long long n8,
                                                                 uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const long long stride = static_cast<long long>(gridDim.x) * kCkThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kCkThreads + threadIdx.x; i < n8; i += stride) {
    float v[8];
    load8<F32>(x, i, v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
      m = b > m ? b : m;
    }
    // (n8 % 4 == 0: the four lanes of a block are all active)
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      const uint32_t o = __shfl_xor(m, off, kWave);
      m = o > m ? o : m;
    }
    const uint32_t byte = mx_scale_byte(m);
    const float inv = mx_inverse(byte);
    const u32x2v w = {mx_encode4(v[0], v[1], v[2], v[3], inv), mx_encode4(v[4], v[5], v[6], v[7], inv)};
    reinterpret_cast<u32x2v*>(q)[i] = w;
    if ((i & 3) == 0) scale[i >> 2] = static_cast<uint8_t>(byte);
  }
}

template <bool F32>
__global__ __launch_bounds__(kCkThreads) void dequantize_mx_kernel(const uint8_t* __restrict__ q,
                                                                   const uint8_t* __restrict__ scale, long long n8,
                                                                   void* __restrict__ out) {
  const long long stride = static_cast<long long>(gridDim.x) * kCkThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kCkThreads + threadIdx.x; i < n8; i += stride) {
    float v[8];
    mx_decode8(load_codes(q, i), mx_scale(scale[i >> 2]), v);
    store8<F32>(out, i, v);
  }
}

// one workgroup per token: its values to the k rows its slots name (negative positions: no row)
template <bool F32>
__global__ __launch_bounds__(kCkThreads) void dequantize_rows_mx_kernel(const uint8_t* __restrict__ q,
                                                                        const uint8_t* __restrict__ scale, int cols8,
                                                                        int k, const int32_t* __restrict__ send_pos,
                                                                        long long out_rows, void* __restrict__ out) {
  const size_t t = blockIdx.x;
  for (int c = threadIdx.x; c < cols8; c += kCkThreads) {
    const size_t i = t * cols8 + c;
    float v[8];
    mx_decode8(load_codes(q, i), mx_scale(scale[i >> 2]), v);
    for (int j = 0; j < k; ++j) {
      const int r = send_pos[t * k + j];
      if (r < 0 || r >= out_rows) continue;
      store8<F32>(out, static_cast<size_t>(r) * cols8 + c, v);
    }
  }
}

// TPR threads per slot (16, a wave, or the workgroup): slot s is row send_pos[s] (or s)
template <bool F32, int TPR>
__global__ __launch_bounds__(kCkThreads) void swiglu_backward_mx_kernel(
    const uint8_t* __restrict__ au, const uint8_t* __restrict__ au_scale, const void* __restrict__ dh, int rows, int I,
    int slots, const int32_t* __restrict__ send_pos, const float* __restrict__ gate, void* __restrict__ d_au,
    void* __restrict__ h, float* __restrict__ d_gate) {
  constexpr int kPer = kCkThreads / TPR;
  __shared__ float red[kCkThreads / kWave];
  const int l = threadIdx.x % TPR;
  const long long s = static_cast<long long>(blockIdx.x) * kPer + threadIdx.x / TPR;
  if (s >= slots) return;   // (TPR = 256: the whole workgroup)
  const long long r = send_pos != nullptr ? send_pos[s] : s;
  if (r < 0 || r >= rows) {   // a dropped slot
    if (l == 0 && d_gate != nullptr) d_gate[s] = 0.0f;
    return;
  }
  const float g = gate != nullptr ? gate[s] : 1.0f;
  const int c8 = I / 8;       // 8-column groups of a half row
  const size_t a0 = static_cast<size_t>(r) * 2 * c8, h0 = static_cast<size_t>(r) * c8;
  float dot = 0.0f;
  for (int c = l; c < c8; c += TPR) {
    float a[8], u[8], d[8], da[8], du[8], hv[8];
    const uint2 qa = load_codes(au, a0 + c), qu = load_codes(au, a0 + c8 + c);
    const uint32_t ba = au_scale[(a0 + c) >> 2], bu = au_scale[(a0 + c8 + c) >> 2];
    load8<F32>(dh, h0 + c, d);
    mx_decode8(qa, mx_scale(ba), a);
    mx_decode8(qu, mx_scale(bu), u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sg = sigmoid_f32(a[j]);
      const float as = a[j] * sg, hj = as * u[j], gd = g * d[j];
      dot = fmaf(d[j], hj, dot);
      da[j] = gd * u[j] * fmaf(as, 1.0f - sg, sg);
      du[j] = gd * as;
      hv[j] = g * hj;
    }
    store8<F32>(d_au, a0 + c, da);
    store8<F32>(d_au, a0 + c8 + c, du);
    store8<F32>(h, h0 + c, hv);
  }
  if (d_gate == nullptr) return;   // (uniform)
  constexpr int kSpan = TPR < kWave ? TPR : kWave;
#pragma unroll
  for (int off = kSpan / 2; off > 0; off >>= 1) dot += __shfl_xor(dot, off, kWave);
  if constexpr (TPR > kWave) {
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = dot;
    __syncthreads();
    dot = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / kWave; ++w) dot += red[w];
  }
  if (l == 0) d_gate[s] = dot;
}

unsigned flat_grid(long long n8) {
  const long long b = (n8 + kCkThreads - 1) / kCkThreads;
  return static_cast<unsigned>(b < 16384 ? b : 16384);
}

}  // namespace

hipError_t launch_quantize_mx(const void* x, bool f32, long long rows, int cols, uint8_t* q, uint8_t* scale,
                              hipStream_t s) {
  const long long n8 = rows * (cols / 8);
  if (f32)
    hipLaunchKernelGGL(quantize_mx_kernel<true>, dim3(flat_grid(n8)), dim3(kCkThreads), 0, s, x, n8, q, scale);
  else
    hipLaunchKernelGGL(quantize_mx_kernel<false>, dim3(flat_grid(n8)), dim3(kCkThreads), 0, s, x, n8, q, scale);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx(const uint8_t* q, const uint8_t* scale, long long rows, int cols, int k,
                                const int32_t* send_pos, long long out_rows, void* out, bool f32, hipStream_t s) {
  if (send_pos != nullptr) {
    const dim3 grid(static_cast<unsigned>(rows));
    if (f32)
      hipLaunchKernelGGL(dequantize_rows_mx_kernel<true>, grid, dim3(kCkThreads), 0, s, q, scale, cols / 8, k,
                         send_pos, out_rows, out);
    else
      hipLaunchKernelGGL(dequantize_rows_mx_kernel<false>, grid, dim3(kCkThreads), 0, s, q, scale, cols / 8, k,
                         send_pos, out_rows, out);
    return hipGetLastError();
  }
  const long long n8 = rows * (cols / 8);
  if (f32)
    hipLaunchKernelGGL(dequantize_mx_kernel<true>, dim3(flat_grid(n8)), dim3(kCkThreads), 0, s, q, scale, n8, out);
  else
    hipLaunchKernelGGL(dequantize_mx_kernel<false>, dim3(flat_grid(n8)), dim3(kCkThreads), 0, s, q, scale, n8, out);
  return hipGetLastError();
}

template <bool F32>
static hipError_t swiglu_mx(const uint8_t* au, const uint8_t* au_scale, const void* dh, int rows, int I, int slots,
                            const int32_t* send_pos, const float* gate, void* d_au, void* h, float* d_gate,
                            hipStream_t s) {
#define MOE_SWIGLU_MX(TPR_)                                                                                       \
  hipLaunchKernelGGL((swiglu_backward_mx_kernel<F32, TPR_>),                                                      \
                     dim3(static_cast<unsigned>((static_cast<long long>(slots) * TPR_ + kCkThreads - 1) / kCkThreads)), \
                     dim3(kCkThreads), 0, s, au, au_scale, dh, rows, I, slots, send_pos, gate, d_au, h, d_gate)
  // lanes of a slot by its width (us with 16 / 64 / 256 lanes):
  //   65536 slots of I 64: 10 / 24 / 53, of I 256: 31 / 31 / 64, of I 512: 62 / 56 / 69,
  //   of I 2048: 257 / 224 / 226; 256 slots of I 2048: 11 / 4.6 / 3.1, of I 14336: 93 / 28 / 12
  if (I <= 256) MOE_SWIGLU_MX(16);
  else if (I < 2048) MOE_SWIGLU_MX(64);
  else MOE_SWIGLU_MX(256);
#undef MOE_SWIGLU_MX
  return hipGetLastError();
}

hipError_t launch_swiglu_backward_mx(const uint8_t* au, const uint8_t* au_scale, const void* dh, bool f32, int rows,
                                     int I, int slots, const int32_t* send_pos, const float* gate, void* d_au, void* h,
                                     float* d_gate, hipStream_t s) {
  return f32 ? swiglu_mx<true>(au, au_scale, dh, rows, I, slots, send_pos, gate, d_au, h, d_gate, s)
             : swiglu_mx<false>(au, au_scale, dh, rows, I, slots, send_pos, gate, d_au, h, d_gate, s);
}

}  // namespace moe
