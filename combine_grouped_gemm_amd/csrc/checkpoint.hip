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
// All three move each byte once and are bound by memory; a lane takes 16 bytes of adjacent values (8
// columns of bf16, 4 of fp32), four or eight lanes a block, so that a wave's accesses are contiguous, and every stream
// is touched once (non-temporal).  Measured, bf16: 8191 x 7168 quantized in 31 us (5.8 TB/s) and
// written to 8 expert-ordered rows each in 178 us (5.6 TB/s); SwiGLU backward of 65536 slots of I
// 2048 with gates in 255 us (5.3 TB/s; a 1 GiB copy on the card: 5.15).  fp32: 15672 slots of I 6688
// in 376 us (5.0 TB/s), 8191 x 4096 quantized and written to 4 rows each in 143 us (5.2 TB/s).
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

// Columns of a lane: 16 bytes of values, so that a wave's access is contiguous (fp32 with 8 columns a
// lane writes every second 16 bytes at a time: 3.4 TB/s in the SwiGLU backward)
template <bool F32>
constexpr int kCols = F32 ? 4 : 8;

// the adjacent values at column group i
template <bool F32>
__device__ __forceinline__ void load_cols(const void* p, size_t i, float (&v)[kCols<F32>]) {
  const u32x4v a = __builtin_nontemporal_load(reinterpret_cast<const u32x4v*>(p) + i);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (F32) {
      v[j] = __uint_as_float(a[j]);
    } else {
      v[2 * j] = __uint_as_float(a[j] << 16);
      v[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void store_cols(void* p, size_t i, const float (&v)[kCols<F32>]) {
  u32x4v a;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (F32) a[j] = __float_as_uint(v[j]);
    else a[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  }
  __builtin_nontemporal_store(a, reinterpret_cast<u32x4v*>(p) + i);
}
template <bool F32>
__device__ __forceinline__ uint2 load_codes(const uint8_t* q, size_t i) {
  if constexpr (F32) return make_uint2(__builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q) + i), 0u);
  const u32x2v w = __builtin_nontemporal_load(reinterpret_cast<const u32x2v*>(q) + i);
  return make_uint2(w[0], w[1]);
}
template <bool F32>
__device__ __forceinline__ void decode_cols(uint2 q, float s, float (&v)[kCols<F32>]) {
  if constexpr (F32) mx_decode4(q.x, s, v[0], v[1], v[2], v[3]);
  else mx_decode8(q, s, v);
}
template <bool F32>
__device__ __forceinline__ size_t block_of(size_t i) { return i / (32 / kCols<F32>); }

// Rows of cols % 32 == 0 columns lie one after the other, so blocks never straddle rows and the
// tensor is a flat run of n column groups (4 or 8 a block).
template <bool F32>
__global__ __launch_bounds__(kCkThreads) void quantize_mx_kernel(const void* __restrict__ x, long long n,
                                                                 uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  constexpr int V = kCols<F32>;
  const long long stride = static_cast<long long>(gridDim.x) * kCkThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kCkThreads + threadIdx.x; i < n; i += stride) {
    float v[V];
    load_cols<F32>(x, i, v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
      m = b > m ? b : m;
    }
    // (n is a multiple of a block's groups: the lanes of a block are all active)
#pragma unroll
    for (int off = 1; off < 32 / V; off <<= 1) {
      const uint32_t o = __shfl_xor(m, off, kWave);
      m = o > m ? o : m;
    }
    const uint32_t byte = mx_scale_byte(m);
    const float inv = mx_inverse(byte);
    if constexpr (F32) {
      reinterpret_cast<uint32_t*>(q)[i] = mx_encode4(v[0], v[1], v[2], v[3], inv);
    } else {
      const u32x2v w = {mx_encode4(v[0], v[1], v[2], v[3], inv), mx_encode4(v[4], v[5], v[6], v[7], inv)};
      reinterpret_cast<u32x2v*>(q)[i] = w;
    }
    if (i % (32 / V) == 0) scale[block_of<F32>(i)] = static_cast<uint8_t>(byte);
  }
}

template <bool F32>
__global__ __launch_bounds__(kCkThreads) void dequantize_mx_kernel(const uint8_t* __restrict__ q,
                                                                   const uint8_t* __restrict__ scale, long long n,
                                                                   void* __restrict__ out) {
  const long long stride = static_cast<long long>(gridDim.x) * kCkThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kCkThreads + threadIdx.x; i < n; i += stride) {
    float v[kCols<F32>];
    decode_cols<F32>(load_codes<F32>(q, i), mx_scale(scale[block_of<F32>(i)]), v);
    store_cols<F32>(out, i, v);
  }
}

// TPT threads per token (a wave or the workgroup): its values to the k rows its slots name (negative
// positions: no row); groups: column groups of a row
template <bool F32, int TPT>
__global__ __launch_bounds__(kCkThreads) void dequantize_rows_mx_kernel(const uint8_t* __restrict__ q,
                                                                        const uint8_t* __restrict__ scale,
                                                                        long long rows, int groups, int k,
                                                                        const int32_t* __restrict__ send_pos,
                                                                        long long out_rows, void* __restrict__ out) {
  const long long t = static_cast<long long>(blockIdx.x) * (kCkThreads / TPT) + threadIdx.x / TPT;
  if (t >= rows) return;
  for (int c = threadIdx.x % TPT; c < groups; c += TPT) {
    const size_t i = static_cast<size_t>(t) * groups + c;
    float v[kCols<F32>];
    decode_cols<F32>(load_codes<F32>(q, i), mx_scale(scale[block_of<F32>(i)]), v);
    for (int j = 0; j < k; ++j) {
      const int r = send_pos[t * k + j];
      if (r < 0 || r >= out_rows) continue;
      store_cols<F32>(out, static_cast<size_t>(r) * groups + c, v);
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
  constexpr int V = kCols<F32>;
  const int n = I / V;        // column groups of a half row
  const size_t a0 = static_cast<size_t>(r) * 2 * n, h0 = static_cast<size_t>(r) * n;
  float dot = 0.0f;
  for (int c = l; c < n; c += TPR) {
    float a[V], u[V], d[V], da[V], du[V], hv[V];
    const uint2 qa = load_codes<F32>(au, a0 + c), qu = load_codes<F32>(au, a0 + n + c);
    const uint32_t ba = au_scale[block_of<F32>(a0 + c)], bu = au_scale[block_of<F32>(a0 + n + c)];
    load_cols<F32>(dh, h0 + c, d);
    decode_cols<F32>(qa, mx_scale(ba), a);
    decode_cols<F32>(qu, mx_scale(bu), u);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float sg = sigmoid_f32(a[j]);
      const float as = a[j] * sg, hj = as * u[j], gd = g * d[j];
      dot = fmaf(d[j], hj, dot);
      da[j] = gd * u[j] * fmaf(as, 1.0f - sg, sg);
      du[j] = gd * as;
      hv[j] = g * hj;
    }
    store_cols<F32>(d_au, a0 + c, da);
    store_cols<F32>(d_au, a0 + n + c, du);
    store_cols<F32>(h, h0 + c, hv);
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

unsigned flat_grid(long long n) {
  const long long b = (n + kCkThreads - 1) / kCkThreads;
  return static_cast<unsigned>(b < 16384 ? b : 16384);
}

}  // namespace

hipError_t launch_quantize_mx(const void* x, bool f32, long long rows, int cols, uint8_t* q, uint8_t* scale,
                              hipStream_t s) {
  const long long n = rows * (cols / (f32 ? kCols<true> : kCols<false>));
  if (f32)
    hipLaunchKernelGGL(quantize_mx_kernel<true>, dim3(flat_grid(n)), dim3(kCkThreads), 0, s, x, n, q, scale);
  else
    hipLaunchKernelGGL(quantize_mx_kernel<false>, dim3(flat_grid(n)), dim3(kCkThreads), 0, s, x, n, q, scale);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx(const uint8_t* q, const uint8_t* scale, long long rows, int cols, int k,
                                const int32_t* send_pos, long long out_rows, void* out, bool f32, hipStream_t s) {
  if (send_pos != nullptr) {
    const int groups = cols / (f32 ? kCols<true> : kCols<false>);
#define MOE_DEQUANTIZE_ROWS(F32_, TPT_)                                                                            \
  hipLaunchKernelGGL((dequantize_rows_mx_kernel<F32_, TPT_>),                                                      \
                     dim3(static_cast<unsigned>((rows * TPT_ + kCkThreads - 1) / kCkThreads)), dim3(kCkThreads), 0, s, q, \
                     scale, rows, groups, k, send_pos, out_rows, out)
    // a wave per token while the row is one pass of it (us with 256 / 64 threads, bf16, 30000 rows: 256 columns
    // to 1 row 10.6 / 7.4, to 8 rows 41 / 28; 512 columns 13.9 / 10.2, 54 / 46; 1024 columns 20 / 18, 97 / 99;
    // 300 rows of 1024 columns to 8 rows 3.7 / 5.4)
    const bool wave = groups <= kWave;
    if (f32 && wave) MOE_DEQUANTIZE_ROWS(true, kWave);
    else if (f32) MOE_DEQUANTIZE_ROWS(true, kCkThreads);
    else if (wave) MOE_DEQUANTIZE_ROWS(false, kWave);
    else MOE_DEQUANTIZE_ROWS(false, kCkThreads);
#undef MOE_DEQUANTIZE_ROWS
    return hipGetLastError();
  }
  const long long n = rows * (cols / (f32 ? kCols<true> : kCols<false>));
  if (f32)
    hipLaunchKernelGGL(dequantize_mx_kernel<true>, dim3(flat_grid(n)), dim3(kCkThreads), 0, s, q, scale, n, out);
  else
    hipLaunchKernelGGL(dequantize_mx_kernel<false>, dim3(flat_grid(n)), dim3(kCkThreads), 0, s, q, scale, n, out);
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
