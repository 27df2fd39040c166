// Dropout at the layer's end, and its gradient:
//   combine      y_t = residual_t + D(sum_{j<k} g_{t,j} expert_out[send_pos[t*k+j]] (+ shared_out_t))
//   its gradient d = D(dy_t): d_expert_out[send_pos[s]] = g_s d, d_gate[s] = <d, expert_out[send_pos[s]]>, d_shared_t = d
//   rows         y = residual + D(x)
// D drops and scales element by element, from numbers that are computed where they are used (philox.h):
// the element's place in y is its counter, so forward and backward agree without a stored mask.
#include <type_traits>

#include "moe_common.h"
#include "moe_launch.h"
#include "philox.h"
#include "row_load.h"

namespace moe {
namespace {

constexpr int kDropThreads = 256;
constexpr long long kMostItems = (1ll << 32) - 1;   // work-items of a launch

__device__ __forceinline__ int in_rows(int r, int rows) { return r < rows ? r : -1; }   // (-1: no row)

// One workgroup takes a token and a span of its columns, a lane 8 columns; the rows are summed in slot
// order in batches of KMAX whose loads go out together, then the shared row, in fp32.
template <int KMAX, bool EO32, bool Y32>
__global__ __launch_bounds__(kDropThreads) void combine_dropout_kernel(
    const void* __restrict__ eo, int rows, int H, int k, const int32_t* __restrict__ send_pos,
    const float* __restrict__ gate,
    const void* __restrict__ shared, const void* residual, DropArgs drop, void* y, int spans) {
  const int t = blockIdx.x / spans, span = blockIdx.x % spans;
  const DropState ds = drop_state(drop);
  const int groups8 = H / 8;
  const int c = span * static_cast<int>(blockDim.x) + threadIdx.x;
  const int step = spans * static_cast<int>(blockDim.x);
  const int32_t* sp = send_pos + static_cast<size_t>(t) * k;
  const float* gp = gate + static_cast<size_t>(t) * k;
  for (int g8 = c; g8 < groups8; g8 += step) {
    const size_t at = static_cast<size_t>(t) * groups8 + g8;
    Raw8<EO32> sh;
    Raw8<Y32> re;
    if (shared != nullptr) sh = load_group<EO32>(shared, at);
    if (residual != nullptr) re = load_group<Y32>(residual, at);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < k; j0 += KMAX) {
      Raw8<EO32> b[KMAX];
      int r[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j) r[j] = j0 + j < k ? in_rows(sp[j0 + j], rows) : -1;
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (r[j] >= 0) b[j] = load_group<EO32>(eo, static_cast<size_t>(r[j]) * groups8 + g8);
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        if (r[j] < 0) continue;
        const float g = gate != nullptr ? gp[j0 + j] : 1.0f;
        float v[8];
        raw_values<EO32>(b[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(g, v[i], acc[i]);
      }
    }
    if (shared != nullptr) {
      float v[8];
      raw_values<EO32>(sh, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
    drop8(ds, philox(ds, at), acc);
    if (residual != nullptr) {
      float v[8];
      raw_values<Y32>(re, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
    store_group<Y32>(y, at, acc);
  }
}

// One workgroup takes a token: a lane forms d for its 8 columns once and goes through the token's rows
// in batches of KMAX (k > KMAX: d again for each batch, so d_shared, which may be dy, is written in the
// last one); the rows' dot products are kept per lane and summed over the workgroup at the end of a batch,
// in a fixed order.  8192 tokens of 7168, k 8, shared rows: 398 us (5.3 TB/s) with non-temporal stores of
// d_expert_out, 428 without.
template <int KMAX, bool DT32, bool DY32, bool NT>
__global__ void combine_dropout_backward_kernel(const void* dy, int rows, int H, int k,
                                                const int32_t* __restrict__ send_pos, const float* __restrict__ gate,
                                                const void* __restrict__ eo, DropArgs drop, void* __restrict__ d_eo,
                                                float* __restrict__ d_gate, void* d_shared) {
  __shared__ float red[16][KMAX];
  const int t = blockIdx.x;
  const DropState ds = drop_state(drop);
  const int groups8 = H / 8;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int32_t* sp = send_pos + static_cast<size_t>(t) * k;
  for (int j0 = 0; j0 < k; j0 += KMAX) {
    int r[KMAX];
    float g[KMAX], dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      r[j] = j0 + j < k ? in_rows(sp[j0 + j], rows) : -1;
      g[j] = gate != nullptr && j0 + j < k ? gate[static_cast<size_t>(t) * k + j0 + j] : 1.0f;
      dot[j] = 0.0f;
    }
    for (int g8 = threadIdx.x; g8 < groups8; g8 += blockDim.x) {
      const size_t at = static_cast<size_t>(t) * groups8 + g8;
      const Raw8<DY32> rd = load_group<DY32>(dy, at);
      Raw8<DT32> b[KMAX];
      if (d_gate != nullptr) {
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
          if (r[j] >= 0) b[j] = load_group<DT32>(eo, static_cast<size_t>(r[j]) * groups8 + g8);
      }
      const uint4 w = philox(ds, at);
      float d[8];
      raw_values<DY32>(rd, d);
      drop8(ds, w, d);
      uint32_t kept[DT32 ? 8 : 4];
      keep8<DT32>(ds, w, kept);
      if (d_shared != nullptr && j0 + KMAX >= k) store_group<DT32>(d_shared, at, d);
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        if (r[j] < 0) continue;
        float v[8];
        if (d_gate != nullptr) {
          mask_raw<DT32>(b[j], kept);   // (0 times an infinity would be NaN)
          raw_values<DT32>(b[j], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], v[i], dot[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = g[j] * d[i];
        store_group<DT32, NT>(d_eo, static_cast<size_t>(r[j]) * groups8 + g8, v);
      }
    }
    if (d_gate == nullptr) continue;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off, 64);
      if (lane == 0) red[wave][j] = dot[j];
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < KMAX && j0 + static_cast<int>(threadIdx.x) < k) {
      float s = 0.0f;   // (a slot without a row: 0)
      for (int w = 0; w < waves; ++w) s += red[w][threadIdx.x];
      d_gate[static_cast<size_t>(t) * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// groups of 8 elements, one a lane (more where n needs more lanes than a launch takes); the last n % 8
// elements one by one
template <bool X32, bool Y32>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(const void* x, long long n, DropArgs drop,
                                                               const void* residual,
                                                               void* y) {
  const DropState ds = drop_state(drop);
  const long long step = static_cast<long long>(gridDim.x) * kDropThreads;
  long long i = static_cast<long long>(blockIdx.x) * kDropThreads + threadIdx.x;
  for (; i < n / 8; i += step) {
    const Raw8<X32> a = load_group<X32>(x, i);
    Raw8<Y32> re;
    if (residual != nullptr) re = load_group<Y32>(residual, i);
    const uint4 w = philox(ds, i);
    float v[8];
    raw_values<X32>(a, v);
    drop8(ds, w, v);
    if (residual != nullptr) {
      float q[8];
      raw_values<Y32>(re, q);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += q[j];
    }
    store_group<Y32>(y, i, v);
  }
  if (i == n / 8 && n % 8 != 0) {
    const uint4 w = philox(ds, i);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int tail = static_cast<int>(n % 8);
    auto get = [](const void* p, bool f32, long long at) {
      return f32 ? reinterpret_cast<const float*>(p)[at] : bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[at]);
    };
    for (int j = 0; j < 8; ++j)
      if (j < tail) v[j] = get(x, X32, 8 * i + j);
    drop8(ds, w, v);
    for (int j = 0; j < 8; ++j) {
      if (j >= tail) break;
      if (residual != nullptr) v[j] += get(residual, Y32, 8 * i + j);
      if (Y32) reinterpret_cast<float*>(y)[8 * i + j] = v[j];
      else reinterpret_cast<uint16_t*>(y)[8 * i + j] = f32_to_bf16(v[j]);
    }
  }
}

template <typename F>
void two(bool a, bool b, F&& f) {
  if (a && b) f(std::true_type{}, std::true_type{});
  else if (a) f(std::true_type{}, std::false_type{});
  else if (b) f(std::false_type{}, std::true_type{});
  else f(std::false_type{}, std::false_type{});
}

}  // namespace

hipError_t launch_combine_dropout(const void* eo, bool eo_f32, int rows, int N, int H, int k, const int32_t* send_pos,
                                  const float* gate, const void* shared, const void* residual, double p,
                                  const uint64_t* rng, void* y, bool y_f32, hipStream_t s) {
  const int groups8 = H / 8;
  // one pass a lane: 8192 tokens of 7168, k 8, fp32 y and residual took 255 us (6.0 TB/s) with 7 workgroups of
  // 128 lanes a token, 300 with one of 7 passes; 256 lanes leave more of the last pass idle (270).  Few
  // tokens: workgroups of one wave
  const int threads = N < 1024 || groups8 <= 64 ? 64 : 128;
  const long long passes = (groups8 + threads - 1) / threads, most = kMostItems / threads / N;   // (N < 2^24: 2 or more)
  const int spans = static_cast<int>(passes < most ? passes : most);
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(N) * spans)), block(threads);
  const DropArgs d = drop_args(p, rng);
  two(eo_f32, y_f32, [&](auto a, auto b) {
    constexpr bool A = decltype(a)::value, B = decltype(b)::value;
    if (k <= 2)
      hipLaunchKernelGGL((combine_dropout_kernel<2, A, B>), grid, block, 0, s, eo, rows, H, k, send_pos, gate, shared,
                         residual, d, y, spans);
    else if (k <= 4)
      hipLaunchKernelGGL((combine_dropout_kernel<4, A, B>), grid, block, 0, s, eo, rows, H, k, send_pos, gate, shared,
                         residual, d, y, spans);
    else
      hipLaunchKernelGGL((combine_dropout_kernel<8, A, B>), grid, block, 0, s, eo, rows, H, k, send_pos, gate, shared,
                         residual, d, y, spans);
  });
  return hipGetLastError();
}

hipError_t launch_combine_dropout_backward(const void* dy, bool dy_f32, bool f32, int rows, int N, int H, int k,
                                           const int32_t* send_pos, const float* gate, const void* eo, double p,
                                           const uint64_t* rng, void* d_eo, float* d_gate, void* d_shared,
                                           hipStream_t s) {
  const int groups8 = H / 8;
  // few tokens: larger workgroups, up to the row's groups
  int threads = 256;
  while (threads < 1024 && threads < groups8 && N * (threads / 256) < 512) threads *= 2;
  const dim3 grid(static_cast<unsigned>(N)), block(threads);
  const bool nt = stream_stores(static_cast<size_t>(N) * k * H * (f32 ? 4 : 2));
  const DropArgs d = drop_args(p, rng);
  two(f32, dy_f32, [&](auto a, auto b) {
    constexpr bool A = decltype(a)::value, B = decltype(b)::value;
    auto go = [&](auto kmax, auto stream) {
      hipLaunchKernelGGL((combine_dropout_backward_kernel<decltype(kmax)::value, A, B, decltype(stream)::value>), grid,
                         block, 0, s, dy, rows, H, k, send_pos, gate, eo, d, d_eo, d_gate, d_shared);
    };
    auto size = [&](auto stream) {
      if (k <= 2) go(std::integral_constant<int, 2>{}, stream);
      else if (k <= 4) go(std::integral_constant<int, 4>{}, stream);
      else go(std::integral_constant<int, 8>{}, stream);
    };
    if (nt) size(std::true_type{});
    else size(std::false_type{});
  });
  return hipGetLastError();
}

hipError_t launch_dropout(const void* x, bool x_f32, long long n, double p, const uint64_t* rng, const void* residual,
                          void* y, bool y_f32, hipStream_t s) {
  const long long groups = ((n + 7) / 8 + kDropThreads - 1) / kDropThreads;
  const dim3 grid(static_cast<unsigned>(groups < kMostItems / kDropThreads ? groups : kMostItems / kDropThreads));
  const dim3 block(kDropThreads);
  const DropArgs d = drop_args(p, rng);
  two(x_f32, y_f32, [&](auto a, auto b) {
    constexpr bool A = decltype(a)::value, B = decltype(b)::value;
    hipLaunchKernelGGL((dropout_kernel<A, B>), grid, block, 0, s, x, n, d, residual, y);
  });
  return hipGetLastError();
}

}  // namespace moe
