// Gradient of the experts' activations and biases: for u = a W_e^T + b_e and h = act(u) (gated:
// h = act(u_g) u_u, u = (u_g, u_u))
//   du = d_out act'(u)           (gated: du_g = d_out u_u act'(u_g), du_u = d_out act(u_g))
//   db_e = sum of du over the rows of expert e
//   h recomputed (the next product's weight gradient reads it)
// One pass over the rows: a workgroup takes a range of rows and a block of columns, a lane 8 columns of
// every few rows.  It sums du (fp32, before du is rounded) over each expert's rows within its range,
// over its lanes in a fixed order, and writes one row of partial sums per (range, expert) that meet;
// a second kernel adds an expert's partial rows in order.  Range c and expert e meet in place c + e of
// the partial rows: along the rows either c or e grows by one, so no two pairs share a place.
#include <type_traits>

#include "activation.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "row_load.h"

namespace moe {
namespace {

constexpr int kActThreads = 256;

struct ActBwdArgs {
  const void* z;        // [rows, Nw] or null (act none, not gated)
  const void* d_out;    // [rows, N]
  const int32_t* offsets;   // [E + 1] or null (one expert: all rows)
  void* dz;             // [rows, Nw] or null
  void* h;              // [rows, N] or null
  float* part;          // [ranges + E, Nw] or null
  void* db;             // [E, Nw]
  int E, rows, N, act, range, lx, db_f32;
};

template <bool F32>
__device__ __forceinline__ void get8(const void* p, size_t i, float (&v)[8]) {   // 8 values of group i
  raw_values<F32>(load_group<F32>(p, i), v);
}

__device__ __forceinline__ int clamp_row(int r, int rows) { return r < 0 ? 0 : (r > rows ? rows : r); }

// NT: dz and h past the caches
template <bool F32, bool GATED, bool NT>
__global__ __launch_bounds__(kActThreads) void act_backward_kernel(ActBwdArgs p) {
  constexpr int kHalves = GATED ? 2 : 1;
  __shared__ float4 red[kActThreads * 2 * kHalves];
  const int lx = p.lx, tx = threadIdx.x % lx, ty = threadIdx.x / lx, ny = kActThreads / lx;
  const int groups = p.N / 8, gw = groups * kHalves;   // 8-column groups of a row of d_out, of z
  const int g = blockIdx.x * lx + tx;
  const bool on = g < groups;
  const int c = blockIdx.y;
  const int r0 = c * p.range, r1 = p.rows - r0 < p.range ? p.rows : r0 + p.range;
  int e = 0, lo = 0, hi = p.rows;
  if (p.offsets != nullptr) {   // the first expert that ends behind r0
    const int lane = threadIdx.x & 63;   // (every wave counts the experts that end at or before r0)
    for (int b = 0; b < p.E; b += 64) e += __popcll(__ballot(b + lane < p.E && p.offsets[b + lane + 1] <= r0));
  }
  for (; e < p.E; ++e) {
    if (p.offsets != nullptr) {
      lo = clamp_row(p.offsets[e], p.rows);
      hi = clamp_row(p.offsets[e + 1], p.rows);
    }
    if (lo >= r1) break;
    const int b0 = lo > r0 ? lo : r0, b1 = hi < r1 ? hi : r1;
    if (b1 <= b0) continue;
    float sum[kHalves][8] = {};
    if (on) {
#pragma unroll 2
      for (int r = b0 + ty; r < b1; r += ny) {
        float d[8], u[8], s[8];
        get8<F32>(p.d_out, static_cast<size_t>(r) * groups + g, d);
        if (GATED) {
          float w[8];
          get8<F32>(p.z, static_cast<size_t>(r) * gw + g, u);
          get8<F32>(p.z, static_cast<size_t>(r) * gw + groups + g, w);
          act8_slope<F32>(p.act, u, s);
          float h[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            h[i] = u[i] * w[i];
            s[i] = d[i] * w[i] * s[i];
            u[i] = d[i] * u[i];
            sum[0][i] += s[i];
            sum[kHalves - 1][i] += u[i];
          }
          if (p.dz != nullptr) {
            store_group<F32, NT>(p.dz, static_cast<size_t>(r) * gw + g, s);
            store_group<F32, NT>(p.dz, static_cast<size_t>(r) * gw + groups + g, u);
          }
          if (p.h != nullptr) store_group<F32, NT>(p.h, static_cast<size_t>(r) * groups + g, h);
        } else if (p.z != nullptr) {
          get8<F32>(p.z, static_cast<size_t>(r) * groups + g, u);
          act8_slope<F32>(p.act, u, s);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s[i] *= d[i];
            sum[0][i] += s[i];
          }
          if (p.dz != nullptr) store_group<F32, NT>(p.dz, static_cast<size_t>(r) * groups + g, s);
          if (p.h != nullptr) store_group<F32, NT>(p.h, static_cast<size_t>(r) * groups + g, u);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0][i] += d[i];
          if (p.dz != nullptr) store_group<F32, NT>(p.dz, static_cast<size_t>(r) * groups + g, d);
        }
      }
    }
    if (p.part == nullptr) continue;
    // lanes of one column over ty, in order
    __syncthreads();   // (the last expert's sums have been read)
#pragma unroll
    for (int q = 0; q < 2 * kHalves; ++q)
      red[q * kActThreads + threadIdx.x] =
          make_float4(sum[q / 2][4 * (q & 1)], sum[q / 2][4 * (q & 1) + 1], sum[q / 2][4 * (q & 1) + 2],
                      sum[q / 2][4 * (q & 1) + 3]);
    __syncthreads();
    for (int i = threadIdx.x; i < lx * 2 * kHalves; i += kActThreads) {
      const int q = i / lx, x = i % lx, gg = blockIdx.x * lx + x;
      if (gg >= groups) continue;
      float4 s = red[q * kActThreads + x];
      for (int y = 1; y < ny; ++y) {
        const float4 v = red[q * kActThreads + y * lx + x];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      const size_t at = static_cast<size_t>(c + e) * gw + (q / 2) * groups + gg;
      reinterpret_cast<float4*>(p.part)[2 * at + (q & 1)] = s;
    }
  }
}

// db_e: the partial rows of expert e, in order; 64 lanes of 4 columns, the ranges dealt to 4 waves
__global__ __launch_bounds__(256) void bias_sum_kernel(ActBwdArgs p, int Nw) {
  __shared__ float4 red[4][64];
  const int e = blockIdx.y, x = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col4 = blockIdx.x * 64 + x;
  int lo = 0, hi = p.rows;
  if (p.offsets != nullptr) {
    lo = clamp_row(p.offsets[e], p.rows);
    hi = clamp_row(p.offsets[e + 1], p.rows);
  }
  float4 s = make_float4(0, 0, 0, 0);
  if (hi > lo && col4 < Nw / 4) {
    const int c0 = lo / p.range, n = (hi - 1) / p.range - c0 + 1;
    const int a = n * wave / 4, b = n * (wave + 1) / 4;   // (a wave's share: consecutive ranges)
    const float4* q = reinterpret_cast<const float4*>(p.part) + static_cast<size_t>(c0 + e) * (Nw / 4) + col4;
#pragma unroll 8
    for (int i = a; i < b; ++i) {
      const float4 v = q[static_cast<size_t>(i) * (Nw / 4)];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  red[wave][x] = s;
  __syncthreads();
  if (wave != 0 || col4 >= Nw / 4) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float4 v = red[w][x];
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  const size_t at = static_cast<size_t>(e) * (Nw / 4) + col4;
  if (p.db_f32) reinterpret_cast<float4*>(p.db)[at] = s;
  else reinterpret_cast<uint2*>(p.db)[at] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// (the ranges follow from the columns of z, so that the workspace does not depend on what they mean)
int act_lx(int N) {   // lanes of a workgroup along the columns: a power of two up to 64
  int lx = 8;
  while (lx < 64 && lx < N / 8) lx *= 2;
  return lx;
}
// rows of a range: about 2048 workgroups, 4 rows (a workgroup goes through the experts of its range one
// after the other: with 8 rows a lane, 368 rows of 93 experts took 20 us) to 4096 rows
int act_range(int rows, int N) {
  const int lx = act_lx(N), ny = kActThreads / lx;
  const long long blocks = (N / 8 + lx - 1) / lx;
  long long r = (static_cast<long long>(rows) * blocks + 2047) / 2048;
  if (r > ny) r = (r + ny - 1) / ny * ny;
  const long long least = (rows + 32767ll) / 32768 > 4 ? (rows + 32767ll) / 32768 : 4;   // (grid y: 32768 ranges)
  const long long most = least > 4096 ? least : 4096;
  return static_cast<int>(r < least ? least : (r > most ? most : r));
}

}  // namespace

size_t act_backward_ws_bytes(int rows, int Nw, int E) {
  if (rows <= 0) return 0;
  const int range = act_range(rows, Nw);
  const size_t ranges = (static_cast<size_t>(rows) + range - 1) / range;
  return (ranges + E) * static_cast<size_t>(Nw) * 4;
}

hipError_t launch_act_backward(const void* z, const void* d_out, bool f32, const int32_t* offsets, int E, int rows,
                               int N, int act, bool gated, void* dz, void* db, bool db_f32, void* h, void* ws,
                               hipStream_t s) {
  ActBwdArgs p{};
  p.z = z;
  p.d_out = d_out;
  p.offsets = offsets;
  p.dz = dz;
  p.h = h;
  p.part = db != nullptr ? static_cast<float*>(ws) : nullptr;
  p.db = db;
  p.E = E;
  p.rows = rows;
  p.N = N;
  p.act = act;
  p.db_f32 = db_f32;
  p.lx = act_lx(N);
  const bool nt = stream_stores(static_cast<size_t>(rows) * N * (f32 ? 4 : 2) * (gated ? 2 : 1));
  p.range = rows > 0 ? act_range(rows, gated ? 2 * N : N) : 1;
  if (rows > 0) {
    const dim3 grid((N / 8 + p.lx - 1) / p.lx, (rows + p.range - 1) / p.range), block(kActThreads);
    auto go = [&](auto f, auto g) {
      constexpr bool F = decltype(f)::value, G = decltype(g)::value;
      if (nt) hipLaunchKernelGGL((act_backward_kernel<F, G, true>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((act_backward_kernel<F, G, false>), grid, block, 0, s, p);
    };
    if (f32 && gated) go(std::true_type{}, std::true_type{});
    else if (f32) go(std::true_type{}, std::false_type{});
    else if (gated) go(std::false_type{}, std::true_type{});
    else go(std::false_type{}, std::false_type{});
  }
  if (db != nullptr) {
    const int Nw = gated ? 2 * N : N;
    hipLaunchKernelGGL(bias_sum_kernel, dim3((Nw / 4 + 63) / 64, E), dim3(256), 0, s, p, Nw);
  }
  return hipGetLastError();
}

}  // namespace moe
