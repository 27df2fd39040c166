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
// Few rows (act_direct): a workgroup takes all rows of one expert and 32 columns and writes db itself.
// Bound by memory: 65536 rows of I 2048, gated, with h 309 us (5.2 TB/s); db alone of a plain product's
// 65536 x 7168 172 us (5.5 TB/s).
#include <type_traits>

#include "activation.h"
#include "moe_common.h"
#include "moe_launch.h"
#include "row_load.h"

namespace moe {
namespace {

constexpr int kActThreads = 256;
constexpr int kDirectThreads = 512, kDirectLanes = 4;   // few rows: lanes, and those of them along the columns

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

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// four sums of db's group i (4 columns)
__device__ __forceinline__ void put_db(const ActBwdArgs& p, size_t i, float4 s) {
  if (p.db_f32) reinterpret_cast<float4*>(p.db)[i] = s;
  else reinterpret_cast<uint2*>(p.db)[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// NT: dz and h past the caches.  DIRECT: workgroup y is an expert, and the sums go to db.
template <bool F32, bool GATED, bool NT, bool DIRECT>
__global__ __launch_bounds__(DIRECT ? kDirectThreads : kActThreads) void act_backward_kernel(ActBwdArgs p) {
  constexpr int kHalves = GATED ? 2 : 1, kThreads = DIRECT ? kDirectThreads : kActThreads;
  __shared__ float4 red[kThreads * 2 * kHalves];
  const int lx = DIRECT ? kDirectLanes : p.lx, tx = threadIdx.x % lx, ty = threadIdx.x / lx, ny = kThreads / lx;
  const int groups = p.N / 8, gw = groups * kHalves;   // 8-column groups of a row of d_out, of z
  const int g = blockIdx.x * lx + tx;
  const bool on = g < groups;
  const int c = DIRECT ? 0 : blockIdx.y;
  const int r0 = c * p.range, r1 = p.rows - r0 < p.range ? p.rows : r0 + p.range;
  int e = DIRECT ? blockIdx.y : 0, lo = 0, hi = p.rows;
  const int end = DIRECT ? e + 1 : p.E;
  if (!DIRECT && p.offsets != nullptr) {   // the first expert that ends behind r0
    const int lane = threadIdx.x & 63;   // (every wave counts the experts that end at or before r0)
    for (int b = 0; b < p.E; b += 64) e += __popcll(__ballot(b + lane < p.E && p.offsets[b + lane + 1] <= r0));
  }
  for (; e < end; ++e) {
    if (p.offsets != nullptr) {
      lo = clamp_row(p.offsets[e], p.rows);
      hi = clamp_row(p.offsets[e + 1], p.rows);
    }
    if (!DIRECT && lo >= r1) break;
    const int b0 = lo > r0 ? lo : r0, b1 = hi < r1 ? hi : r1;
    if (!DIRECT && b1 <= b0) continue;
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
    if (!DIRECT && p.part == nullptr) continue;
    // lanes of one column over ty, in order
    __syncthreads();   // (the last expert's sums have been read)
#pragma unroll
    for (int q = 0; q < 2 * kHalves; ++q)
      red[q * kThreads + threadIdx.x] =
          make_float4(sum[q / 2][4 * (q & 1)], sum[q / 2][4 * (q & 1) + 1], sum[q / 2][4 * (q & 1) + 2],
                      sum[q / 2][4 * (q & 1) + 3]);
    __syncthreads();
    if constexpr (DIRECT) {   // kParts lanes a group of 4 columns: a few sums each, then joined between lanes
      constexpr int kParts = kThreads / (kDirectLanes * 2 * kHalves);
      const int i = threadIdx.x / kParts, q = i / kDirectLanes, x = i % kDirectLanes, part = threadIdx.x % kParts;
      float4 s = red[q * kThreads + part * kDirectLanes + x];
#pragma unroll
      for (int y = part + kParts; y < kThreads / kDirectLanes; y += kParts)
        s = add4(s, red[q * kThreads + y * kDirectLanes + x]);
#pragma unroll
      for (int off = 1; off < kParts; off <<= 1)
        s = add4(s, make_float4(__shfl_xor(s.x, off, 64), __shfl_xor(s.y, off, 64), __shfl_xor(s.z, off, 64),
                                __shfl_xor(s.w, off, 64)));
      const int gg = blockIdx.x * kDirectLanes + x;
      if (part == 0 && gg < groups)
        put_db(p, 2 * (static_cast<size_t>(e) * gw + (q / 2) * groups + gg) + (q & 1), s);
    } else {
      for (int i = threadIdx.x; i < lx * 2 * kHalves; i += kThreads) {
        const int q = i / lx, x = i % lx, gg = blockIdx.x * lx + x;
        if (gg >= groups) continue;
        float4 s = red[q * kThreads + x];
        for (int y = 1; y < ny; ++y) s = add4(s, red[q * kThreads + y * lx + x]);
        const size_t at = static_cast<size_t>(c + e) * gw + (q / 2) * groups + gg;
        reinterpret_cast<float4*>(p.part)[2 * at + (q & 1)] = s;
      }
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
    for (int i = a; i < b; ++i) s = add4(s, q[static_cast<size_t>(i) * (Nw / 4)]);
  }
  red[wave][x] = s;
  __syncthreads();
  if (wave != 0 || col4 >= Nw / 4) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) s = add4(s, red[w][x]);
  put_db(p, static_cast<size_t>(e) * (Nw / 4) + col4, s);
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

// Whether one launch does all: a workgroup an expert and 32 columns, 128 rows at a time.  us of the two
// launches against it, experts of equal rows (all rows on one): 301 rows of 520 columns, fp32, GELU, 7 experts
// 10.8 (10.1) against 4.4 (7.5); 512 rows 11.1 (9.9) against 5.2 (11.2), 1024 rows 11.3 (11.7) against 8.1 (19.4);
// bf16, 512 rows of 4096: 7 experts 11.2 (10.3) against 7.7 (9.1), 24 experts 10.2 against 13.4; 300 rows of
// 28672, one expert 21.0 against 29.5.
bool act_direct(int rows, int Nw, int E) {
  return rows > 0 && rows <= 512 && static_cast<long long>(rows) * Nw <= 1 << 21 && (Nw + 31ll) / 32 * E <= 1280;
}

}  // namespace

size_t act_backward_ws_bytes(int rows, int Nw, int E) {
  if (rows <= 0 || act_direct(rows, Nw, E)) return 0;
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
  const int Nw = gated ? 2 * N : N;
  const bool direct = db != nullptr && act_direct(rows, Nw, E);
  p.lx = act_lx(N);
  const bool nt = stream_stores(static_cast<size_t>(rows) * N * (f32 ? 4 : 2) * (gated ? 2 : 1));
  p.range = direct ? rows : act_range(rows, Nw);
  if (rows > 0) {
    const int lx = direct ? kDirectLanes : p.lx;
    const dim3 grid((N / 8 + lx - 1) / lx, direct ? E : (rows + p.range - 1) / p.range);
    const dim3 block(direct ? kDirectThreads : kActThreads);
    auto go = [&](auto f, auto g) {
      constexpr bool F = decltype(f)::value, G = decltype(g)::value;
      if (direct) hipLaunchKernelGGL((act_backward_kernel<F, G, false, true>), grid, block, 0, s, p);
      else if (nt) hipLaunchKernelGGL((act_backward_kernel<F, G, true, false>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((act_backward_kernel<F, G, false, false>), grid, block, 0, s, p);
    };
    if (f32 && gated) go(std::true_type{}, std::true_type{});
    else if (f32) go(std::true_type{}, std::false_type{});
    else if (gated) go(std::false_type{}, std::true_type{});
    else go(std::false_type{}, std::false_type{});
  }
  if (db != nullptr && !direct)
    hipLaunchKernelGGL(bias_sum_kernel, dim3((Nw / 4 + 63) / 64, E), dim3(256), 0, s, p, Nw);
  return hipGetLastError();
}

}  // namespace moe
