// The experts' product with its epilogue ("MoE part 4" page, section 2: one launch for many expert GEMMs
// with differing row counts), for experts with biases and any activation:
//
//   u[r] = a[r'] . W_e^T + b_e,   out[r] = act(u[r]) (+ residual[r])            r in segment e
//   gated: out[r] = act(u[r, 0 .. N-1]) * u[r, N .. 2N-1] (+ residual[r])
//
// r' = r, or the token src_slot[r] / k.  u is kept on demand (training).  Sizes are multiples of 8; the
// products are bf16 with fp32 sums, or fp32.
//
// A workgroup computes TM rows x TN weight rows (gated: TN / 2 rows of either half, so that a lane holds
// both factors).  K advances in stages of 128 bytes a row (64 bf16, 32 fp32), loaded straight to LDS
// through buffer windows: rows past the segment, weight rows past the matrix and columns past K read as
// zeros, so no size needs a kernel of its own.  Chunk c of 16 bytes of row r lies in slot c ^ key(r), so
// that a load (8 rows) and a fragment read (32 rows, two chunks) touch every bank once.  A fragment is one
// chunk a lane for either type: 8 bf16 for one 32x32x16 product, 4 fp32 for four 32x32x2 ones (both
// operands take their k in the same order).  The weights are the first operand: a lane's accumulators are
// 4 adjacent columns of one row, and one exchange between lanes l and l + 32 makes them 8, which is what
// bias, residual, u and out are read and written in (16 bytes a bf16 row).
#include <type_traits>

#include "activation.h"
#include "gemm_device.h"
#include "grouped_gemm.h"
#include "moe_common.h"
#include "moe_launch.h"

namespace moe {
namespace {

struct LinearArgs {
  const uint8_t* a;          // [rows or a_nrows, K]
  const uint8_t* w;          // [E, Nw, K]
  const uint8_t* bias;       // [E, Nw] fp32 or of the operands' type, or null
  const uint8_t* residual;   // [rows, N] or null
  uint8_t* out;              // [rows, N]
  uint8_t* z;                // [rows, Nw] or null
  const int32_t* offsets;    // [E + 1] or null (E = 1: all rows)
  const int32_t* a_rows;     // [rows] or null: row r is row a_rows[r] / a_div of a
  int a_div, a_nrows;
  int E, rows, K, N, act, bias_f32;
};

constexpr uint32_t kOutside = 0xFFFFFFF0u;   // past every window (windows are below 2^32 - 2^12 bytes)

__device__ __forceinline__ int lin_key(int r) { return (r & 7) ^ ((r >> 3) & 1); }

__device__ __forceinline__ void lin_segment(const LinearArgs& p, int e, int& lo, int& hi) {
  if (p.offsets == nullptr) {
    lo = 0;
    hi = p.rows;
    return;
  }
  lo = p.offsets[e];
  hi = p.offsets[e + 1];
  lo = lo < 0 ? 0 : (lo > p.rows ? p.rows : lo);
  hi = hi < lo ? lo : (hi > p.rows ? p.rows : hi);
}

typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <bool F32>
__device__ __forceinline__ f32x16_t lin_mma(uint4 a, uint4 b, f32x16_t c) {
  if constexpr (F32) {
    const f32x4_t x = __builtin_bit_cast(f32x4_t, a), y = __builtin_bit_cast(f32x4_t, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[i], y[i], c, 0, 0, 0);
    return c;
  } else {
    return mma_bf16(a, b, c);
  }
}

// two groups of 4 columns (2 u and 2 u + 1 of the accumulators) of lanes l and l + 32 -> this lane's 8
// adjacent columns 16 u + 8 (l / 32) + 0 .. 7
__device__ __forceinline__ void pair8(const f32x16_t& c, int u, float (&v)[8]) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(c[8 * u + i]), __float_as_uint(c[8 * u + 4 + i]),
                                                     false, false);
    v[i] = __uint_as_float(s[0]);
    v[4 + i] = __uint_as_float(s[1]);
  }
}

template <bool F32>
__device__ __forceinline__ void lin_load8(const uint8_t* p, size_t i, float (&v)[8]) {   // elements i .. i + 7
  if (F32) {
    const float4* q = reinterpret_cast<const float4*>(p + i * 4);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p + i * 2);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void lin_store8(uint8_t* p, size_t i, const float (&v)[8]) {
  if (F32) {
    float4* q = reinterpret_cast<float4*>(p + i * 4);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p + i * 2) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// v: 8 columns from column col of the weights of expert e, without the bias; adds it and keeps u
template <bool F32>
__device__ __forceinline__ void lin_bias(const LinearArgs& p, int Nw, int e, size_t row, int col, float (&v)[8]) {
  if (p.bias != nullptr) {
    float b[8];
    const size_t at = static_cast<size_t>(e) * Nw + col;
    if (F32 || p.bias_f32) lin_load8<true>(p.bias, at, b);
    else lin_load8<false>(p.bias, at, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (p.z != nullptr) lin_store8<F32>(p.z, row * Nw + col, v);
}

// the epilogue of 8 columns of a row: v (gated: and w, the same columns of the second half)
template <bool F32, bool GATED>
__device__ __forceinline__ void lin_finish(const LinearArgs& p, int e, size_t row, int col, float (&v)[8],
                                           float (&w)[8]) {
  const int Nw = GATED ? 2 * p.N : p.N;
  lin_bias<F32>(p, Nw, e, row, col, v);
  if constexpr (GATED) lin_bias<F32>(p, Nw, e, row, p.N + col, w);
  act8<F32>(p.act, v);
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= w[i];
  }
  if (p.residual != nullptr) {
    float q[8];
    lin_load8<F32>(p.residual, row * p.N + col, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += q[i];
  }
  lin_store8<F32>(p.out, row * p.N + col, v);
}

// The tile of this workgroup: m-tiles of TM rows of every expert, in the order expert -> group of 8
// m-tiles -> column block -> m-tile of the group (the tiles that share weight rows, and those that share
// activation rows, run close together); contiguous ranges of the order go to the XCDs (workgroup i runs
// on XCD i mod 8).  The launch has as many workgroups as any routing can need; false: nothing to do.
struct LinTile {
  int e, m0, mend, nblk;
};
template <int TM, int THREADS>
__device__ __forceinline__ bool lin_tile(const LinearArgs& p, int nN, int32_t* scan, LinTile& t) {
  int total = 0;
  const int tid = threadIdx.x;
  if (p.E == 1) {
    int lo, hi;
    lin_segment(p, 0, lo, hi);
    total = (hi - lo + TM - 1) / TM;
  } else {
    // scan[e]: m-tiles before expert e; 4 experts a thread (E <= 1024), 256 threads
    int32_t* part = scan + MOE_MAX_EXPERTS + 1;
    int n[4], sum = 0;
    if (tid < 256) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * tid + i;
        int lo = 0, hi = 0;
        if (e < p.E) lin_segment(p, e, lo, hi);
        n[i] = (hi - lo + TM - 1) / TM;
        sum += n[i];
      }
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(inc, off, 64);
      if ((tid & 63) >= off) inc += v;
    }
    if ((tid & 63) == 63 && tid < 256) part[tid >> 6] = inc;
    __syncthreads();
    if (tid < 256) {
      int at = inc - sum;
      for (int w = 0; w < (tid >> 6); ++w) at += part[w];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * tid + i <= p.E) scan[4 * tid + i] = at;
        at += n[i];
      }
      if (tid == 255 && p.E == MOE_MAX_EXPERTS) scan[MOE_MAX_EXPERTS] = at;
    }
    __syncthreads();
    total = scan[p.E];
  }
  const long long tiles = static_cast<long long>(total) * nN;
  const long long per = (tiles + kNumXcd - 1) / kNumXcd;
  const long long slot = blockIdx.x / kNumXcd, L = (blockIdx.x % kNumXcd) * per + slot;
  if (slot >= per || L >= tiles) return false;
  int e = 0, before = 0, mt = total;
  if (p.E > 1) {   // the last expert whose tiles start at or before L (an empty expert has none)
    int a = 0, b = p.E - 1;
    while (a < b) {
      const int m = (a + b + 1) >> 1;
      if (static_cast<long long>(scan[m]) * nN <= L) a = m;
      else b = m - 1;
    }
    e = __builtin_amdgcn_readfirstlane(a);
    before = __builtin_amdgcn_readfirstlane(scan[e]);
    mt = __builtin_amdgcn_readfirstlane(scan[e + 1]) - before;
  }
  const int local = static_cast<int>(L - static_cast<long long>(before) * nN);
  constexpr int kGroup = 8;
  const int grp = local / (kGroup * nN), in = local - grp * kGroup * nN;
  const int gm = mt - grp * kGroup < kGroup ? mt - grp * kGroup : kGroup;
  const int mtile = grp * kGroup + in % gm;
  t.nblk = in / gm;
  t.e = e;
  int lo, hi;
  lin_segment(p, e, lo, hi);
  t.m0 = lo + mtile * TM;
  t.mend = t.m0 + TM < hi ? t.m0 + TM : hi;
  return true;
}

// WM x WN waves; a wave's block is (TM / WM) x (TN / WN) as 32 x 32 products
template <bool F32, bool GATED, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void linear_tile_kernel(LinearArgs p) {
  constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  constexpr int MB = TM / WM / 32, NB = TN / WN / 32;
  constexpr int kLdA = TM / 8 / kWaves, kLdW = TN / 8 / kWaves;   // loads of 8 rows a wave and stage
  constexpr int kStage = (TM + TN) * 128;
  constexpr int kEsz = F32 ? 4 : 2;
  static_assert(MB * WM * 32 == TM && NB * WN * 32 == TN && kLdA * kWaves * 8 == TM && kLdW * kWaves * 8 == TN, "tile");
  static_assert(!GATED || NB % 2 == 0, "a wave holds both factors");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage];
  static_assert(2 * kStage >= (MOE_MAX_EXPERTS + 8) * 4, "the tile search shares the LDS");

  constexpr int kCols = GATED ? TN / 2 : TN;   // output columns of a tile
  const int nN = (p.N + kCols - 1) / kCols;
  LinTile t;
  if (!lin_tile<TM, kThreads>(p, nN, reinterpret_cast<int32_t*>(lds), t)) return;
  __syncthreads();   // (the search's words have been read)

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_byte*)lds));
  const uint32_t rb = static_cast<uint32_t>(p.K) * kEsz;   // bytes of a row of a and of W
  const int Nw = GATED ? 2 * p.N : p.N;
  const int c0 = t.nblk * kCols;
  const int ncols = p.N - c0 < kCols ? p.N - c0 : kCols;
  const int mrows = t.mend - t.m0;
  const int nk = (rb + 127) / 128;

  // windows: a's rows of the tile (gathered: all of a), the weight rows of either half
  const uint8_t* a_base = p.a_rows != nullptr ? p.a : p.a + static_cast<size_t>(t.m0) * rb;
  const uint32_t a_size = static_cast<uint32_t>(p.a_rows != nullptr ? p.a_nrows : mrows) * rb;
  const uint8_t* w_base = p.w + (static_cast<size_t>(t.e) * Nw + c0) * rb;
  const uint32_t w_size = static_cast<uint32_t>(ncols) * rb;
  const uint8_t* w2_base = w_base + static_cast<size_t>(p.N) * rb;

  // load j of a part fills the 8-row group wave + kWaves j: lane l slot l % 8 of row l / 8
  const int lrow = lane >> 3;
  uint32_t va[kLdA], vw[kLdW], ca[kLdA], cw[kLdW];   // (ca, cw: the chunk's first byte in the stage)
#pragma unroll
  for (int j = 0; j < kLdA; ++j) {
    const int r = (wave + kWaves * j) * 8 + lrow;
    ca[j] = ((lane & 7) ^ lin_key(r)) * 16;
    if (r >= mrows) {
      va[j] = kOutside;
    } else {
      int row = r;
      if (p.a_rows != nullptr) {
        row = p.a_rows[t.m0 + r] / p.a_div;
        row = row < 0 ? 0 : (row < p.a_nrows ? row : p.a_nrows - 1);
      }
      va[j] = static_cast<uint32_t>(row) * rb + ca[j];
    }
  }
#pragma unroll
  for (int j = 0; j < kLdW; ++j) {
    const int r = (wave + kWaves * j) * 8 + lrow, c = GATED ? r % (TN / 2) : r;
    cw[j] = ((lane & 7) ^ lin_key(r)) * 16;
    vw[j] = c < ncols ? static_cast<uint32_t>(c) * rb + cw[j] : kOutside;
  }
  auto load_stage = [&](int ks, int buf) __attribute__((always_inline)) {
    const uint32_t k0 = static_cast<uint32_t>(ks) * 128;
    const uint32_t left = rb - k0;   // bytes of a row from this stage on
    const u32x4_t ra = buffer_window(a_base + k0, a_size - k0);
    const u32x4_t rw = buffer_window(w_base + k0, w_size - k0);
    const u32x4_t rw2 = buffer_window(w2_base + k0, w_size - k0);
    const uint32_t at = lds0 + buf * kStage + wave * 1024;
#pragma unroll
    for (int j = 0; j < kLdA; ++j)
      dma16_window(ra, left < 128 && ca[j] >= left ? kOutside : va[j], at + j * kWaves * 1024);
#pragma unroll
    for (int j = 0; j < kLdW; ++j)
      dma16_window(GATED && (wave + kWaves * j) * 8 >= TN / 2 ? rw2 : rw, left < 128 && cw[j] >= left ? kOutside : vw[j],
                   at + TM * 128 + j * kWaves * 1024);
  };

  f32x16_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x16_t{};
  // first row of the wave's block m of activations, n of weight rows (gated: the first NB / 2 blocks
  // are of the first half)
  auto a_row = [&](int m) { return (wm * MB + m) * 32; };
  auto w_row = [&](int n) {
    return GATED ? (n / (NB / 2)) * (TN / 2) + (wn * (NB / 2) + n % (NB / 2)) * 32 : (wn * NB + n) * 32;
  };
  uint32_t fb[4];   // the lane's fragment of k-step s
#pragma unroll
  for (int s = 0; s < 4; ++s) fb[s] = (lane & 31) * 128 + ((2 * s + (lane >> 5)) ^ lin_key(lane & 31)) * 16;

  load_stage(0, 0);
  for (int ks = 0; ks < nk; ++ks) {
    const int buf = ks & 1;
    wait_vmcnt<0>();    // stage ks has landed; every wave is past its reads of the other buffer
    block_barrier();
    if (ks + 1 < nk) load_stage(ks + 1, buf ^ 1);
    const uint8_t* la = lds + buf * kStage;
    const uint8_t* lw = la + TM * 128;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint4 fa[MB], fw[NB];
#pragma unroll
      for (int m = 0; m < MB; ++m) fa[m] = *reinterpret_cast<const uint4*>(la + a_row(m) * 128 + fb[s]);
#pragma unroll
      for (int n = 0; n < NB; ++n) fw[n] = *reinterpret_cast<const uint4*>(lw + w_row(n) * 128 + fb[s]);
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[m][n] = lin_mma<F32>(fw[n], fa[m], acc[m][n]);
    }
    wait_lgkmcnt_all();   // (this wave's reads of the stage are done before it meets the next barrier)
  }

  constexpr int kOutB = GATED ? NB / 2 : NB;
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int r = a_row(m) + (lane & 31);
#pragma unroll
    for (int n = 0; n < kOutB; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float v[8], w[8];
        pair8(acc[m][n], u, v);   // (every lane takes part in the exchange)
        if constexpr (GATED) pair8(acc[m][n + kOutB], u, w);
        const int col = (wn * kOutB + n) * 32 + 16 * u + 8 * (lane >> 5);
        if (r < mrows && col < ncols)
          lin_finish<F32, GATED>(p, t.e, static_cast<size_t>(t.m0) + r, c0 + col, v, w);
      }
  }
}

template <bool F32, bool GATED, int TM, int TN, int WM, int WN>
void launch_tiles(const LinearArgs& p, hipStream_t s) {
  constexpr int kCols = GATED ? TN / 2 : TN;
  const long long nN = (p.N + kCols - 1) / kCols;
  const long long mt = (p.rows + TM - 1) / TM + (p.E > 1 ? (p.E - 1 < p.rows ? p.E - 1 : p.rows) : 0);
  const long long grid = (mt * nN + kNumXcd - 1) / kNumXcd * kNumXcd;
  hipLaunchKernelGGL((linear_tile_kernel<F32, GATED, TM, TN, WM, WN>), dim3(static_cast<unsigned>(grid)),
                     dim3(64 * WM * WN), 0, s, p);
}

}  // namespace

// whether the tiles of the smallest shape fit a launch
bool expert_linear_grid_fits(int rows, int N, int E) {
  return (rows / 64ll + 1 + E) * (N / 32ll + 1) < (1ll << 31) - 8;
}

size_t expert_linear_ws_bytes(int rows, int K, int Nw, int E, bool f32) { return 0; }

hipError_t launch_expert_linear(const void* a, bool f32, int a_nrows, const int32_t* src_slot, int k,
                                const int32_t* offsets, int E, int rows, int K, int N, const void* w, const void* bias,
                                bool bias_f32, int act, bool gated, const void* residual, void* out, void* z, void* ws,
                                hipStream_t s) {
  LinearArgs p{};
  p.a = static_cast<const uint8_t*>(a);
  p.w = static_cast<const uint8_t*>(w);
  p.bias = static_cast<const uint8_t*>(bias);
  p.residual = static_cast<const uint8_t*>(residual);
  p.out = static_cast<uint8_t*>(out);
  p.z = static_cast<uint8_t*>(z);
  p.offsets = offsets;
  p.a_rows = src_slot;
  p.a_div = k;
  p.a_nrows = a_nrows;
  p.E = E;
  p.rows = rows;
  p.K = K;
  p.N = N;
  p.act = act;
  p.bias_f32 = bias_f32;
  if (f32 && gated) launch_tiles<true, true, 128, 128, 2, 2>(p, s);
  else if (f32) launch_tiles<true, false, 128, 128, 2, 2>(p, s);
  else if (gated) launch_tiles<false, true, 128, 128, 2, 2>(p, s);
  else launch_tiles<false, false, 128, 128, 2, 2>(p, s);
  return hipGetLastError();
}

}  // namespace moe
