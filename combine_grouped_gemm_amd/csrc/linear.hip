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
// both factors); an expert's rows are split evenly into as few tiles as hold them, and a wave skips the
// products of 32-row blocks without rows.  K advances in stages of 128 bytes a row (64 bf16, 32 fp32),
// loaded straight to LDS through buffer windows: rows past the segment, weight rows past the matrix and columns past K read as
// zeros, so no size needs a kernel of its own.  Chunk c of 16 bytes of row r lies in slot c ^ key(r), so
// that a load (8 rows) and a fragment read (32 rows, two chunks) touch every bank once.  A fragment is one
// chunk a lane for either type: 8 bf16 for one 32x32x16 product, 4 fp32 for four 32x32x2 ones (both
// operands take their k in the same order).  The weights are the first operand: a lane's accumulators are
// 4 adjacent columns of one row, and one exchange between lanes l and l + 32 makes them 8, which is what
// bias, residual, u and out are read and written in (16 bytes a bf16 row).
//
// A ring of S stages is kept ahead.  Every k-step's products run between the LDS reads of the next
// k-step's fragments; before a stage's last k-step, whose fragments are read by then, the workgroup
// meets, so the next stage's first reads and the loads into the slot just left hide under that k-step's
// products too, and the matrix pipes never wait at the barrier.  Shapes: 320 x 256 (8 waves of 160 x 64,
// two stages, one workgroup a CU) reads 0.7 fragments a product and loads least: 256 x 256 took 1.13
// times as long on 4096 x 14336 x 4096, 128 x 128 with two workgroups a CU 1.2 times; 128 x 256 (three
// stages) for fewer rows; 64 x 64 (three stages, three workgroups a CU) where there are few tiles,
// with K in parts when even those leave CUs idle.  Stages of 64 bytes took as long or longer.  fp32: 128 x
// 128 (four waves), and 32 x 64 whose wave pairs share a stage's k-steps: the fp32 products bound it, so
// small tiles, dealt more evenly, win over fewer loads (64 x 64 against it: 999 rows of 6 experts, K 520,
// N 1016 26.7 and 23.0 us; 500 x 1024 x 1024 24.3 and 17.6; 32 experts of 125 rows, gated, K 1024, N 512
// 113 and 101; 512 x 4096 x 4096 145 and 153).
#include <type_traits>
#include <utility>

#include "activation.h"
#include "gemm_device.h"
#include "grouped_gemm.h"
#include "linear_plan.h"
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
  int tile_rows;             // rows of a tile at most: the tile's, or fewer (linear_tile_kernel)
  float* part;               // split K: [split, rows, Nw] sums instead of the epilogue, or null
  int split;
};

static_assert(kLinXcds == kNumXcd, "the launch counts the XCDs");
constexpr uint32_t kOutside = 0xFFFFFFF0u;   // past every window (windows are below 2^32 - 2^12 bytes)

// slot of chunk c of row r: c ^ key
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

// 8 biases from column col of expert e's weights (0 without biases)
template <bool F32>
__device__ __forceinline__ void lin_bias(const LinearArgs& p, int Nw, int e, int col, float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.0f;
  if (p.bias == nullptr) return;
  const size_t at = static_cast<size_t>(e) * Nw + col;
  if (F32 || p.bias_f32) lin_load8<true>(p.bias, at, b);
  else lin_load8<false>(p.bias, at, b);
}

// 8 columns of a row as they lie
template <bool F32>
struct Raw {
  uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw<F32> lin_raw(const uint8_t* p, size_t i) {   // elements i .. i + 7
  Raw<F32> r;
  const uint4* q = reinterpret_cast<const uint4*>(p + i * (F32 ? 4 : 2));
  r.w[0] = q[0];
  if constexpr (F32) r.w[1] = q[1];
  return r;
}
template <bool F32>
__device__ __forceinline__ void lin_values(const Raw<F32>& r, float (&v)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (F32) {
      v[2 * j] = __uint_as_float(w[2 * j]);
      v[2 * j + 1] = __uint_as_float(w[2 * j + 1]);
    } else {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// the epilogue of 8 columns of a row: sums v (gated: and w, the same columns of the second half), their
// biases bv (and bw), the residual's values res (read when there is one)
template <bool F32, bool GATED>
__device__ __forceinline__ void lin_finish(const LinearArgs& p, size_t row, int col, float (&v)[8], float (&w)[8],
                                           const float (&bv)[8], const float (&bw)[8], const Raw<F32>& res) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] += bv[i];
    if constexpr (GATED) w[i] += bw[i];
  }
  if (p.z != nullptr) {
    const size_t at = row * (GATED ? 2 * p.N : p.N) + col;
    lin_store8<F32>(p.z, at, v);
    if constexpr (GATED) lin_store8<F32>(p.z, at + p.N, w);
  }
  act8<F32>(p.act, v);
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= w[i];
  }
  if (p.residual != nullptr) {
    float q[8];
    lin_values<F32>(res, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += q[i];
  }
  lin_store8<F32>(p.out, row * p.N + col, v);
}
// the same, its biases and residual read here
template <bool F32, bool GATED>
__device__ __forceinline__ void lin_finish_one(const LinearArgs& p, int e, size_t row, int col, float (&v)[8],
                                               float (&w)[8]) {
  const int Nw = GATED ? 2 * p.N : p.N;
  float bv[8], bw[8];
  lin_bias<F32>(p, Nw, e, col, bv);
  if constexpr (GATED) lin_bias<F32>(p, Nw, e, p.N + col, bw);
  Raw<F32> res{};
  if (p.residual != nullptr) res = lin_raw<F32>(p.residual, row * p.N + col);
  lin_finish<F32, GATED>(p, row, col, v, w, bv, bw, res);
}

// The tile of this workgroup: m-tiles of at most tile_rows rows of every expert, in the order expert -> group of 8
// m-tiles -> column block -> m-tile of the group (the tiles that share weight rows, and those that share
// activation rows, run close together); contiguous ranges of the order go to the XCDs (workgroup i runs
// on XCD i mod 8).  The launch has as many workgroups as any routing can need; false: nothing to do.
// Every wave searches for itself, an expert a lane (E > 64: first the run of up to 16 experts, a run a
// lane), so that the search costs one or two memory latencies and no barrier.
struct LinTile {
  int e, m0, mend, nblk, part;
};

// sum over lanes up to this one: within rows of 16 lanes, then over rows (lanes without a source add 0)
__device__ __forceinline__ int wave_prefix(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // lane 15 of a row to the next: rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // lane 31 to rows 2 and 3
  return v;
}

__device__ __forceinline__ bool lin_tile(const LinearArgs& p, int nN, int unit, LinTile& t) {
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](int lo, int hi) { return (hi - lo + p.tile_rows - 1) / p.tile_rows; };
  int run = 1, run_sum = 0, run_end = 0, total = 0;
  if (p.E > 64) {
    run = (p.E + 63) / 64;
    for (int i = 0; i < run; ++i) {
      int lo = 0, hi = 0;
      if (lane * run + i < p.E) lin_segment(p, lane * run + i, lo, hi);
      run_sum += tiles_of(lo, hi);
    }
    run_end = wave_prefix(run_sum);
    total = __builtin_amdgcn_readlane(run_end, 63);
  }
  int e0 = 0, before = 0, lo = 0, hi = 0, end = 0;
  auto expert_lanes = [&](int n) __attribute__((always_inline)) {   // experts e0 .. e0 + n - 1
    lo = hi = 0;
    if (lane < n) lin_segment(p, e0 + lane, lo, hi);
    end = before + wave_prefix(tiles_of(lo, hi));
  };
  if (p.E <= 64) {
    expert_lanes(p.E);
    total = __builtin_amdgcn_readlane(end, 63);
  }
  const long long tiles = static_cast<long long>(total) * nN, all = tiles * p.split;
  const long long per = (all + kNumXcd - 1) / kNumXcd;
  const long long slot = blockIdx.x / kNumXcd;
  long long L = (blockIdx.x % kNumXcd) * per + slot;
  if (slot >= per || L >= all) return false;
  t.part = 0;
  if (p.split > 1) {   // (the parts of K outermost: an XCD holds few of them)
    t.part = static_cast<int>(L / tiles);
    L -= t.part * tiles;
  }
  if (p.E > 64) {
    const int l = __builtin_ctzll(__ballot(static_cast<long long>(run_end) * nN > L));
    e0 = l * run;
    before = __builtin_amdgcn_readlane(run_end - run_sum, l);
    expert_lanes(p.E - e0 < run ? p.E - e0 : run);
  }
  // the expert: the first whose tiles end behind L (of an empty expert nothing does)
  const int l = __builtin_ctzll(__ballot(static_cast<long long>(end) * nN > L));
  lo = __builtin_amdgcn_readlane(lo, l);
  hi = __builtin_amdgcn_readlane(hi, l);
  t.e = e0 + l;
  const int mt = tiles_of(lo, hi);
  const int local = static_cast<int>(L - static_cast<long long>(__builtin_amdgcn_readlane(end, l) - mt) * nN);
  constexpr int kGroup = 8;
  const int grp = local / (kGroup * nN), in = local - grp * kGroup * nN;
  const int gm = mt - grp * kGroup < kGroup ? mt - grp * kGroup : kGroup;
  const int mtile = grp * kGroup + in % gm;
  t.nblk = in / gm;
  // (a multiple of the rows that the row waves share, 64 of two: 288 rows take a wave's five blocks as 320
  // do; at most tile_rows, which unit divides)
  const int rpt = ((hi - lo + mt - 1) / mt + unit - 1) / unit * unit;
  t.m0 = lo + mtile * rpt;
  t.mend = t.m0 + rpt < hi ? t.m0 + rpt : hi;
  return t.m0 < t.mend;
}

// WM x WN waves; a wave's block is (TM / WM) x (TN / WN) as 32 x 32 products.  WK times as many waves: they
// share a stage's four k-steps, and the first WM x WN add the others' sums in order.
template <bool F32, bool GATED, int TM, int TN, int WM, int WN, int S, int WK>
__global__ __launch_bounds__(64 * WM * WN * WK) void linear_tile_kernel(LinearArgs p) {
  constexpr int kWaves = WM * WN * WK, kSteps = 4 / WK;   // k-steps of a wave and stage
  constexpr int MB = TM / WM / 32, NB = TN / WN / 32;
  constexpr int kLdA = TM / 8 / kWaves, kLdW = TN / 8 / kWaves;   // loads a wave and stage
  constexpr int kStage = (TM + TN) * kLinRow;
  constexpr int kEsz = F32 ? 4 : 2;
  static_assert(MB * WM * 32 == TM && NB * WN * 32 == TN && kLdA * kWaves * 8 == TM && kLdW * kWaves * 8 == TN, "tile");
  static_assert(!GATED || NB % 2 == 0, "a wave holds both factors");
  static_assert(WK == 1 || WK == 2, "k-steps are taken in pairs");
  __shared__ __attribute__((aligned(16))) uint8_t lds[S * kStage];

  constexpr int kCols = GATED ? TN / 2 : TN;   // output columns of a tile
  const int nN = (p.N + kCols - 1) / kCols;
  LinTile t;
  if (!lin_tile(p, nN, 32 * WM, t)) return;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN % WM, wn = wave % WN, wk = wave / (WM * WN);
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_byte*)lds));
  const uint32_t rb = static_cast<uint32_t>(p.K) * kEsz;   // bytes of a row of a and of W
  const int Nw = GATED ? 2 * p.N : p.N;
  const int c0 = t.nblk * kCols;
  const int ncols = p.N - c0 < kCols ? p.N - c0 : kCols;
  const int mrows = t.mend - t.m0;
  const int nkt = (rb + kLinRow - 1) / kLinRow;   // stages; this part's: [ks0, ks0 + nk)
  const int ks0 = nkt * t.part / p.split, nk = nkt * (t.part + 1) / p.split - ks0;

  // windows: a's rows of the tile (gathered: all of a), the weight rows of either half
  const uint8_t* a_base = p.a_rows != nullptr ? p.a : p.a + static_cast<size_t>(t.m0) * rb;
  const uint32_t a_size = static_cast<uint32_t>(p.a_rows != nullptr ? p.a_nrows : mrows) * rb;
  const uint8_t* w_base = p.w + (static_cast<size_t>(t.e) * Nw + c0) * rb;
  const uint32_t w_size = static_cast<uint32_t>(ncols) * rb;
  const uint8_t* w2_base = w_base + static_cast<size_t>(p.N) * rb;

  // load j of an operand fills the 8-row group wave + kWaves j: lane l slot l % 8 of row l / 8, so chunk
  // ch / 16 of it (kWaves is even: the group's parity is the wave's)
  static_assert(kWaves % 2 == 0, "one chunk a lane");
  const int lrow = lane >> 3;
  const uint32_t ch = ((lane & 7) ^ lin_key((wave & 1) * 8 + lrow)) * 16;
  uint32_t va[kLdA], vw[kLdW];
#pragma unroll
  for (int j = 0; j < kLdA; ++j) {
    const int r = (wave + kWaves * j) * 8 + lrow;
    va[j] = kOutside;
    if (r < mrows) {
      int row = r;
      if (p.a_rows != nullptr) {
        row = p.a_rows[t.m0 + r] / p.a_div;
        row = row < 0 ? 0 : (row < p.a_nrows ? row : p.a_nrows - 1);
      }
      va[j] = static_cast<uint32_t>(row) * rb + ch;
    }
  }
#pragma unroll
  for (int j = 0; j < kLdW; ++j) {
    const int r = (wave + kWaves * j) * 8 + lrow, c = GATED ? r % (TN / 2) : r;
    vw[j] = c < ncols ? static_cast<uint32_t>(c) * rb + ch : kOutside;
  }
  // loads J of a stage into its slot: the rows of a first, then the weight rows
  constexpr int kLoads = kLdA + kLdW;   // a wave and stage
  struct Stage {
    u32x4_t a, w, w2;
    uint32_t left, at;   // bytes of a row from this stage on; the slot
  };
  auto stage_of = [&](int ks, int slot) __attribute__((always_inline)) {
    const uint32_t k0 = static_cast<uint32_t>(ks) * kLinRow;
    Stage g;
    g.a = buffer_window(a_base + k0, a_size - k0);
    g.w = buffer_window(w_base + k0, w_size - k0);
    g.w2 = GATED ? buffer_window(w2_base + k0, w_size - k0) : g.w;
    g.left = rb - k0;
    g.at = lds0 + slot * kStage + wave * 1024;
    return g;
  };
  auto load_one = [&](const Stage& g, int j) __attribute__((always_inline)) {   // (j is a constant after unrolling)
    if (j < kLdA) {
      dma16_window(g.a, ch >= g.left ? kOutside : va[j], g.at + j * kWaves * 1024);
    } else {
      const int i = j - kLdA;
      dma16_window(GATED && (wave + kWaves * i) * 8 >= TN / 2 ? g.w2 : g.w,
                   ch >= g.left ? kOutside : vw[i], g.at + TM * kLinRow + i * kWaves * 1024);
    }
  };

  f32x16_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x16_t{};
  // first row of the wave's block m of activations, n of weight rows (gated: the first NB / 2 blocks
  // are of the first half)
  auto a_row = [&](int m) { return (m * WM + wm) * 32; };   // (dealt in turn: short tiles leave no wave idle)
  auto w_row = [&](int n) {
    return GATED ? (n / (NB / 2)) * (TN / 2) + (wn * (NB / 2) + n % (NB / 2)) * 32 : (wn * NB + n) * 32;
  };
  uint32_t fb[kSteps];   // the lane's fragment of the wave's k-step s
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    fb[s] = (lane & 31) * kLinRow + ((2 * (kSteps * wk + s) + (lane >> 5)) ^ lin_key(lane & 31)) * 16;

  static_assert(S * kLoads < 64, "the load counter");
  for (int i = 0; i < S; ++i) {
    if (i >= nk) break;
    const Stage g = stage_of(ks0 + i, i);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load_one(g, j);
  }
  if (nk >= S) wait_vmcnt<(S - 1) * kLoads>();
  else wait_vmcnt<0>();
  block_barrier();   // stage 0 has landed
  auto k_loop = [&](auto act_c) __attribute__((always_inline)) {
    constexpr int ACT = decltype(act_c)::value;   // row blocks of this wave that hold rows
    constexpr int kSlots = ACT > 0 ? ACT * NB : 1, kReads = ACT > 0 ? ACT + NB : 0;
    uint4 f0[ACT + NB], f1[ACT + NB];   // fragments of this k-step and of the next: rows of a, weight rows
    // fragment r in the order of its first use: a's block 0, the weight blocks, a's other blocks
    auto read = [&](uint4(&f)[ACT + NB], int r, int slot, int s) __attribute__((always_inline)) {
      const uint8_t* st = lds + slot * kStage;
      const int m = r == 0 ? 0 : r - NB, n = r - 1;
      if (r >= 1 && r <= NB)
        f[ACT + n] = *reinterpret_cast<const uint4*>(st + TM * kLinRow + w_row(n) * kLinRow + fb[s]);
      else
        f[m] = *reinterpret_cast<const uint4*>(st + a_row(m) * kLinRow + fb[s]);
    };
    // the products of a k-step; ahead of each the next reads of the k-step after it (slot, s), so that the
    // last have landed when that begins, and behind each the next loads of a later stage
    constexpr int kReadEach = (kReads + kSlots - 1) / kSlots, kLoadEach = (kLoads + kSlots - 1) / kSlots;
    auto step = [&]<bool READ, bool LOAD>(const uint4(&f)[ACT + NB], uint4(&n)[ACT + NB], int slot, int s,
                                          const Stage& g) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if constexpr (READ) {
#pragma unroll
          for (int r = kReadEach * i; r < kReadEach * (i + 1); ++r)
            if (r < kReads) read(n, r, slot, s);
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (ACT > 0) acc[i / NB][i % NB] = lin_mma<F32>(f[ACT + i % NB], f[i / NB], acc[i / NB][i % NB]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (LOAD) {
#pragma unroll
          for (int j = kLoadEach * i; j < kLoadEach * (i + 1); ++j)
            if (j < kLoads) load_one(g, j);
        }
      }
    };
    int slot = 0;
    Stage none{};
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(f0, r, 0, 0);
    auto first = [&]() __attribute__((always_inline)) {   // all k-steps but the last of the stage in slot
      step.template operator()<true, false>(f0, f1, slot, 1, none);
      if constexpr (WK == 1) {
        step.template operator()<true, false>(f1, f0, slot, 2, none);
        step.template operator()<true, false>(f0, f1, slot, 3, none);
      }
    };
    // this wave's reads of the stage are done, and its loads of the next have landed (all but those of the
    // LEFT stages behind it); behind the barrier every wave's are and have
    auto meet = [&]<int LEFT>() __attribute__((always_inline)) {
      wait_lgkmcnt_all();
      wait_vmcnt<LEFT * kLoads>();
      block_barrier();
    };
    int ks = 0;
    for (; ks < nk - S; ++ks) {
      const int next = slot == S - 1 ? 0 : slot + 1;
      first();
      meet.template operator()<S - 2>();
      const Stage g = stage_of(ks0 + ks + S, slot);
      step.template operator()<true, true>(f1, f0, next, 0, g);
      slot = next;
    }
    for (; ks < nk - 1; ++ks) {   // (no further stage to load)
      const int next = slot == S - 1 ? 0 : slot + 1;
      first();
      meet.template operator()<0>();
      step.template operator()<true, false>(f1, f0, next, 0, none);
      slot = next;
    }
    first();
    step.template operator()<false, false>(f1, f0, 0, 0, none);
  };
  const int nblk = (mrows + 31) / 32;
  const int act = nblk > wm ? (nblk - wm + WM - 1) / WM : 0;
  if (act >= MB) {
    k_loop(std::integral_constant<int, MB>{});
  } else {
    [&]<int... A>(std::integer_sequence<int, A...>) {
      ((act == A ? k_loop(std::integral_constant<int, A>{}) : void()), ...);
    }(std::make_integer_sequence<int, MB>{});
  }

  if constexpr (WK == 2) {
    static_assert(MB * NB * WM * WN * 4096 <= S * kStage, "the sums' LDS");
    float* const red = reinterpret_cast<float*>(lds) + (wm * WN + wn) * MB * NB * 1024 + lane;
    __syncthreads();   // (every wave's reads of the last stage are done)
#pragma unroll
    for (int i = 0; i < MB * NB * 16; ++i)
      if (wk != 0) red[i * 64] = acc[i / 16 / NB][i / 16 % NB][i % 16];
    __syncthreads();
    if (wk != 0) return;
#pragma unroll
    for (int i = 0; i < MB * NB * 16; ++i) acc[i / 16 / NB][i / 16 % NB][i % 16] += red[i * 64];
  }

  // epilogue: 8 columns (n, u) of row block m a lane; their biases once, a row block's residual together
  constexpr int kOutB = GATED ? NB / 2 : NB;
  auto row_of = [&](int m) __attribute__((always_inline)) { return a_row(m) + (lane & 31); };
  auto col_of = [&](int n, int u) __attribute__((always_inline)) {
    return (wn * kOutB + n) * 32 + 16 * u + 8 * (lane >> 5);
  };
  if (p.part != nullptr) {   // one part of K: the sums join in another kernel
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int n = 0; n < kOutB; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float v[8], w[8];
          pair8(acc[m][n], u, v);   // (every lane takes part in the exchange)
          if constexpr (GATED) pair8(acc[m][n + kOutB], u, w);
          if (row_of(m) >= mrows || col_of(n, u) >= ncols) continue;
          float* q = p.part + (static_cast<size_t>(t.part) * p.rows + t.m0 + row_of(m)) * Nw + c0 + col_of(n, u);
          lin_store8<true>(reinterpret_cast<uint8_t*>(q), 0, v);
          if constexpr (GATED) lin_store8<true>(reinterpret_cast<uint8_t*>(q + p.N), 0, w);
        }
    return;
  }
  float bias[NB][2][8];   // (gated: [n + kOutB] the second half's)
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int col = col_of(n % kOutB, u);
      lin_bias<F32>(p, Nw, t.e, (n < kOutB ? 0 : p.N) + c0 + (col < ncols ? col : 0), bias[n][u]);
    }
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    Raw<F32> res[kOutB][2];
    if (p.residual != nullptr) {
#pragma unroll
      for (int n = 0; n < kOutB; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (row_of(m) < mrows && col_of(n, u) < ncols)
            res[n][u] = lin_raw<F32>(p.residual, (static_cast<size_t>(t.m0) + row_of(m)) * p.N + c0 + col_of(n, u));
    }
#pragma unroll
    for (int n = 0; n < kOutB; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float v[8], w[8];
        pair8(acc[m][n], u, v);
        if constexpr (GATED) pair8(acc[m][n + kOutB], u, w);
        if (row_of(m) < mrows && col_of(n, u) < ncols)
          lin_finish<F32, GATED>(p, static_cast<size_t>(t.m0) + row_of(m), c0 + col_of(n, u), v, w, bias[n][u],
                                 bias[GATED ? n + kOutB : n][u], res[n][u]);
      }
  }
}

// the parts of K joined in order: a lane 8 columns of a row
template <bool F32, bool GATED>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs p) {
  const int groups = p.N / 8;
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long row = i / groups;
  if (row >= p.rows) return;
  const int col = static_cast<int>(i - row * groups) * 8;
  int e = 0;
  if (p.offsets != nullptr) {   // the row's expert: the last that starts at or before it
    int a = 0, b = p.E - 1;
    while (a < b) {
      const int m = (a + b + 1) >> 1;
      if (p.offsets[m] <= row) a = m;
      else b = m - 1;
    }
    e = a;
    if (row < p.offsets[e] || row >= p.offsets[e + 1]) return;
  }
  const int Nw = GATED ? 2 * p.N : p.N;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int s = 0; s < p.split; ++s) {
    const float* q = p.part + (static_cast<size_t>(s) * p.rows + row) * Nw + col;
    float t[8];
    lin_load8<true>(reinterpret_cast<const uint8_t*>(q), 0, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += t[j];
    if constexpr (GATED) {
      lin_load8<true>(reinterpret_cast<const uint8_t*>(q + p.N), 0, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] += t[j];
    }
  }
  lin_finish_one<F32, GATED>(p, e, row, col, v, w);
}

// ------------------------------------------------------------------------------------
// Few rows an expert (serving: single tokens and small batches): bound by the weights' bytes.  A
// workgroup takes 32 weight rows (gated: 16 of either half) or half as many, and the rows of one expert, up
// to 32 at a time; its waves split K in contiguous parts.  Each wave streams its part through a ring of stages of its
// own in LDS (128 bytes of the weight rows and of the rows of a), without meeting the others until the
// end, when their sums are added in order.  The mean load chooses this kernel, so an expert may have many
// rows all the same, each 32 of them another pass over its weights: 64 experts of K 2048, N 1408, 512 rows took
// 63 us with 8 each, 77 with half of them on one and 64 with all on one (17 as one expert's tiles).
// ------------------------------------------------------------------------------------

template <bool F32>
__device__ __forceinline__ f32x4_t few_mma(uint4 a, uint4 b, f32x4_t c) {
  if constexpr (F32) {
    const f32x4_t x = __builtin_bit_cast(f32x4_t, a), y = __builtin_bit_cast(f32x4_t, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
}

// Weight rows and waves of a workgroup: 32 and 4 (two workgroups a CU), or, where those would leave CUs
// idle, 16 and 8 (one).  RING: stages of a wave's ring with 16 MB rows of a.
template <int WB>
struct Few {
  static constexpr int kRows = 16 * WB, kWaves = WB == 2 ? 4 : 8, kThreads = 64 * kWaves;
  static constexpr int kLds = WB == 2 ? 72 * 1024 : 144 * 1024;
  template <int MB>
  static constexpr int kStage = (kRows + 16 * MB) * kLinRow;
  template <int MB>
  static constexpr int kRing = WB == 2 ? (MB == 1 ? 3 : 2) : (MB == 1 ? 4 : 3);
  static_assert(kRing<1> * kStage<1> * kWaves <= kLds && kRing<2> * kStage<2> * kWaves <= kLds, "the rings' LDS");
};

// rows [m0, m0 + 16 MB) of expert e against the workgroup's weight rows
template <bool F32, bool GATED, int MB, int WB>
__device__ __forceinline__ void few_rows(const LinearArgs& p, int e, int m0, int mend, int c0, uint8_t* lds) {
  using F = Few<WB>;
  constexpr int kCols = GATED ? 8 * WB : 16 * WB, S = F::template kRing<MB>, kLdW = 2 * WB, kLd = kLdW + 2 * MB;
  constexpr int kStage = F::template kStage<MB>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const mine = lds + wave * (F::kLds / F::kWaves);
  const uint32_t at0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_byte*)mine));
  const uint32_t rb = static_cast<uint32_t>(p.K) * (F32 ? 4 : 2);
  const int Nw = GATED ? 2 * p.N : p.N;
  const int ncols = p.N - c0 < kCols ? p.N - c0 : kCols;
  const int mrows = mend - m0 < 16 * MB ? mend - m0 : 16 * MB;
  const uint8_t* w_base = p.w + (static_cast<size_t>(e) * Nw + c0) * rb;
  const uint8_t* w2_base = w_base + static_cast<size_t>(p.N) * rb;
  const uint32_t w_size = static_cast<uint32_t>(ncols) * rb;
  const uint8_t* a_base = p.a_rows != nullptr ? p.a : p.a + static_cast<size_t>(m0) * rb;
  const uint32_t a_size = static_cast<uint32_t>(p.a_rows != nullptr ? p.a_nrows : mrows) * rb;
  // a load fills 8 rows: lane l slot l % 8 of row l / 8
  uint32_t vw[kLdW], va[2 * MB], ch[2];   // (ch: the chunk's first byte, rows of even and odd groups)
#pragma unroll
  for (int j = 0; j < 2; ++j) ch[j] = ((lane & 7) ^ lin_key(j * 8 + (lane >> 3))) * 16;
#pragma unroll
  for (int j = 0; j < 2 * MB; ++j) {
    const int r = j * 8 + (lane >> 3);
    va[j] = kOutside;
    if (r < mrows) {
      int row = r;
      if (p.a_rows != nullptr) {
        row = p.a_rows[m0 + r] / p.a_div;
        row = row < 0 ? 0 : (row < p.a_nrows ? row : p.a_nrows - 1);
      }
      va[j] = static_cast<uint32_t>(row) * rb + ch[j & 1];
    }
  }
#pragma unroll
  for (int j = 0; j < kLdW; ++j) {
    const int r = j * 8 + (lane >> 3), c = GATED ? r % kCols : r;
    vw[j] = c < ncols ? static_cast<uint32_t>(c) * rb + ch[j & 1] : kOutside;
  }
  auto load = [&](int ks, int slot) __attribute__((always_inline)) {
    const uint32_t k0 = static_cast<uint32_t>(ks) * 128, left = rb - k0;
    const u32x4_t rw = buffer_window(w_base + k0, w_size - k0);
    const u32x4_t rw2 = GATED ? buffer_window(w2_base + k0, w_size - k0) : rw;
    const u32x4_t ra = buffer_window(a_base + k0, a_size - k0);
    const uint32_t at = at0 + slot * kStage;
    const bool in[2] = {left >= 128 || ch[0] < left, left >= 128 || ch[1] < left};   // (past K: zeros)
#pragma unroll
    for (int j = 0; j < kLdW; ++j) dma16_window(GATED && j >= WB ? rw2 : rw, in[j & 1] ? vw[j] : kOutside, at + j * 1024);
#pragma unroll
    for (int j = 0; j < 2 * MB; ++j) dma16_window(ra, in[j & 1] ? va[j] : kOutside, at + (kLdW + j) * 1024);
  };
  const int nkt = (rb + 127) / 128;
  const int s0 = nkt * wave / F::kWaves, nk = nkt * (wave + 1) / F::kWaves - s0;
  f32x4_t acc[MB][WB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int c = 0; c < WB; ++c) acc[m][c] = f32x4_t{};
  uint32_t fb[2];   // fragment of k-step s: row l % 16, chunk 4 s + l / 16
#pragma unroll
  for (int s = 0; s < 2; ++s) fb[s] = (lane & 15) * 128 + ((4 * s + (lane >> 4)) ^ lin_key(lane & 15)) * 16;
  for (int i = 0; i < S - 1; ++i)
    if (i < nk) load(s0 + i, i);
  int slot = 0;
  for (int ks = 0; ks < nk; ++ks) {
    if (ks + S - 1 <= nk) wait_vmcnt<(S - 2) * kLd>();
    else wait_vmcnt<0>();
    __asm__ volatile("" ::: "memory");
    // (the slot of stage ks - 1, whose fragments have been read)
    if (ks + S - 1 < nk) load(s0 + ks + S - 1, slot == 0 ? S - 1 : slot - 1);
    const uint8_t* st = mine + slot * kStage;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint4 fw[WB], fa[MB];
#pragma unroll
      for (int c = 0; c < WB; ++c) fw[c] = *reinterpret_cast<const uint4*>(st + c * 16 * 128 + fb[s]);
#pragma unroll
      for (int m = 0; m < MB; ++m) fa[m] = *reinterpret_cast<const uint4*>(st + (F::kRows + m * 16) * 128 + fb[s]);
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int c = 0; c < WB; ++c) acc[m][c] = few_mma<F32>(fw[c], fa[m], acc[m][c]);
    }
    wait_lgkmcnt_all();
    __asm__ volatile("" ::: "memory");
    slot = slot == S - 1 ? 0 : slot + 1;
  }
  // lane l holds weight rows 4 (l / 16) .. + 3 of block c for row l % 16: red[wave][m][row][weight row]
  float* const red = reinterpret_cast<float*>(lds);
  __syncthreads();
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int c = 0; c < WB; ++c)
      *reinterpret_cast<f32x4_t*>(red + ((wave * MB + m) * 16 + (lane & 15)) * F::kRows + c * 16 + 4 * (lane >> 4)) =
          acc[m][c];
  __syncthreads();
  constexpr int kGroups = kCols / 8;   // 8 columns of a row a lane
  for (int i = threadIdx.x; i < MB * 16 * kGroups; i += F::kThreads) {
    const int r = i / kGroups, col = (i % kGroups) * 8;
    if (r >= mrows || col >= ncols) continue;
    float v[8], w[8];
#pragma unroll
    for (int c = 0; c < (GATED ? 2 : 1); ++c) {
      float t[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < F::kWaves; ++q) {
        const float4* x = reinterpret_cast<const float4*>(red + (q * MB * 16 + r) * F::kRows + c * kCols + col);
        const float4 a = x[0], b = x[1];
        t[0] += a.x; t[1] += a.y; t[2] += a.z; t[3] += a.w;
        t[4] += b.x; t[5] += b.y; t[6] += b.z; t[7] += b.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) (c == 0 ? v : w)[j] = t[j];
    }
    lin_finish_one<F32, GATED>(p, e, static_cast<size_t>(m0) + r, c0 + col, v, w);
  }
  __syncthreads();   // (the sums have been read before the next rows' stages land)
}

// workgroup x: 16 WB weight rows; y: an expert (slots < E: the y-th expert that has rows)
template <bool F32, bool GATED, int WB>
__global__ __launch_bounds__(Few<WB>::kThreads) void linear_few_kernel(LinearArgs p, int slots) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[Few<WB>::kLds];
  const int lane = threadIdx.x & 63;
  int e = blockIdx.y;
  if (slots < p.E) {
    int seen = 0, found = -1;
    for (int b = 0; b < p.E && found < 0; b += 64) {   // (every wave the same search)
      int lo = 0, hi = 0;
      if (b + lane < p.E) lin_segment(p, b + lane, lo, hi);
      const uint64_t some = __ballot(hi > lo);
      const int n = __popcll(some), want = static_cast<int>(blockIdx.y) - seen;
      if (want < n) {
        const uint64_t below = some & ((1ull << lane) - 1);
        const uint64_t mine = __ballot(((some >> lane) & 1) != 0 && __popcll(below) == want);
        found = b + __builtin_ctzll(mine);
      }
      seen += n;
    }
    if (found < 0) return;
    e = __builtin_amdgcn_readfirstlane(found);
  }
  int lo, hi;
  lin_segment(p, e, lo, hi);
  const int c0 = blockIdx.x * (GATED ? 8 * WB : 16 * WB);
  for (int m0 = lo; m0 < hi; m0 += 32) {
    if (hi - m0 <= 16) few_rows<F32, GATED, 1, WB>(p, e, m0, hi, c0, lds);
    else few_rows<F32, GATED, 2, WB>(p, e, m0, hi, c0, lds);
  }
}

template <bool F32, bool GATED, int WB>
void launch_few(const LinearArgs& p, int slots, hipStream_t s) {
  constexpr int kCols = GATED ? 8 * WB : 16 * WB;
  hipLaunchKernelGGL((linear_few_kernel<F32, GATED, WB>), dim3((p.N + kCols - 1) / kCols, slots),
                     dim3(Few<WB>::kThreads), 0, s, p, slots);
}

template <bool F32, bool GATED>
void launch_few(const LinearArgs& p, hipStream_t s) {
  const int slots = p.E < p.rows ? p.E : p.rows;
  const long long groups = (static_cast<long long>(GATED ? 2 * p.N : p.N) + 31) / 32 * slots;
  // half as many weight rows where 256 CUs then get a workgroup each (one row, N 4096, K 14336: 28 -> 22 us,
  // fp32 K 4096 17 -> 13; with twice the rows, N 8192, K 4096, they took 14 against 13)
  if (groups <= 128) launch_few<F32, GATED, 1>(p, slots, s);
  else launch_few<F32, GATED, 2>(p, slots, s);
}

template <bool F32, bool GATED, int KIND, int TM, int TN, int WM, int WN, int S, int WK = 1>
void launch_tiles(LinearArgs p, hipStream_t s, const LinPlan& plan, void* ws) {
  constexpr LinShape kShape = lin_shape(KIND, F32, GATED);
  static_assert(kShape.rows == TM && kShape.cols == (GATED ? TN / 2 : TN) && kShape.threads == 64 * WM * WN * WK,
                "the shape that the plan counts");
  const int split = plan.split;
  p.tile_rows = plan.tile_rows > 0 ? plan.tile_rows : TM;
  const long long grid = lin_tile_groups(p.rows, p.E, p.N, p.tile_rows, kShape.cols, split);
  p.split = split;
  p.part = split > 1 ? static_cast<float*>(ws) : nullptr;
  hipLaunchKernelGGL((linear_tile_kernel<F32, GATED, TM, TN, WM, WN, S, WK>), dim3(static_cast<unsigned>(grid)),
                     dim3(64 * WM * WN * WK), 0, s, p);
  if (split > 1) {
    const long long lanes = static_cast<long long>(p.rows) * (p.N / 8);
    hipLaunchKernelGGL((linear_join_kernel<F32, GATED>), dim3(static_cast<unsigned>((lanes + 255) / 256)), dim3(256), 0, s,
                       p);
  }
}

}  // namespace

// whether a call's launches fit
bool expert_linear_grid_fits(int rows, int K, int N, int E, bool f32, bool gated) {
  return lin_fits(rows, K, N, E, f32, gated);
}

size_t expert_linear_ws_bytes(int rows, int K, int Nw, int E, bool f32) {
  const int split = lin_plan(rows, K, Nw, E, f32).split;
  return split > 1 ? static_cast<size_t>(split) * rows * Nw * sizeof(float) : 0;
}

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
  const LinPlan plan = lin_plan(rows, K, gated ? 2 * N : N, E, f32);
  auto go = [&](auto f, auto g) {
    constexpr bool F = decltype(f)::value, G = decltype(g)::value;
    if (plan.kind == LIN_FEW) launch_few<F, G>(p, s);
    else if constexpr (F) {
      if (plan.kind == LIN_32) launch_tiles<F, G, LIN_32, 32, G ? 128 : 64, 1, 2, 3, 2>(p, s, plan, ws);
      else launch_tiles<F, G, LIN_128, 128, 128, 2, 2, 2>(p, s, plan, ws);
    } else {
      if (plan.kind == LIN_64) launch_tiles<F, G, LIN_64, 64, G ? 128 : 64, 2, 2, 3>(p, s, plan, ws);
      else if (plan.kind == LIN_128) launch_tiles<F, G, LIN_128, 128, 256, 2, 4, 3>(p, s, plan, ws);
      else launch_tiles<F, G, LIN_320, 320, 256, 2, 4, 2>(p, s, plan, ws);
    }
  };
  using T = std::true_type;
  using U = std::false_type;
  if (f32 && gated) go(T{}, T{});
  else if (f32) go(T{}, U{});
  else if (gated) go(U{}, T{});
  else go(U{}, U{});
  return hipGetLastError();
}

}  // namespace moe
