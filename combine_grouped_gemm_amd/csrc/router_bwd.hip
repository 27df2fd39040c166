// The router's gradients from a dense logit gradient dz [N, E] ("EP / DeepEP explanation" page,
// section 2: z = x W_r^T; the balance loss reaches every expert's logit, so its dz has no zeros):
//
//   wgrad:  dW_r[e, h] = sum_t dz[t, e] x[t, h]
//   dgrad:  dx[t, h]   = sum_e dz[t, e] W_r[e, h]  (+ rest[t, h])
//
// Both are skinny (E up to 1024 beside thousands of tokens and columns): x, rest and dx are the
// bytes that count, dz and W_r stay in the caches.
//
// bf16 operands (fp32 sums) run on v_mfma_f32_32x32x16_bf16 over tiles of TM rows x 128 columns
// (rows: experts in wgrad, tokens in dgrad), K (tokens; experts) in stages of 32 through a ring of
// three LDS slots filled by direct-to-LDS loads two and a half stages ahead, fragments one K step
// ahead of their MFMAs.  Every stage of an operand is read through a buffer window that ends after its last
// valid element, so rows past the data load zeros.  Operands whose K index is the slow one (dz and
// x in wgrad, W_r in dgrad) lie in LDS as in memory and are read transposed.  A wgrad tile row past E
// and a column past H hold other elements' products and are not stored.  In dgrad the K tail of a
// row is the next row's values: fragments past E are cleared, as 0 times their W_r row of zeros would
// keep a NaN.  dz rows that are not multiples of 16 bytes (E % 8 != 0) come through registers.
//
// dz in three bf16 planes, whose sum is an fp32 value digit for digit (8 + 8 + 8 bits), gives products
// of the fp32 dz: a stage of 32 becomes three, one for each plane of dz beside the same stage of the other
// operand, which is loaded with the first and stays for the other two.
//
// wgrad has few tiles (E / TM x H / 128), so the tokens are cut into S ranges whose fp32 partial
// sums a second launch adds in order: the result has the same bits on every run.
//
// fp32 operands run on v_mfma_f32_32x32x2_f32 (products and sums in fp32).
//
// Measured, bf16, N 8192, E 256, H 7168, over changing inputs: wgrad 55 us with the sum of its 4 parts (117 MB of
// x, 29 MB of partial sums out and back; a bf16 library product 84); dgrad with rest 77 us (53 us of it are rest
// and dx, as with E = 8; about 0.1 us an expert comes on top; the library's sum and product 100).  With three
// planes of dz 128 and 149 us (113 and 120 on the same inputs again and again, 97 and 111 as steps of the layer);
// N 4096, E 8, H 4096: 23 and 21 us against 12 and 11.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "gemm_device.h"
#include "grouped_gemm.h"
#include "moe_common.h"
#include "moe_launch.h"

namespace moe {
namespace {

constexpr int kRbThreads = 256;
constexpr int kRbTN = 128;   // tile columns
constexpr int kRbKS = 32;    // K per stage
constexpr int kRbSlots = 3;

struct RbArgs {
  const void* dz;     // [N, E], or three planes of it
  const void* b;      // wgrad: x [N, H]; dgrad: W_r [E, H]
  const void* rest;   // dgrad: [N, H] or null
  void* out;          // wgrad: partial sums [S, E, H] fp32, or dW_r when S = 1; dgrad: dx
  int N, E, H;
  int S, span;        // wgrad: part s covers tokens s span .. (s + 1) span - 1
  int out_f32;
};

template <int TM>
struct RbCfg {
  static constexpr int kWM = TM / 64, kWN = 4 / kWM;       // waves along rows, columns
  static constexpr int kMB = 2, kNB = kRbTN / 32 / kWN;    // 32 x 32 blocks of a wave
  static constexpr int kABytes = TM * kRbKS * 2, kBBytes = kRbTN * kRbKS * 2;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kAOps = kABytes / 4096, kBOps = kBBytes / 4096;   // 1 KB loads per wave
};

// Swizzle of the strided operands: 16-byte chunk c of K-row r of `pitch` bytes lies in slot c ^
// key(r), so that the four rows of a transposing read hit distinct banks
template <int PITCH>
__device__ __forceinline__ int strided_key(int r) {
  if constexpr (PITCH >= 256) return 4 * (r & 3);
  else return 4 * ((r >> 1) & 1);
}
// dgrad's dz rows of 64 bytes
__device__ __forceinline__ int row_key(int r) { return (r >> 2) & 3; }

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) u32x4_t lds_vec16;

// Byte offset of the lane's first transposing read of columns col0 .. col0 + 31: lane i of group g
// (16 lanes) addresses 8 bytes of K-row 8 (g / 2) + i / 4
template <int PITCH>
__device__ __forceinline__ uint32_t strided_off(int col0, int lane) {
  const int g = lane >> 4, i = lane & 15;
  const int row = 8 * (g >> 1) + (i >> 2);
  const int byte = (col0 + 16 * (g & 1) + 4 * (i & 3)) * 2;
  return static_cast<uint32_t>(row * PITCH + ((((byte >> 4) ^ strided_key<PITCH>(row)) << 4) | (byte & 15)));
}
// Lane l: column col0 + l % 32, K-rows 16 s + 8 (l / 32) + 0..7
template <int PITCH>
__device__ __forceinline__ uint4 strided_frag(uint32_t addr, int s) {
  uint2 h[2];
#pragma unroll
  for (int r = 0; r < 2; ++r)
    h[r] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_v4s*>(
                                         static_cast<uintptr_t>(addr + (16 * s + 4 * r) * PITCH))));
  return make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
}

// DGRAD: dx; otherwise wgrad.  DMA: dz rows are multiples of 16 bytes from a 16-byte base.  PLANES: of dz
// (1 or 3)
template <bool DGRAD, int TM, bool DMA, int PLANES>
__global__ __launch_bounds__(kRbThreads, 2) void router_grad_kernel(RbArgs p) {
  using C = RbCfg<TM>;
  constexpr int kMB = C::kMB, kNB = C::kNB, kAOps = C::kAOps, kBOps = C::kBOps;
  constexpr int kADma = DMA ? kAOps : 0, kOps = kADma + kBOps;
  static_assert(PLANES == 1 || PLANES == kRbSlots, "plane p of a stage lies in slot p");
  constexpr int kPitch = kNB * 32 + 4;   // dgrad epilogue: floats of a staged row
  constexpr int kLds = DGRAD && 4 * 32 * kPitch * 4 > kRbSlots * C::kStage ? 4 * 32 * kPitch * 4 : kRbSlots * C::kStage;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_byte*)lds));
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::kWN, wn = wave % C::kWN;

  // ---- the tile: each XCD takes a contiguous range (wgrad: part -> row block -> column block,
  // so a part's dz stays in one L2; dgrad: token block -> column block)
  const int nT = (p.H + kRbTN - 1) / kRbTN;
  const int rowsM = DGRAD ? p.N : p.E;
  const int mT = (rowsM + TM - 1) / TM;
  const long long total = static_cast<long long>(mT) * nT * (DGRAD ? 1 : p.S);
  const long long per_xcd = (total + kNumXcd - 1) / kNumXcd;
  const long long slot = blockIdx.x / kNumXcd;
  const long long L = blockIdx.x % kNumXcd * per_xcd + slot;
  if (slot >= per_xcd || L >= total) return;
  const int n0 = static_cast<int>(L % nT) * kRbTN;
  const int m0 = static_cast<int>(L / nT % mT) * TM;
  const int part = static_cast<int>(L / nT / mT);
  const int k_lo = DGRAD ? 0 : part * p.span;
  const int k_hi = DGRAD ? p.E : (k_lo + p.span < p.N ? k_lo + p.span : p.N);
  const int nk = (k_hi - k_lo + kRbKS - 1) / kRbKS;
  const int mcount = rowsM - m0 < TM ? rowsM - m0 : TM;
  const int ncols = p.H - n0 < kRbTN ? p.H - n0 : kRbTN;
  const uint16_t* dz0 = reinterpret_cast<const uint16_t*>(p.dz);
  const size_t dz_n = static_cast<size_t>(p.N) * p.E;   // elements of a plane
  auto plane_of = [&](int plane) { return PLANES == 1 ? dz0 : dz0 + plane * dz_n; };
  const uint16_t* bm = reinterpret_cast<const uint16_t*>(p.b);

  // ---- loads: op j of a wave fills 1 KB group wave + 4 j of its operand
  constexpr int kACh = DGRAD ? 4 : TM / 8;       // 16-byte chunks of a dz row in LDS
  constexpr int kBCh = kRbTN / 8;
  auto a_row = [&](int j) { return (wave + 4 * j) * (64 / kACh) + lane / kACh; };
  auto a_key = [&](int r) { return DGRAD ? row_key(r) : strided_key<DGRAD ? 256 : TM * 2>(r); };
  uint32_t voff_a[kAOps], voff_b[kBOps];
#pragma unroll
  for (int j = 0; j < kAOps; ++j)
    voff_a[j] = static_cast<uint32_t>(a_row(j)) * p.E * 2 + (((lane % kACh) ^ a_key(a_row(j))) << 4);
#pragma unroll
  for (int j = 0; j < kBOps; ++j) {
    const int r = (wave + 4 * j) * (64 / kBCh) + lane / kBCh;
    voff_b[j] = static_cast<uint32_t>(r) * p.H * 2 + (((lane % kBCh) ^ strided_key<kRbTN * 2>(r)) << 4);
  }
  // stage ks of a plane into slot sl; the other operand's (with plane 0) into that of slot bsl
  auto load_stage = [&](int ks, int plane, int sl, int bsl) __attribute__((always_inline)) {
    const uint16_t* dz = plane_of(plane);
    const int k0 = k_lo + ks * kRbKS;
    const int left = k_hi - k0 < kRbKS ? k_hi - k0 : kRbKS;
    const uint32_t base = __builtin_amdgcn_readfirstlane(lds0 + sl * C::kStage);
    if constexpr (DMA) {
      const u32x4_t wa =
          DGRAD ? buffer_window(dz + static_cast<size_t>(m0) * p.E + k0,
                                (static_cast<uint32_t>(mcount - 1) * p.E + left) * 2)
                : buffer_window(dz + static_cast<size_t>(k0) * p.E + m0,
                                (static_cast<uint32_t>(left - 1) * p.E + mcount) * 2);
#pragma unroll
      for (int j = 0; j < kAOps; ++j) dma16_window(wa, voff_a[j], base + (wave + 4 * j) * 1024);
    }
    if (PLANES > 1 && plane != 0) return;
    const uint32_t base_b = PLANES == 1 ? base : __builtin_amdgcn_readfirstlane(lds0 + bsl * C::kStage);
    const u32x4_t wb = buffer_window(bm + static_cast<size_t>(k0) * p.H + n0,
                                     (static_cast<uint32_t>(left - 1) * p.H + ncols) * 2);
#pragma unroll
    for (int j = 0; j < kBOps; ++j) dma16_window(wb, voff_b[j], base_b + C::kABytes + (wave + 4 * j) * 1024);
  };
  // (rows that are not multiples of 16 bytes) one 16-byte chunk of 8 elements per op: a load of 2-byte
  // alignment while all 8 lie in dz, element by element at its end.  Zeros past the rows and, in
  // dgrad, past the columns of dz.
  auto read_a = [&](int ks, int plane, uint4 (&v)[kAOps]) __attribute__((always_inline)) {
    const uint16_t* dz = plane_of(plane);
    struct __attribute__((packed, aligned(2))) Chunk {
      uint32_t w[4];
    };
    const int k0 = k_lo + ks * kRbKS;
#pragma unroll
    for (int j = 0; j < kAOps; ++j) {
      const int r = a_row(j), c = (lane % kACh) ^ a_key(r);
      const int row = DGRAD ? m0 + r : k0 + r, col = (DGRAD ? k0 : m0) + 8 * c;
      const size_t at = static_cast<size_t>(row) * p.E + col;
      v[j] = make_uint4(0, 0, 0, 0);
      if (row >= (DGRAD ? p.N : k_hi) || col >= p.E) continue;
      if (at + 8 <= dz_n) {
        const Chunk q = *reinterpret_cast<const Chunk*>(dz + at);
        v[j] = make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
      } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = at + i < dz_n ? dz[at + i] : 0u;
        v[j] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
      }
      if constexpr (DGRAD) {
        const int n = p.E - col;   // elements of the row
        auto keep = [&](uint32_t w, int i) { return n >= i + 2 ? w : (n > i ? w & 0xFFFFu : 0u); };
        v[j] = make_uint4(keep(v[j].x, 0), keep(v[j].y, 2), keep(v[j].z, 4), keep(v[j].w, 6));
      }
    }
  };
  auto put_a = [&](int sl, const uint4 (&v)[kAOps]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kAOps; ++j)
      *reinterpret_cast<uint4*>(lds + sl * C::kStage + (wave + 4 * j) * 1024 + lane * 16) = v[j];
  };

  // ---- fragment addresses inside a slot
  uint32_t fo_a[2], fo_b[kNB];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (DGRAD) {   // i: K half; row block 32 further is 2 KB further
      const int r = wm * 64 + (lane & 31);
      fo_a[i] = static_cast<uint32_t>(r * 64 + (((2 * i + (lane >> 5)) ^ row_key(r)) << 4));
    } else {                 // i: row block
      fo_a[i] = strided_off<TM * 2>(wm * 64 + 32 * i, lane);
    }
  }
#pragma unroll
  for (int j = 0; j < kNB; ++j) fo_b[j] = C::kABytes + strided_off<kRbTN * 2>((wn * kNB + j) * 32, lane);

  f32x16_t acc[kMB][kNB];
#pragma unroll
  for (int i = 0; i < kMB; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[i][j] = f32x16_t{};

  // ---- K loop.  Stage st (stage ks of a plane), two K steps of 16, fragments one step ahead of their MFMAs:
  //   read step 1; multiply step 0; wait for stage st + 1 and synchronise (every wave has now read
  //   all of stage st); load stage st + 3 into its slot; read step 0 of stage st + 1; multiply step 1
  // With three planes slot sl is that of plane sl, and the other operand's stages go round the three slots
  // by themselves: stage ks + 1 is loaded while plane 0 of stage ks is multiplied, into the place of ks - 2.
  struct Frags {
    uint4 a[kMB], b[kNB];
  };
  auto read_frags = [&](int sl, int bsl, int s, Frags& f) __attribute__((always_inline)) {
    const uint32_t sb = lds0 + sl * C::kStage, bb = PLANES == 1 ? sb : lds0 + bsl * C::kStage;
#pragma unroll
    for (int i = 0; i < kMB; ++i) {
      if constexpr (DGRAD)
        f.a[i] = __builtin_bit_cast(uint4, *reinterpret_cast<lds_vec16*>(static_cast<uintptr_t>(sb + fo_a[s] + i * 2048)));
      else
        f.a[i] = strided_frag<TM * 2>(sb + fo_a[i], s);
    }
#pragma unroll
    for (int j = 0; j < kNB; ++j) f.b[j] = strided_frag<kRbTN * 2>(bb + fo_b[j], s);
  };
  auto multiply = [&](int ks, int s, Frags& f) __attribute__((always_inline)) {
    if constexpr (DGRAD) {
      if (ks == nk - 1) {   // dz past the row's end: the next row's values
        const bool past = ks * kRbKS + 16 * s + 8 * (lane >> 5) >= p.E;
#pragma unroll
        for (int i = 0; i < kMB; ++i)
          if (past) f.a[i] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j)
        acc[i][j] = DGRAD ? mma_bf16(f.b[j], f.a[i], acc[i][j]) : mma_bf16(f.a[i], f.b[j], acc[i][j]);
  };
  constexpr int kLanes = kNB * 4;                    // dgrad epilogue: lanes along a row, 8 columns each
  constexpr int kRest = DGRAD ? 32 * kLanes / 64 : 1;   // and the 16-byte words of rest they add
  uint4 rest_w[kMB][kRest];
  const uint16_t* rest = reinterpret_cast<const uint16_t*>(p.rest);
  auto load_rest = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < kRest; ++t) {
      const int row = m0 + wm * 64 + i * 32 + t * (64 / kLanes) + lane / kLanes;
      const int col = n0 + wn * kNB * 32 + 8 * (lane % kLanes);
      rest_w[i][t] = rest != nullptr && row < p.N && col < p.H
                         ? *reinterpret_cast<const uint4*>(rest + static_cast<size_t>(row) * p.H + col)
                         : make_uint4(0, 0, 0, 0);
    }
  };
  // rest is read ahead of everything else, as far as registers go (256-row tiles: the first of the
  // wave's two row blocks, the second in the epilogue); read where it is added it cost 7 us of 60
  // at N 8192, E 8, H 7168
  constexpr int kEarly = TM < 256 ? kMB : 1;
  if constexpr (DGRAD) {
#pragma unroll
    for (int i = 0; i < kEarly; ++i) load_rest(i);
  }
  uint4 va[kAOps];
  auto first_stage = [&](int st) __attribute__((always_inline)) {
    const int ks = PLANES == 1 ? st : 0, plane = PLANES == 1 ? 0 : st;
    load_stage(ks, plane, st, 0);
    if constexpr (!DMA) {
      read_a(ks, plane, va);
      put_a(st, va);
    }
  };
  const int nst = nk * PLANES;
  first_stage(0);
  if (nst > 1) first_stage(1);
  if (nst > 2) first_stage(2);
  if constexpr (PLANES > 1) wait_vmcnt<2 * kADma>();   // (stages 1 and 2 are planes of the same stage)
  else if (nk > 2) wait_vmcnt<2 * kOps>();
  else if (nk > 1) wait_vmcnt<kOps>();
  else wait_vmcnt<0>();
  wait_lgkmcnt_all();
  block_barrier();
  Frags f0, f1;
  read_frags(0, 0, 0, f0);
  int sl = 0, ks = 0, bsl = 0;   // ring slot of stage st; its K stage; slot of the other operand's stage
  for (int st = 0; st < nst; ++st) {
    const bool next = st + 1 < nst, load = st + kRbSlots < nst;
    const int ks3 = PLANES == 1 ? ks + kRbSlots : ks + 1;   // (stage st + 3: with planes, the same plane)
    const int plane3 = PLANES == 1 ? 0 : sl;
    if constexpr (!DMA) {
      if (load) read_a(ks3, plane3, va);
    }
    read_frags(sl, bsl, 1, f1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(ks, 0, f0);
    const int sl1 = sl + 1 == kRbSlots ? 0 : sl + 1, bsl3 = bsl + 1 == kRbSlots ? 0 : bsl + 1;
    const bool turn = PLANES == 1 || sl1 == 0;   // stage st + 1 is another K stage
    const int bsl1 = turn ? bsl3 : bsl;
    if (next) {
      wait_lgkmcnt_all();
      if (st + 2 >= nst) wait_vmcnt<0>();
      else if (PLANES == 1 || sl == 1) wait_vmcnt<kOps>();   // stage st + 2 has loads of both operands
      else wait_vmcnt<kADma>();
      block_barrier();
      if (load) {
        load_stage(ks3, plane3, sl, bsl3);
        if constexpr (!DMA) put_a(sl, va);
      }
      read_frags(sl1, bsl1, 0, f0);
      __builtin_amdgcn_sched_barrier(0);
    }
    multiply(ks, 1, f1);
    sl = sl1;
    bsl = bsl1;
    if (turn) ++ks;
  }

  if constexpr (!DGRAD) {
    // lane l holds column l % 32 of a block and, in register v, row 8 (v / 4) + 4 (l / 32) + v % 4:
    // each store writes two rows' 128 bytes, through a window that ends with the tile's last
    // element (lanes past the columns take an offset behind it)
    const uint32_t esz = p.out_f32 ? 4 : 2;
    uint8_t* const base = reinterpret_cast<uint8_t*>(p.out) + ((static_cast<size_t>(part) * p.E + m0) * p.H + n0) * esz;
    const __amdgpu_buffer_rsrc_t win = __builtin_amdgcn_make_buffer_rsrc(
        base, 0, static_cast<int>((static_cast<uint32_t>(mcount - 1) * p.H + ncols) * esz), 0x00020000);
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j) {
        const int n = (wn * kNB + j) * 32 + (lane & 31);
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int r = wm * 64 + i * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
          const int off = n < ncols ? static_cast<int>((static_cast<uint32_t>(r) * p.H + n) * esz) : INT_MIN;
          if (p.out_f32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][v]), win, off, 0, 0);
          else __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(acc[i][j][v]), win, off, 0, 0);
        }
      }
  } else {
    // lane l holds token l % 32 of a block and runs of 4 columns: a wave's 32 rows go through LDS in
    // fp32, then 8 columns a lane along the rows, rest added, one rounding
    wait_lgkmcnt_all();
    block_barrier();   // every wave is past its last fragment reads
    float* st = reinterpret_cast<float*>(lds) + wave * 32 * kPitch;
#pragma unroll
    for (int i = 0; i < kMB; ++i) {
      if (i + 1 < kMB && i + 1 >= kEarly) load_rest(i + 1);
#pragma unroll
      for (int j = 0; j < kNB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16_t& a = acc[i][j];
          *reinterpret_cast<float4*>(st + (lane & 31) * kPitch + j * 32 + 8 * q + 4 * (lane >> 5)) =
              make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      wait_lgkmcnt_all();
#pragma unroll
      for (int t = 0; t < kRest; ++t) {
        const int r = t * (64 / kLanes) + lane / kLanes, c = 8 * (lane % kLanes);
        const int row = m0 + wm * 64 + i * 32 + r, col = n0 + wn * kNB * 32 + c;
        if (row >= p.N || col >= p.H) continue;
        const float4 x = *reinterpret_cast<const float4*>(st + r * kPitch + c);
        const float4 y = *reinterpret_cast<const float4*>(st + r * kPitch + c + 4);
        float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        const size_t o = static_cast<size_t>(row) * p.H + col;
        const uint4 q = rest_w[i][t];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[2 * k] += __uint_as_float(w[k] << 16);
          v[2 * k + 1] += __uint_as_float(w[k] & 0xFFFF0000u);
        }
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + o) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// fp32: tiles of 64 rows x 128 columns on v_mfma_f32_32x32x2_f32 (4 waves of 32 x 64; lane l supplies
// row l % 32 at k = l / 32 of both operands), K in steps of 16 through two LDS buffers, the next
// step's elements in registers meanwhile.  Both operands lie k-row after k-row, rows padded so that
// the two k-rows of a fragment read fall into different halves of the banks.
constexpr int kF32TM = 64, kF32TN = 128, kF32KS = 16;
constexpr int kF32APitch = kF32TM + 32, kF32BPitch = kF32TN + 32;
static_assert(kF32APitch % 64 == 32 && kF32BPitch % 64 == 32, "k-rows alternate between the bank halves");

template <bool DGRAD>
__global__ __launch_bounds__(kRbThreads) void router_grad_f32_kernel(RbArgs p) {
  __shared__ float as[2][kF32KS][kF32APitch];
  __shared__ __attribute__((aligned(16))) float bs[2][kF32KS][kF32BPitch];
  const float* dz = reinterpret_cast<const float*>(p.dz);
  const float* b = reinterpret_cast<const float*>(p.b);
  const int tid = threadIdx.x, lane = tid & 63, wm = tid >> 7, wn = (tid >> 6) & 1;
  const int m0 = blockIdx.x * kF32TM, n0 = blockIdx.y * kF32TN, part = blockIdx.z;
  const int M = DGRAD ? p.N : p.E;
  const int k_lo = DGRAD ? 0 : part * p.span;
  const int k_hi = DGRAD ? p.E : (k_lo + p.span < p.N ? k_lo + p.span : p.N);
  const bool vec = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.dz) % 16 == 0;   // dz rows by 16 bytes
  // A: 4 elements a thread, contiguous in memory: wgrad expert run 4 (tid % 16) of token tid / 16;
  // dgrad expert run 4 (tid / 64) of token tid % 64
  const int ak = DGRAD ? 4 * (tid >> 6) : tid >> 4, am = DGRAD ? tid & 63 : 4 * (tid & 15);
  // B: columns 4 (tid % 32) .. + 3 of k-rows tid / 32 and tid / 32 + 8
  const int bk = tid >> 5, bn = 4 * (tid & 31);
  float ra[4];
  float4 rb[2];
  auto load = [&](int k0) __attribute__((always_inline)) {
    const int row = DGRAD ? m0 + am : k0 + ak, col = DGRAD ? k0 + ak : m0 + am;   // of dz
    const bool in = row < (DGRAD ? M : k_hi);
    const float* at = dz + static_cast<size_t>(row) * p.E + col;
    if (vec) {
      const float4 q = in && col < p.E ? *reinterpret_cast<const float4*>(at) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      ra[0] = q.x; ra[1] = q.y; ra[2] = q.z; ra[3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) ra[i] = in && col + i < p.E ? at[i] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = k0 + bk + 8 * u, n = n0 + bn;
      rb[u] = k < k_hi && n < p.H ? *reinterpret_cast<const float4*>(b + static_cast<size_t>(k) * p.H + n)
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // (H % 4 == 0)
    }
  };
  auto store = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) as[buf][DGRAD ? ak + i : ak][DGRAD ? am : am + i] = ra[i];
#pragma unroll
    for (int u = 0; u < 2; ++u) *reinterpret_cast<float4*>(&bs[buf][bk + 8 * u][bn]) = rb[u];
  };
  f32x16_t acc[2] = {};
  load(k_lo);
  // rest is read before the K loop: between the stores, each read would wait for the one before
  // (N 2048, E 128, H 8192: 90 -> 68 us; N 300, E 16, H 4096: 14 -> 6 us)
  float rest[DGRAD ? 2 : 1][16];
  if constexpr (DGRAD) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int n = n0 + wn * 64 + j * 32 + (lane & 31), m = m0 + wm * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
        rest[j][v] = p.rest != nullptr && m < M && n < p.H
                         ? reinterpret_cast<const float*>(p.rest)[static_cast<size_t>(m) * p.H + n]
                         : 0.0f;
      }
  }
  store(0);
  __syncthreads();
  int buf = 0;
  for (int k0 = k_lo; k0 < k_hi; k0 += kF32KS) {
    const bool next = k0 + kF32KS < k_hi;
    if (next) load(k0 + kF32KS);
#pragma unroll
    for (int s = 0; s < kF32KS / 2; ++s) {
      const int k = 2 * s + (lane >> 5);
      const float fa = as[buf][k][wm * 32 + (lane & 31)];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa, bs[buf][k][wn * 64 + j * 32 + (lane & 31)], acc[j], 0, 0, 0);
    }
    if (next) store(buf ^ 1);
    __syncthreads();
    buf ^= 1;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = n0 + wn * 64 + j * 32 + (lane & 31);
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int m = m0 + wm * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
      if (m >= M || n >= p.H) continue;
      float x = acc[j][v];
      const size_t o = (static_cast<size_t>(DGRAD ? 0 : part) * M + m) * p.H + n;
      if constexpr (DGRAD) x += rest[j][v];
      if (p.out_f32) reinterpret_cast<float*>(p.out)[o] = x;
      else reinterpret_cast<uint16_t*>(p.out)[o] = f32_to_bf16(x);
    }
  }
}

// dW_r = part_0 + part_1 + ... in that order (n4 groups of 4; S = 0: zeros)
__global__ __launch_bounds__(kRbThreads) void router_wgrad_sum_kernel(const float4* __restrict__ part, int S,
                                                                      long long n4, void* __restrict__ dw, int f32) {
  const long long step = static_cast<long long>(gridDim.x) * kRbThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kRbThreads + threadIdx.x; i < n4; i += step) {
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = 0; s0 < S; s0 += 8) {   // (eight parts' loads together)
      float4 b[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        b[u] = s0 + u < S ? part[(s0 + u) * n4 + i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        a.x += b[u].x;
        a.y += b[u].y;
        a.z += b[u].z;
        a.w += b[u].w;
      }
    }
    if (f32) reinterpret_cast<float4*>(dw)[i] = a;
    else reinterpret_cast<uint2*>(dw)[i] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

// dgrad: 256 tokens halve the reads of W_r, but two workgroups fit a CU (128 tokens: three, 64: four).
// Up to 128 experts the reads and writes of rest and dx count for more and smaller tiles keep more of them in
// flight; with few tiles they also use more CUs and end sooner.  Measured with rest, us on 64 / 128 / 256
// tokens (tiles of 64 tokens):
//   N 300,  H 7168 (280):   E 8    4.3 /  5.3 /  8.2    E 256    7.8 /  8.2 / 12.2
//   N 2048, H 2048 (512):   E 64   5.6 /  6.4 /  8.9    E 512   12.9 / 13.2 / 17.2
//   N 1024, H 7168 (896):   E 64   8.8 /  9.5 / 11.0    E 256   15.0 / 14.1 / 14.8
//   N 4096, H 4096 (2048):  E 8   13.5 / 14.9 / 14.1    E 256   23.2 / 23.1 / 22.1
//   N 8192, H 4096 (4096):  E 64  39.3 / 37.1 / 36.0    E 256   57.6 / 51.9 / 48.9
//   N 8192, H 7168 (7168):  E 64  63.0 / 58.4 / 60.2    E 256  103.9 / 86.6 / 82.7
// dz rows through registers wait in each stage, and more workgroups share the waits:
//   N 4096, H 4096 (2048):  E 60  16.5 / 19.3 / 17.5    E 250  30.1 / 34.1 / 32.1
//   N 8192, H 7168 (7168):  E 60  64.1 / 61.0 / 66.0    E 250  108.7 / 100.7 / 121.8
// Three planes of dz follow the same rule:
//   N 1024, H 7168 (896):   E 64  10.9 / 11.4 / 12.5    E 256  24.6 / 23.3 / 24.1
//   N 4096, H 4096 (2048):  E 64  19.5 / 20.3 / 19.1    E 512  79 / 69 / 59
//   N 8192, H 7168 (7168):  E 64  51 / 54 / 59          E 256  134 / 126 / 118
int rb_dgrad_rows(int N, int E, int H, bool dma) {
  const long long t64 = static_cast<long long>((N + 63) / 64) * ((H + kRbTN - 1) / kRbTN);
  if (!dma) return t64 <= 4096 ? 64 : 128;
  if (E <= 128) return t64 <= 2048 ? 64 : 128;
  return t64 <= 640 ? 64 : (t64 <= 1024 ? 128 : 256);
}

// Row tile and token ranges of a wgrad.
// bf16: the pair with the least of
//   stages of a range * t  +  (more than one range: 2 + (S + 3) * 8 E H bytes / 10 TB/s + S / 8 * 0.5)   us
// where t is a stage's time by tile rows while a CU has one workgroup, and the second part the sum's
// launch, the partial sums' way out and back, and the sum's batches of eight.  Workgroups beyond 256
// take the CU's time from each other, so there are no more unless the tiles alone are.  dz rows that
// come through registers wait for their loads in each stage: t is longer, and workgroups share the
// waits; so do three planes of dz, whose stages bring only dz rows two times of three.  Measured with
// the sum, us by S = 1 / 2 / 4 / 8 / 16 (64-row tiles to E 64, then 128, 256):
//   N 300,  H 7168, E 8     5.7 /  6.7 /  6.4 /  6.8        E 256  13.3 / 20.3 / 23.5 / 24.0
//   N 1024, H 1024, E 8    10.9 /  9.1 /  7.3 /  6.4 /  6.7   E 256  22.7 / 18.3 / 15.4 / 16.2 / 19.5
//   N 1024, H 7168, E 64   11.4 / 11.3 / 11.6 / 15.9 / 18.4   E 256  24.2 / 25.8 / 23.6 / 28.1 / 44.2
//   N 4096, H 7168, E 64   35.1 / 22.0 / 16.2 / 17.9 / 21.0   E 256  71.7 / 47.5 / 36.5 / 39.3 / 62.5
//   N 2500, H 7168, E 60   51.7 / 31.0 / 20.3 / 16.6 / 18.2   E 250  94.0 / 56.8 / 39.2 / 36.6 / 54.0
//   N 8192, H 7168, E 256: 4 ranges 55, 9 ranges 62;  E 5: 8 ranges 38, 16 ranges 29
// and by tile rows 64 / 128 / 256 with the best S of each:
//   N 300,  H 2048, E 256   5.8 /  8.1 / 12.5     N 1000, H 7168, E 256  12.4 / 15.5 / 23.8
//   N 8192, H 2048, E 256  24.1 / 22.1 / 26.6     N 8192, H 7168, E 256  89.1 / 60.9 / 55.5
// Three planes, S = 4 / 8 / 16: N 8192, H 8192, E 32  77 / 46 / 42 (with 256 workgroups at most 60);
//   N 8192, H 7168, 256-row tiles, E 256: 4 ranges 134, 8 ranges 103, 9 ranges 114;  E 128 (128 rows): 4 ranges 80, 9
//   ranges 59;  N 1024, H 7168, E 64: 16.4 / 18.3;  N 300, H 2048, E 256: 1 range 11.9, 5 ranges 14.2.
// From 90 MB of x on, 64-row tiles are bound by its reading (inputs that no cache holds): where 256 workgroups
// are not a whole number of tiles, 512 fill the CUs better.  us with 256 / 512 / 1024 workgroups at most:
//   N 8192,  H 5632 (44 tiles):  E 8  25.6 / 22.6 / 24.7    E 32  26.0 / 24.6 / 28.0    E 64  27.0 / 27.6 / 32.7
//   N 8192,  H 6656 (52):        E 8  29.6 / 24.8 / 27.8    E 32  30.1 / 27.0 / 31.2    E 64  31.3 / 30.1 / 35.8
//   N 6400,  H 7168 (56):        E 8  24.7 / 21.9 / 24.3    E 32  25.1 / 23.7 / 27.7    E 64  26.7 / 27.2 / 32.5
//   N 16384, H 7168 (56):        E 8  52.8 / 45.9 / 49.8    E 32  53.2 / 48.5 / 53.6    E 64  54.6 / 53.3 / 58.9
//   N 16384, H 5120 (40):        E 8  37.8 / 35.5 / 38.2    E 32  38.9 / 38.0 / 41.5    E 64  41.7 / 41.1 / 46.1
// and where they are:
//   N 16384, H 4096 (32):        E 8  30.5 / 30.8 / 34.5    E 32  31.3 / 32.7 / 37.4    E 64  33.2 / 35.2 / 40.6
//   N 8192,  H 8192 (64):        E 8  28.7 / 30.0 / 33.0    E 32  29.6 / 32.7 / 37.3    E 64  31.4 / 37.3 / 44.1
// fp32 (N 2048, E 128, H 8192, 256 / 512 / 1024 workgroups: 84 / 59 / 57 us; E 64, H 4096: 28 / 24 / 27):
// 512, of at least two steps.
struct RbSplit {
  int S, span, rows;
};
RbSplit rb_split(int N, int H, int E, bool bf16, int planes) {
  const int step = bf16 ? kRbKS : kF32KS, steps = (N - 1) / step + 1;
  const int n_tiles = bf16 ? (H + kRbTN - 1) / kRbTN : (H + kF32TN - 1) / kF32TN;
  auto tiles = [&](int rows) { return static_cast<long long>((E + rows - 1) / rows) * n_tiles; };
  auto at_most = [&](int groups, int rows) { return tiles(rows) >= groups ? 1 : static_cast<int>(groups / tiles(rows)); };
  int S = 1, rows = kF32TM;
  if (!bf16) {
    const int most = (steps + 1) / 2;
    S = at_most(512, rows) < most ? at_most(512, rows) : most;
  } else if (planes == 1 && E <= 64 && E % 8 == 0 && static_cast<long long>(N) * H >= 45000000 && tiles(64) * at_most(256, 64) <= 240) {
    rows = 64;
    S = at_most(512, rows);
  } else {
    const bool waits = E % 8 != 0 || planes > 1;
    const float move = static_cast<float>(E) * static_cast<float>(H) * 8e-7f;
    const float stage[2][3] = {{0.25f, 0.33f, 0.5f}, {0.5f, 0.7f, 1.1f}};
    const int groups[3] = {1024, 512, 512};
    float best = 0.0f;
    for (int i = 0; i < 3; ++i) {
      const int r = 64 << i, most = at_most(waits ? groups[i] : 256, r);
      for (int c = 1; c <= most && c <= steps; ++c) {
        const float load = static_cast<float>(tiles(r)) * static_cast<float>(c) * (1.0f / 256);
        const float t = stage[waits][i] * (load <= 1.0f ? 1.0f : (waits ? sqrtf(load) : load));
        float us = static_cast<float>((steps + c - 1) / c * planes) * t;
        if (c > 1) us += 2.0f + static_cast<float>(c + 3) * move + 0.5f * static_cast<float>((c + 7) / 8);
        if ((i == 0 && c == 1) || us < best) {
          best = us;
          S = c;
          rows = r;
        }
      }
      if (r >= E) break;
    }
  }
  const long long span = static_cast<long long>((steps + S - 1) / S) * step;   // whole steps
  return {static_cast<int>((N + span - 1) / span), static_cast<int>(span < INT_MAX ? span : INT_MAX), rows};
}

unsigned rb_grid(long long tiles) {
  return static_cast<unsigned>((tiles + kNumXcd - 1) / kNumXcd * kNumXcd);
}

template <bool DGRAD, int TM, int PLANES>
hipError_t rb_launch(const RbArgs& p, bool dma, long long tiles, hipStream_t s) {
  if (dma)
    hipLaunchKernelGGL((router_grad_kernel<DGRAD, TM, true, PLANES>), dim3(rb_grid(tiles)), dim3(kRbThreads), 0, s, p);
  else if constexpr (!DGRAD || TM < 256)   // (a dgrad takes 256 tokens with 16-byte dz rows only)
    hipLaunchKernelGGL((router_grad_kernel<DGRAD, TM, false, PLANES>), dim3(rb_grid(tiles)), dim3(kRbThreads), 0, s, p);
  else
    return hipErrorNotSupported;
  return hipGetLastError();
}

bool rb_dma(const RbArgs& p) { return p.E % 8 == 0 && reinterpret_cast<uintptr_t>(p.dz) % 16 == 0; }

template <bool DGRAD, int PLANES>
hipError_t rb_run(const RbArgs& p, int tm, hipStream_t s) {
  const int rows = DGRAD ? p.N : p.E;
  const bool dma = rb_dma(p);
  const long long tiles = static_cast<long long>((rows + tm - 1) / tm) * ((p.H + kRbTN - 1) / kRbTN) * (DGRAD ? 1 : p.S);
  if (tm == 256) return rb_launch<DGRAD, 256, PLANES>(p, dma, tiles, s);
  if (tm == 128) return rb_launch<DGRAD, 128, PLANES>(p, dma, tiles, s);
  return rb_launch<DGRAD, 64, PLANES>(p, dma, tiles, s);
}

}  // namespace

size_t router_wgrad_ws_bytes(int N, int H, int E, bool bf16, int planes) {
  if (N <= 0) return 0;
  const RbSplit r = rb_split(N, H, E, bf16, planes);
  return r.S <= 1 ? 0 : (static_cast<size_t>(r.S) * E * H * sizeof(float) + 255) & ~static_cast<size_t>(255);
}

hipError_t launch_router_dense_wgrad(const void* dz, int planes, const void* x, bool bf16, int N, int E, int H,
                                     void* dw, bool dw_f32, void* ws, hipStream_t s) {
  const RbSplit r = N > 0 ? rb_split(N, H, E, bf16, planes) : RbSplit{0, 0, 0};
  RbArgs p = {dz, x, nullptr, r.S > 1 ? ws : dw, N, E, H, r.S, r.span, r.S > 1 || dw_f32 ? 1 : 0};
  if (r.S > 0) {
    hipError_t err = hipSuccess;
    if (bf16) {
      err = planes == 3 ? rb_run<false, 3>(p, r.rows, s) : rb_run<false, 1>(p, r.rows, s);
    } else {
      hipLaunchKernelGGL(router_grad_f32_kernel<false>,
                         dim3((E + kF32TM - 1) / kF32TM, (H + kF32TN - 1) / kF32TN, r.S), dim3(kRbThreads), 0, s, p);
      err = hipGetLastError();
    }
    if (err != hipSuccess || r.S == 1) return err;
  }
  const long long n4 = static_cast<long long>(E) * H / 4;
  const long long blocks = (n4 + kRbThreads - 1) / kRbThreads;
  hipLaunchKernelGGL(router_wgrad_sum_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)),
                     dim3(kRbThreads), 0, s, reinterpret_cast<const float4*>(ws), r.S, n4, dw, dw_f32 ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_router_dense_dgrad(const void* dz, int planes, const void* w_r, bool bf16, int N, int E, int H,
                                     const void* rest, void* dx, hipStream_t s) {
  const RbArgs p = {dz, w_r, rest, dx, N, E, H, 1, 0, bf16 ? 0 : 1};
  if (bf16 && planes == 3) return rb_run<true, 3>(p, rb_dgrad_rows(N, E, H, rb_dma(p)), s);
  if (bf16) return rb_run<true, 1>(p, rb_dgrad_rows(N, E, H, rb_dma(p)), s);
  hipLaunchKernelGGL(router_grad_f32_kernel<true>, dim3((N + kF32TM - 1) / kF32TM, (H + kF32TN - 1) / kF32TN),
                     dim3(kRbThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace moe
