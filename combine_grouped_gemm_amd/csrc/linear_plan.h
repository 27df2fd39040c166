// What the experts' product launches for given sizes: the kernel, the parts of K and the workgroups.  Host
// code without HIP: the launch, its checks, the workspace query and the tests of the choice share it.
#pragma once

namespace moe {

constexpr int kLinRow = 128;   // bytes of a row and stage
constexpr int kLinXcds = 8;

// Which kernel a call runs: the few-rows kernel, or tiles of a shape with K in `split` parts.  Known on
// the host are the sizes, not the rows an expert gets; `each` rows of `hit` experts are expected.  The
// estimate is us = rounds x (stages x time of a stage + overhead), no less than the bytes at 5.2 TB/s, and
// for a split the sums' way through memory.  Its constants are from measured runs of every kernel on the
// same sizes; bf16, one expert, N 4096 (us; the smallest of each column is what the estimate takes, or
// within 3% of it):
//     K, rows           4096: 1   16   64  512 1024 2048    14336: 64  512 1024 2048 4096
//     few rows               9   10   16  100  194  385            54  336  659 1309 2592
//     64 x 64               22   22   23   33   58  111            90  129  243  449  851
//       K in 4 parts        13   14   15   47   85  176            35  139  253  456  822
//     128 x 256             37   37   43   54   56   69           179  192  190  219  438
//       K in 2 parts        24   24   28   40   49   94            98  109  124  243  438
//       K in 4 parts        17   17   20   35   68  121            58   74  140  272  435
//     320 x 256             69   69   72   94   94  110           297  343  333  347  401
//       K in 4 parts        25   25   27   43   56  109            85  108  125  256  404
// (K 14336, 2048 rows: 320 x 256 with 256-row tiles in 2 parts, 214 where 128 x 256 takes 212 in the same
// process.)  fp32, N 4096, K 4096: 2000 rows 32 x 64 560, 128 x 128 491, few rows 842; 512 rows 153, 257 (2
// parts 145), 226; 200 rows 82, 257 (4 parts 77), 96.  Gated calls run 64 x 128 and 32 x 128 tiles in place of
// 64 x 64 and 32 x 64 (half as many, each with twice the work, fewer of them a CU); the estimate takes the plain
// shapes' counts and constants for them, which no gated runs have been fitted to.
enum { LIN_FEW, LIN_64, LIN_128, LIN_320, LIN_32 };   // (bf16: 64, 128, 320; fp32: 32, 128)
struct LinPlan {
  int kind, split, tile_rows;
};

inline long long lin_ceil_div(long long a, long long b) { return (a + b - 1) / b; }

inline LinPlan lin_plan(int rows, int K, int Nw, int E, bool f32) {
  const int esz = f32 ? 4 : 2;
  const double row = 1.0 * K * esz;   // bytes of a row of a and of W
  const double stages = static_cast<double>(lin_ceil_div(1ll * K * esz, kLinRow));
  const int hit = E < rows ? E : rows;
  const double each = static_cast<double>(rows) / hit;
  const double mem = (1.0 * hit * Nw * row + rows * (row + 1.0 * Nw * esz)) / 5.2e6;
  LinPlan best{LIN_64, 1, 0};
  double best_us = 1e30;
  if (each <= 32) {
    const long long groups = hit * lin_ceil_div(Nw, 32);
    const double more = each > 16 ? (E == 1 && groups <= 128 ? 1.1 : 1.3)
                                  : E > 1 && each > 8 ? 1.05 : 1.0;   // (some experts' weights twice)
    const double waves = (groups <= 128 ? 0.5 : static_cast<double>(lin_ceil_div(groups, 512))) * stages / 4 * 0.3 * more *
                         (f32 ? 1.5 : 1.0);
    best = LinPlan{LIN_FEW, 1, 0};
    best_us = 4 + (mem * more > waves ? mem * more : waves);
  }
  struct Shape {
    int kind, tm, tn, per_cu, resident;   // tiles a CU works on at their full pace, and holds
    double overhead, latency, full;   // us of a tile beside its stages; of a stage: without and with all rows
  };
  static const Shape bf16_shapes[] = {{LIN_64, 64, 64, 3, 3, 5, 0.31, 0.4}, {LIN_128, 128, 256, 1, 1, 6, 0.5, 1.02},
                                      {LIN_320, 320, 256, 1, 1, 8, 0.95, 1.75}};
  static const Shape f32_shapes[] = {{LIN_32, 32, 64, 1, 4, 6, 0.28, 0.28}, {LIN_128, 128, 128, 1, 2, 6, 2.0, 2.0}};
  for (int i = 0; i < (f32 ? 2 : 3); ++i) {
    const Shape& s = f32 ? f32_shapes[i] : bf16_shapes[i];
    // m-tiles: uneven experts, a standard deviation of random routes above the mean
    const double even = E == 1 ? static_cast<double>(lin_ceil_div(rows, s.tm))
                               : 1.0 * hit * lin_ceil_div(static_cast<long long>(each + __builtin_sqrt(each)), s.tm);
    const long long nN = lin_ceil_div(Nw, s.tn);
    const double l2 = even * nN * (s.tm + s.tn) * row / 1.7e7;   // what the tiles load, at 17 TB/s
    for (int split = 1; split <= 16 && split * 8 <= (stages > 8 ? stages : 8); split *= 2) {
      const double turns = even * nN * split / (256.0 * s.per_cu);
      const double whole = static_cast<double>(static_cast<long long>(turns + (E == 1 ? 0.999 : 0.94)));
      const double rounds = turns <= 1 ? 1.0 : E == 1 || turns < 4.0 ? whole : turns + 0.15;   // (uneven experts: an estimate)
      // one expert on 320-row tiles: as many as the rounds have room for, so shorter ones (4096 x 14336 x
      // 4096: 256 tiles of 256 rows 375 us, 208 of 320 389; where the rounds are full 320 rows win: N 14336
      // of K 4096, 728 tiles 370 us, 896 of 256 rows 419)
      int tile_rows = 0;
      double mt = even;
      if (E == 1 && s.kind == LIN_320 && rounds * 256 / (nN * split) > mt) {
        const long long room = static_cast<long long>(rounds) * 256 / (nN * split);
        const long long tr = lin_ceil_div(lin_ceil_div(rows, room), 64) * 64;
        if (tr >= 192 && tr < s.tm) {
          tile_rows = static_cast<int>(tr);
          mt = static_cast<double>(lin_ceil_div(rows, tr));
        }
      }
      const double stage = s.latency + (s.full - s.latency) * (rows / (mt * s.tm));
      const double turn_overhead = s.overhead * (rounds * s.per_cu > s.resident ? rounds * s.per_cu / s.resident : 1.0);
      double us = rounds * stage * stages / split + turn_overhead;
      if (us < mem + s.overhead) us = mem + s.overhead;
      if (us < l2 + s.overhead) us = l2 + s.overhead;
      if (split > 1) us += 3 + 8.0 * split * rows * Nw / 4e6;
      if (us < best_us) {
        best_us = us;
        best = LinPlan{s.kind, split, tile_rows};
      }
    }
  }
  return best;
}

// A tile's rows and output columns, and the lanes of its workgroup.
struct LinShape {
  int rows, cols, threads;
};
constexpr LinShape lin_shape(int kind, bool f32, bool gated) {
  if (kind == LIN_32) return LinShape{32, 64, 256};
  if (kind == LIN_64) return LinShape{64, 64, 256};
  if (kind == LIN_128) return f32 ? LinShape{128, gated ? 64 : 128, 256} : LinShape{128, gated ? 128 : 256, 512};
  return LinShape{320, gated ? 128 : 256, 512};
}

// Workgroups of a launch of tiles: as many tiles of tile_rows rows of an expert and cols columns as any
// routing can need, times the parts of K, a whole number an XCD.
inline long long lin_tile_groups(int rows, int E, int N, int tile_rows, int cols, int split) {
  const long long mt = lin_ceil_div(rows, tile_rows) + (E > 1 ? (E - 1 < rows ? E - 1 : rows) : 0);
  return lin_ceil_div(mt * lin_ceil_div(N, cols) * split, kLinXcds) * kLinXcds;
}

// Whether the launches of a call stay below 2^32 work-items each, the most that one takes, and the tiles of every
// shape below the kernels' 32-bit numbers.  (The few-rows kernel's: N / 8 workgroups of 512 lanes at most.)
inline bool lin_fits(int rows, int K, int N, int E, bool f32, bool gated) {
  const long long most = (rows / 32ll + 1 + E) * (N / 32ll + 1) * 16;   // workgroups of any shape and split, but for 8
  if (most >= (1ll << 31) - 8) return false;
  if (most < (1ll << 23) - 8) return true;   // (512 lanes each; a lane of the join has 8 columns of a row)
  const LinPlan plan = lin_plan(rows, K, gated ? 2 * N : N, E, f32);
  if (plan.kind == LIN_FEW) return true;
  const LinShape s = lin_shape(plan.kind, f32, gated);
  const long long groups = lin_tile_groups(rows, E, N, plan.tile_rows > 0 ? plan.tile_rows : s.rows, s.cols, plan.split);
  const long long joined = plan.split > 1 ? static_cast<long long>(rows) * (N / 8) + 255 : 0;   // (linear_join_kernel's)
  return groups * s.threads < (1ll << 32) && joined < (1ll << 32);
}

}  // namespace moe
