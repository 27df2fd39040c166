// Balance loss of the router, the experts' counts, and the gradient of the logits
// ("EP / DeepEP explanation" page, section 4: expert loads n_e and their imbalance; "MoE part 4"
// page, section 4.2: the router's probabilities and top-k).
//
//   p_t     = softmax(z_t + bias)                                  over all E experts
//   c_s[e]  = slots (t, j) of sequence s with topk_idx[t, j] = e,  P_s[e] = mean of p_t[e]
//   L       = alpha / S * sum_s sum_e (E c_s[e] / (k T_s)) P_s[e]  T_s: counted tokens of s
//   dz_t[e] = p_t[e] (a_s[e] - sum_j p_t[j] a_s[j]),  a_s[e] = dL alpha (E c_s[e] - k T_s) / (S k T_s^2)
//             (+ g_j (dg_j - sum_i g_i dg_i) on a token's selected experts)
// The counts are piecewise constant in z, so only P carries a gradient.  a_s is written about the
// even load k T_s / E: a constant in a cancels because p sums to one, and the difference of
// counts is exact, so nearly even loads lose no digits.
//
// A token's E logits are held by a group of G lanes, W V per lane (V runs of W consecutive
// experts, W = 4 where rows keep 16-byte alignment), so each logit is read once per pass and the
// softmax never leaves registers.  Sums over tokens are taken in a fixed order: a workgroup
// covers one chunk of C consecutive tokens and writes one partial sum for each sequence that
// the chunk meets (slot chunk + sequence: along the tokens every step to the next pair raises
// one of the two, so slots are distinct and at most chunks + S - 1); a second launch adds a
// sequence's slots.  Counts are integers, added atomically in LDS: their order does not matter.
//
// Measured: N 8192, E 256, k 8: 5.0 us (8.4 MB of logits) + 6.4 us and, with the gates, 8.6 us
// backward: latencies (loads, the ticket).  N 32768, E 160, 61 sequences: 13.4 + 5.9 and 15.6 us: still
// latencies (groups of 16 lanes with three runs each, a third of the instructions a token, take 15.1
// and 14.6 us in a row of calls against 15.7 and 13.9).  With dz in three planes the backward of N 8192,
// E 256 takes 11.8 us (10 as a step of the layer).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_common.h"
#include "moe_launch.h"

namespace moe {
namespace {

constexpr int kBalThreads = 1024;   // loss: 16 waves, so that a CU's tokens in flight hide their loads
constexpr int kBalWaves = kBalThreads / kWave;
constexpr int kBalMaxChunks = 512;   // two workgroups a CU
constexpr int kBalEx = 16;    // the fewest experts of a second-launch workgroup
constexpr int kBalBatch = 8;  // partial sums a thread of it loads together
constexpr int kBwdThreads = 256;

// Butterfly reductions over groups of G lanes, every lane ending with the result, without LDS:
// within 16 lanes by DPP (lane ^ 1, lane ^ 2, then the 8- and 16-lane mirrors, whose partners hold
// equal values by then), across by gfx950's permlane swaps.  (Shuffles through LDS took about a third
// of the loss kernel's time at E = 256.)
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int G, typename F>
__device__ __forceinline__ float group_reduce(float v, F&& f) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  if constexpr (G >= 2) v = f(v, dpp_f32<0xB1>(v));
  if constexpr (G >= 4) v = f(v, dpp_f32<0x4E>(v));
  if constexpr (G >= 8) v = f(v, dpp_f32<0x141>(v));
  if constexpr (G >= 16) v = f(v, dpp_f32<0x140>(v));
  if constexpr (G >= 32) {
    const u32x2_t t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(t[0]), __uint_as_float(t[1]));
  }
  if constexpr (G >= 64) {
    const u32x2_t t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(t[0]), __uint_as_float(t[1]));
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<G>(v, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ int clamp_token(int t, int N) { return t < 0 ? 0 : (t < N ? t : N); }

// the smallest s with seq_start[s + 1] > t (S: none)
__device__ __forceinline__ int sequence_of(const int32_t* seq_start, int S, int t) {
  if (seq_start == nullptr) return 0;
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_start[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// One token's biased logits: p[v * W + w] is that of expert (v G + l) W + w (-inf past E)
template <int G, int V, int W>
__device__ __forceinline__ void load_logits(const float* zr, int E, int l, float (&p)[V * W]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = (v * G + l) * W;
    if constexpr (W == 4) {
      float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) q = *reinterpret_cast<const float4*>(zr + e);
      p[4 * v] = q.x; p[4 * v + 1] = q.y; p[4 * v + 2] = q.z; p[4 * v + 3] = q.w;
    } else {
      p[v] = e < E ? zr[e] : -INFINITY;
    }
  }
}
// the lane's experts' biases (0 without one: a sum with 0 keeps every logit)
template <int G, int V, int W>
__device__ __forceinline__ void load_bias(const float* bias, int E, int l, float (&b)[V * W]) {
#pragma unroll
  for (int i = 0; i < V * W; ++i) {
    const int e = ((i / W) * G + l) * W + i % W;
    b[i] = bias != nullptr && e < E ? bias[e] : 0.0f;
  }
}
// in place: logits plus biases to probabilities.  A row of -inf has none: all 0.
template <int G, int V, int W>
__device__ __forceinline__ void softmax_row(float (&p)[V * W], const float (&b)[V * W]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V * W; ++i) {
    p[i] += b[i];
    m = fmaxf(m, p[i]);
  }
  m = group_max<G>(m);
  if (m == -INFINITY) m = 0.0f;   // (every exponential is then 0; a NaN logit stays NaN)
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V * W; ++i) {
    // e^x = 2^(x log2 e) on the hardware exponential: within |x| + 2 roundings of fp32
    p[i] = __builtin_amdgcn_exp2f((p[i] - m) * 1.4426950408889634f);
    sum += p[i];
  }
  sum = group_sum<G>(sum);
  // (hardware reciprocal: within one ulp; a probability is two to three times as far off as with
  // correctly rounded exponentials and quotients, near 1e-7, and errors of a mean average out)
  const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
#pragma unroll
  for (int i = 0; i < V * W; ++i) p[i] *= inv;
}

struct BalArgs {
  const float* z;
  const float* bias;
  const int32_t* topk_idx;
  const int32_t* seq_start;
  const uint8_t* mask;
  int N, E, k, S, C, chunks;
  float alpha;
  float* part_p;       // [chunks + S, E]
  int32_t* part_c;     // [chunks + S, E]
  int32_t* part_t;     // [chunks + S]
  float* part_l;       // [S, expert blocks of the second launch]
  int32_t* ticket;
  float* loss;
  int32_t* counts;
  float* prob_mean;
  int32_t* tokens;
};

// SINGLE: at most one chunk of the only sequence; the totals and the loss are written here
template <int G, int V, int W, bool SINGLE>
__global__ __launch_bounds__(kBalThreads) void balance_partial_kernel(BalArgs a) {
  constexpr int kGroups = kBalThreads / G;
  __shared__ float red[kBalWaves * G * V * W];
  __shared__ int32_t hist[G * V * W];
  __shared__ int32_t n_tok;
  const int tid = threadIdx.x, l = tid % G, grp = tid / G, wave = tid / kWave;
  if (!SINGLE && blockIdx.x == 0 && tid == 0) *a.ticket = 0;   // (read by the launch after this one)
  for (int e = tid; e < G * V * W; e += kBalThreads) hist[e] = 0;
  if (tid == 0) n_tok = 0;
  float bias[V * W];
  load_bias<G, V, W>(a.bias, a.E, l, bias);
  const int t0 = blockIdx.x * a.C, t1 = t0 + a.C < a.N ? t0 + a.C : a.N;
  for (int s = SINGLE ? 0 : sequence_of(a.seq_start, a.S, t0); s < a.S; ++s) {
    int lo = t0, hi = t1;
    if (a.seq_start != nullptr) {
      const int b = clamp_token(a.seq_start[s], a.N), e = clamp_token(a.seq_start[s + 1], a.N);
      if (!SINGLE && b >= t1) break;
      lo = b > t0 ? b : t0;
      hi = e < t1 ? e : t1;
    }
    if (!SINGLE && lo >= hi) continue;   // (an empty sequence)
    __syncthreads();          // hist and n_tok are cleared, red has been read
    float acc[V * W];
#pragma unroll
    for (int i = 0; i < V * W; ++i) acc[i] = 0.0f;
    int mine = 0;
    // a token's logits and first expert id are loaded while the one before it is summed
    float next[V * W];
    int next_id = -1;
    bool next_on = false;
    auto fetch = [&](int t) __attribute__((always_inline)) {
      next_on = t < hi && (a.mask == nullptr || a.mask[t] != 0);
      if (!next_on) return;
      load_logits<G, V, W>(a.z + static_cast<size_t>(t) * a.E, a.E, l, next);
      if (l < a.k) next_id = a.topk_idx[static_cast<size_t>(t) * a.k + l];
    };
    fetch(lo + grp);
    for (int t = lo + grp; t < hi; t += kGroups) {
      float p[V * W];
#pragma unroll
      for (int i = 0; i < V * W; ++i) p[i] = next[i];
      const int id = next_id;
      const bool on = next_on;
      fetch(t + kGroups);
      if (!on) continue;
      softmax_row<G, V, W>(p, bias);
#pragma unroll
      for (int i = 0; i < V * W; ++i) acc[i] += p[i];
      if (l < a.k && static_cast<unsigned>(id) < static_cast<unsigned>(a.E)) atomicAdd(&hist[id], 1);
      for (int j = l + G; j < a.k; j += G) {
        const int e = a.topk_idx[static_cast<size_t>(t) * a.k + j];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(a.E)) atomicAdd(&hist[e], 1);
      }
      ++mine;
    }
    if (l == 0 && mine > 0) atomicAdd(&n_tok, mine);
    // a wave's groups, then the waves, each in a fixed order
#pragma unroll
    for (int i = 0; i < V * W; ++i) {
#pragma unroll
      for (int off = G; off < kWave; off <<= 1) acc[i] += __shfl_xor(acc[i], off, kWave);
      if (tid % kWave < G) red[wave * (G * V * W) + ((i / W) * G + l) * W + i % W] = acc[i];
    }
    __syncthreads();
    const size_t slot = static_cast<size_t>(blockIdx.x) + s;
    float share = 0.0f;   // (E <= kBalThreads: one expert a thread)
    if (tid < a.E) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kBalWaves; ++w) v += red[w * (G * V * W) + tid];
      if constexpr (SINGLE) {
        const float T = static_cast<float>(n_tok), mean = n_tok > 0 ? v / T : 0.0f;
        a.counts[tid] = hist[tid];
        a.prob_mean[tid] = mean;
        if (n_tok > 0)
          share = mean * (static_cast<float>(a.E) * static_cast<float>(hist[tid]) / (static_cast<float>(a.k) * T));
      } else {
        a.part_p[slot * a.E + tid] = v;
        a.part_c[slot * a.E + tid] = hist[tid];
        hist[tid] = 0;
      }
    }
    if constexpr (SINGLE) {
      share = group_sum<kWave>(share);
      __syncthreads();   // red has been read
      if (tid % kWave == 0) red[wave] = share;
      __syncthreads();
      if (tid == 0) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kBalWaves; ++w) sum += red[w];
        *a.loss = a.alpha * sum;
        *a.tokens = n_tok;
      }
    } else if (tid == 0) {
      a.part_t[slot] = n_tok;
      n_tok = 0;
    }
    if (hi == t1) break;   // (no later sequence has a token here)
  }
}

__device__ __forceinline__ int block_sum_int(int v, int32_t* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kBalWaves; ++w) v += red[w];
  return v;
}

// workgroup (`ex` experts of block x, sequence y): the chunks' partial sums, then the sequence's
// share of the loss; the last workgroup to finish adds the shares in their order.  Every
// workgroup takes one turn at the ticket, so up to 64 sequences they are kept to about 64, and
// beyond one to each sequence (610 for 61 sequences of 160 experts took 17 us).
__global__ __launch_bounds__(kBalThreads) void balance_total_kernel(BalArgs a, int ex) {
  __shared__ float rp[kBalThreads];
  __shared__ int32_t rc[kBalThreads];
  __shared__ int32_t ri[kBalWaves];
  __shared__ float share[kBalWaves];
  __shared__ int last;
  const int rows = kBalThreads / ex;   // (ex is a power of two)
  const int tid = threadIdx.x, el = tid & (ex - 1), row = tid / ex;
  const int e = blockIdx.x * ex + el, s = blockIdx.y;
  int lo = 0, hi = a.N;
  if (a.seq_start != nullptr) {
    lo = clamp_token(a.seq_start[s], a.N);
    hi = clamp_token(a.seq_start[s + 1], a.N);
  }
  const int c0 = lo < hi ? lo / a.C : 0, c1 = lo < hi ? (hi - 1) / a.C + 1 : 0;   // its chunks
  float p = 0.0f;
  int c = 0, t = 0;
  for (int i = c0 + tid; i < c1; i += kBalThreads) t += a.part_t[i + s];
  for (int i0 = c0 + row; i0 < c1; i0 += kBalBatch * rows) {
    float vp[kBalBatch];
    int vc[kBalBatch];
#pragma unroll
    for (int u = 0; u < kBalBatch; ++u) {
      const int i = i0 + u * rows;
      const size_t o = (static_cast<size_t>(i) + s) * a.E + e;
      const bool in = i < c1 && e < a.E;
      vp[u] = in ? a.part_p[o] : 0.0f;
      vc[u] = in ? a.part_c[o] : 0;
    }
#pragma unroll
    for (int u = 0; u < kBalBatch; ++u) {
      p += vp[u];
      c += vc[u];
    }
  }
  rp[tid] = p;
  rc[tid] = c;
  const int T = block_sum_int(t, ri);   // (synchronises)
  float part = 0.0f;
  if (row == 0 && e < a.E) {
    float ps = 0.0f;
    int cs = 0;
    for (int r = 0; r < rows; ++r) {
      ps += rp[r * ex + el];
      cs += rc[r * ex + el];
    }
    const float mean = T > 0 ? ps / static_cast<float>(T) : 0.0f;
    a.counts[static_cast<size_t>(s) * a.E + e] = cs;
    a.prob_mean[static_cast<size_t>(s) * a.E + e] = mean;
    if (T > 0)
      part = mean * (static_cast<float>(a.E) * static_cast<float>(cs) / (static_cast<float>(a.k) * static_cast<float>(T)));
  }
  if (tid == 0 && blockIdx.x == 0) a.tokens[s] = T;
  part = group_sum<kWave>(part);
  if (tid % kWave == 0) share[tid / kWave] = part;
  __syncthreads();
  const int n = static_cast<int>(gridDim.x * gridDim.y);
  if (tid == 0) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kBalWaves; ++w) sum += share[w];
    const int id = s * gridDim.x + blockIdx.x;
    __hip_atomic_store(a.part_l + id, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
  }
  __syncthreads();
  if (!last) return;
  float sum = 0.0f;
  for (int i = tid; i < n; i += kBalThreads)
    sum += __hip_atomic_load(a.part_l + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = group_sum<kWave>(sum);
  if (tid % kWave == 0) share[tid / kWave] = sum;
  __syncthreads();
  if (tid == 0) {
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kBalWaves; ++w) sum += share[w];
    *a.loss = a.alpha / static_cast<float>(a.S) * sum;
  }
}

struct BalBwdArgs {
  const float* z;
  const float* bias;
  const int32_t* topk_idx;
  const int32_t* seq_start;
  const uint8_t* mask;
  const int32_t* counts;
  const int32_t* tokens;
  const float* d_loss;
  const float* gate;
  const float* d_gate;
  void* dz;
  int N, E, k, S;
  int per;             // tokens of a workgroup
  float alpha;
};

// A run of n (1 or 4) values as three bf16 words each, every one the rounding of what the ones before it
// leave: 8 bits of the significand each, so that their sum is the fp32 value (down to 2^-133; a value that is not
// finite, or past bf16's largest, leaves a NaN)
template <int W>
__device__ __forceinline__ void store_planes(uint16_t* dz, size_t plane, const float* d) {
  float r[W];
#pragma unroll
  for (int i = 0; i < W; ++i) r[i] = d[i];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if constexpr (W == 4) {
      const uint2 w = make_uint2(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]));
      *reinterpret_cast<uint2*>(dz + q * plane) = w;
      r[0] -= __uint_as_float(w.x << 16);
      r[1] -= __uint_as_float(w.x & 0xFFFF0000u);
      r[2] -= __uint_as_float(w.y << 16);
      r[3] -= __uint_as_float(w.y & 0xFFFF0000u);
    } else {
      const uint16_t w = f32_to_bf16(r[0]);
      dz[q * plane] = w;
      r[0] -= bf16_to_f32(w);
    }
  }
}

// a workgroup takes `per` consecutive tokens, a group every kGroups-th of them; dz of DT
template <int G, int V, int W, int DT>
__global__ __launch_bounds__(kBwdThreads) void balance_backward_kernel(BalBwdArgs a) {
  constexpr int kGroups = kBwdThreads / G;
  const int l = threadIdx.x % G, lane = threadIdx.x % kWave;
  const float scale = a.alpha * (a.d_loss != nullptr ? *a.d_loss : 1.0f) / (static_cast<float>(a.S) * static_cast<float>(a.k));
  float bias[V * W], co[V * W];
  load_bias<G, V, W>(a.bias, a.E, l, bias);
  const long long t0 = static_cast<long long>(blockIdx.x) * a.per;
  const long long t1 = t0 + a.per < a.N ? t0 + a.per : a.N;
  int s = -1, s_hi = 0;   // the sequence whose coefficients co holds, and its end
  for (long long t = t0 + threadIdx.x / G; t < t1; t += kGroups) {
    float d[V * W];
    load_logits<G, V, W>(a.z + static_cast<size_t>(t) * a.E, a.E, l, d);
    // (slot l of the token, if it has one: its expert, gate and gate gradient)
    const size_t o = static_cast<size_t>(t) * a.k;
    int id = -1;
    float g = 0.0f, dg = 0.0f;
    if (a.gate != nullptr && l < a.k) {
      id = a.topk_idx[o + l];
      g = a.gate[o + l];
      dg = a.d_gate[o + l];
    }
    // the token's sequence, if it counts
    bool on = a.mask == nullptr || a.mask[t] != 0;
    if (s < 0 || t >= s_hi) {   // (tokens come in order: a sequence's coefficients are loaded once)
      s = sequence_of(a.seq_start, a.S, static_cast<int>(t));
      s_hi = a.N;
      if (a.seq_start != nullptr) s_hi = s < a.S ? a.seq_start[s + 1] : a.N;
      if (s < a.S) {
        // E c - k T in 64 bits, exact for every count: both products pass 2^24 with a few million tokens
        const double E = a.E, kT = static_cast<double>(a.k) * a.tokens[s];
        const float T = static_cast<float>(a.tokens[s]), f = T > 0.0f ? scale / (T * T) : 0.0f;
#pragma unroll
        for (int i = 0; i < V * W; ++i) {
          const int e = ((i / W) * G + l) * W + i % W;
          const int c = e < a.E ? a.counts[static_cast<size_t>(s) * a.E + e] : 0;
          co[i] = e < a.E ? f * static_cast<float>(fma(E, static_cast<double>(c), -kT)) : 0.0f;
        }
      }
    }
    if (a.seq_start != nullptr) on = on && s < a.S && a.seq_start[s < a.S ? s : 0] <= t;
    if (on) {
      softmax_row<G, V, W>(d, bias);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V * W; ++i) dot = fmaf(d[i], co[i], dot);
      dot = group_sum<G>(dot);
#pragma unroll
      for (int i = 0; i < V * W; ++i) d[i] *= co[i] - dot;
    } else {
#pragma unroll
      for (int i = 0; i < V * W; ++i) d[i] = 0.0f;
    }
    if (a.gate != nullptr) {
      float sum = g * dg;
      for (int j = l + G; j < a.k; j += G) sum = fmaf(a.gate[o + j], a.d_gate[o + j], sum);
      sum = group_sum<G>(sum);
      for (int j0 = 0; j0 < a.k; j0 += G) {   // (more slots than lanes only with few experts)
        if (j0 > 0) {
          id = -1;
          if (j0 + l < a.k) {
            id = a.topk_idx[o + j0 + l];
            g = a.gate[o + j0 + l];
            dg = a.d_gate[o + j0 + l];
          }
        }
        const float mine = g * (dg - sum);
        const int n = a.k - j0 < G ? a.k - j0 : G;
        for (int j = 0; j < n; ++j) {
          int idj;
          float dj;
          if constexpr (G == kWave) {
            idj = __builtin_amdgcn_readlane(id, j);
            dj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), j));
          } else {
            idj = __shfl(id, lane - l + j, kWave);
            dj = __shfl(mine, lane - l + j, kWave);
          }
#pragma unroll
          for (int i = 0; i < V * W; ++i)
            if (((i / W) * G + l) * W + i % W == idj) d[i] += dj;
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = (v * G + l) * W;
      if (e >= a.E) continue;
      const size_t o = static_cast<size_t>(t) * a.E + e;
      if constexpr (DT == MOE_BF16X3)
        store_planes<W>(reinterpret_cast<uint16_t*>(a.dz) + o, static_cast<size_t>(a.N) * a.E, d + v * W);
      else if constexpr (DT == MOE_F32 && W == 4)
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.dz) + o) =
            make_float4(d[4 * v], d[4 * v + 1], d[4 * v + 2], d[4 * v + 3]);
      else if constexpr (DT == MOE_F32)
        reinterpret_cast<float*>(a.dz)[o] = d[v];
      else if constexpr (W == 4)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.dz) + o) =
            make_uint2(pack_bf16x2(d[4 * v], d[4 * v + 1]), pack_bf16x2(d[4 * v + 2], d[4 * v + 3]));
      else
        reinterpret_cast<uint16_t*>(a.dz)[o] = f32_to_bf16(d[v]);
    }
  }
}

// lanes of a token's group for E experts, W per lane and run: the smallest power of two that
// holds them, a whole wave (and V runs) beyond 64 W
int group_lanes(int E, int W) {
  int g = W == 4 ? 2 : 8;
  while (g < kWave && g * W < E) g *= 2;
  return g;
}

// f<G, V, W>() for E experts
template <typename F>
void with_group(int E, bool vec, F&& f) {
#define MOE_GROUP(G_, V_, W_) f(std::integral_constant<int, G_>{}, std::integral_constant<int, V_>{}, std::integral_constant<int, W_>{})
  if (vec) {
    switch (group_lanes(E, 4)) {
      case 2: return MOE_GROUP(2, 1, 4);
      case 4: return MOE_GROUP(4, 1, 4);
      case 8: return MOE_GROUP(8, 1, 4);
      case 16: return MOE_GROUP(16, 1, 4);
      case 32: return MOE_GROUP(32, 1, 4);
    }
    if (E <= 256) return MOE_GROUP(64, 1, 4);
    if (E <= 512) return MOE_GROUP(64, 2, 4);
    return MOE_GROUP(64, 4, 4);
  }
  switch (group_lanes(E, 1)) {
    case 8: return MOE_GROUP(8, 1, 1);
    case 16: return MOE_GROUP(16, 1, 1);
    case 32: return MOE_GROUP(32, 1, 1);
  }
  if (E <= 64) return MOE_GROUP(64, 1, 1);
  if (E <= 128) return MOE_GROUP(64, 2, 1);
  if (E <= 256) return MOE_GROUP(64, 4, 1);
  if (E <= 512) return MOE_GROUP(64, 8, 1);
  return MOE_GROUP(64, 16, 1);
#undef MOE_GROUP
}

// tokens of a chunk: at most kBalMaxChunks chunks, and a few tokens per group so that a partial
// sum is worth its write, but no more than an even sequence's: a workgroup takes its sequences one
// after the other, about 1.5 us each (N 315, E 4, 40 sequences, both calls: one chunk 82 us, 40
// chunks 18).  The same for either alignment of z (the workspace depends on it).
int chunk_tokens(int N, int E, int S) {
  const int pass = kBalThreads / group_lanes(E, E % 4 == 0 ? 4 : 1);   // tokens the workgroup holds at a time
  const int need = N / kBalMaxChunks + (N % kBalMaxChunks != 0 ? 1 : 0);
  const int passes = (need + pass - 1) / pass;
  const int full = pass * (passes > 2 ? passes : 2), even = N > S ? (N - 1) / S + 1 : 1;
  return even >= full ? full : (even > need ? even : need);
}

struct BalLayout {
  int C, chunks;
  size_t p, c, t, l, ticket, total;   // byte offsets in the workspace
};
BalLayout balance_layout(int N, int E, int S) {
  BalLayout b;
  b.C = chunk_tokens(N, E, S);
  b.chunks = N > 0 ? (N - 1) / b.C + 1 : 0;
  const size_t slots = static_cast<size_t>(b.chunks) + S;
  b.p = 0;
  b.c = b.p + slots * E * 4;
  b.t = b.c + slots * E * 4;
  b.l = b.t + slots * 4;
  b.ticket = b.l + static_cast<size_t>(S) * ((E + kBalEx - 1) / kBalEx) * 4;
  b.total = (b.ticket + 4 + 255) & ~static_cast<size_t>(255);
  return b;
}

__global__ void balance_clear_kernel(int32_t* ticket) { *ticket = 0; }

}  // namespace

// one launch that needs no workspace
static bool balance_single(const BalLayout& b, int S) { return b.chunks <= 1 && S == 1; }

size_t balance_ws_bytes(int N, int E, int S) {
  const BalLayout b = balance_layout(N, E, S);
  return balance_single(b, S) ? 0 : b.total;
}

hipError_t launch_balance_loss(const float* z, const float* bias, const int32_t* topk_idx, int N, int E, int k,
                               const int32_t* seq_start, int S, const uint8_t* mask, float alpha, float* loss,
                               int32_t* counts, float* prob_mean, int32_t* tokens, void* ws, hipStream_t s) {
  const BalLayout b = balance_layout(N, E, S);
  uint8_t* w = static_cast<uint8_t*>(ws);
  BalArgs a = {z, bias, topk_idx, seq_start, mask, N, E, k, S, b.C, b.chunks, alpha,
               reinterpret_cast<float*>(w + b.p), reinterpret_cast<int32_t*>(w + b.c),
               reinterpret_cast<int32_t*>(w + b.t), reinterpret_cast<float*>(w + b.l),
               reinterpret_cast<int32_t*>(w + b.ticket), loss, counts, prob_mean, tokens};
  const bool vec = E % 4 == 0 && reinterpret_cast<uintptr_t>(z) % 16 == 0;
  const bool single = balance_single(b, S);
  if (single || b.chunks > 0)
    with_group(E, vec, [&](auto g, auto v, auto wd) {
      if (single)
        hipLaunchKernelGGL((balance_partial_kernel<g(), v(), wd(), true>), dim3(1), dim3(kBalThreads), 0, s, a);
      else
        hipLaunchKernelGGL((balance_partial_kernel<g(), v(), wd(), false>), dim3(b.chunks), dim3(kBalThreads), 0, s, a);
    });
  else
    hipLaunchKernelGGL(balance_clear_kernel, dim3(1), dim3(1), 0, s, a.ticket);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || single) return err;
  int ex = kBalEx;
  while (ex < E && static_cast<long long>((E + ex - 1) / ex) * S > 64) ex *= 2;
  hipLaunchKernelGGL(balance_total_kernel, dim3((E + ex - 1) / ex, S), dim3(kBalThreads), 0, s, a, ex);
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const float* z, const float* bias, const int32_t* topk_idx, int N, int E, int k,
                                        const int32_t* seq_start, int S, const uint8_t* mask, float alpha,
                                        const int32_t* counts, const int32_t* tokens, const float* d_loss,
                                        const float* gate, const float* d_gate, void* dz, int dz_dt, hipStream_t s) {
  BalBwdArgs a = {z, bias, topk_idx, seq_start, mask, counts, tokens, d_loss, gate, d_gate, dz,
                  N, E, k, S, 0, alpha};
  const bool vec = E % 4 == 0 && reinterpret_cast<uintptr_t>(z) % 16 == 0 && reinterpret_cast<uintptr_t>(dz) % 16 == 0;
  with_group(E, vec, [&](auto g, auto v, auto wd) {
    // about 2048 workgroups (8 waves a SIMD), each of whole passes
    const int pass = kBwdThreads / g();
    const int passes = ((N + pass - 1) / pass + 2047) / 2048;
    a.per = pass * passes;
    const int blocks = (N + a.per - 1) / a.per;
    if (dz_dt == MOE_F32)
      hipLaunchKernelGGL((balance_backward_kernel<g(), v(), wd(), MOE_F32>), dim3(blocks), dim3(kBwdThreads), 0, s, a);
    else if (dz_dt == MOE_BF16)
      hipLaunchKernelGGL((balance_backward_kernel<g(), v(), wd(), MOE_BF16>), dim3(blocks), dim3(kBwdThreads), 0, s, a);
    else
      hipLaunchKernelGGL((balance_backward_kernel<g(), v(), wd(), MOE_BF16X3>), dim3(blocks), dim3(kBwdThreads), 0, s, a);
  });
  return hipGetLastError();
}

}  // namespace moe
