// Balance loss of the router and its gradient (moe_balance_loss, moe_balance_loss_backward).
//
// Tokens t of sequence s (n_s of them count), scores p[t] = softmax(l[t]) or sigma(l[t]) / sum sigma(l[t]):
//   c[s,e] = number of choices of expert e,  P[s,e] = (1 / n_s) sum_t p[t,e],
//   L = coef / S' * sum_s E / (k n_s) * sum_e c[s,e] P[s,e],          S' = sequences with n_s > 0,
//   dL/dl[t,e] = w_s / n_s * p[t,e] * (c[s,e] - sum_j c[s,j] p[t,j])  [ * (1 - sigma(l[t,e])) ]  (p sums to 1),
//   w_s = coef / S' * E / (k n_s).
// The loss reads the logits once; the gradient needs the counts of all tokens, so it reads them again.
// Sums over tokens run in a fixed order (per warp, per block, then over blocks), so results repeat bit
// for bit; counts are integers.
// T = 32768, E = 256 fp32, loss and gradient: 29.4 us for 101 MB (3.4 TB/s).  Latency bounds it: a row's logits, the
// next row's on their way and the sums or counts take all 128 registers (up to 172 bytes a thread are spilled beyond 128
// experts), which leaves 16 warps an SM; an instruction issues in 45 to 51 % of the cycles, and what a warp waits for most is
// memory.  A block's 3.5 rounds of tokens take four.  T = 512: 10.6 us, two launches and their latencies.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "../../include/moe_b200.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int kWarps = 8;

struct BalanceArgs {
  int T, E, k, S, chunk, chunks, score;
  int clusters;              // the cluster kernel does the sums
  const void* logits;
  long ldl;
  const int32_t* ids;        // [T, k]
  const int32_t* offsets;    // [S + 1] or NULL (one sequence of all tokens)
  const uint8_t* mask;       // [T] or NULL
  float coef;
  // workspace: partial sums of slot chunk + sequence
  float* part_p;             // [slots][E]
  int32_t* part_c;           // [slots][E]
  int32_t* part_n;           // [slots]
  double* part_l;            // [S][ceil(E / 8)]: sums of counts * probs / n
  uint32_t* ticket;
  // results
  float* loss;
  int32_t* counts;           // [S, E]
  float* probs;              // [S, E]
  int32_t* tokens;           // [S]
  // gradient
  const float* grad_loss;
  void* grad;
  long ldg;
  int accumulate;
};

// First tokens of the sequences, inside [0, T] whatever the array holds.  Up to kStarts of them lie in shared
// memory, where a search does not pay a trip to L2 a step.
constexpr int kStarts = 1025;
struct Starts {
  const int32_t* at;                 // shared or global, NULL: one sequence of all tokens
  int S, T;
  __device__ __forceinline__ int operator[](int s) const {
    if (at == nullptr) return s == 0 ? 0 : T;
    return min(max(at[s], 0), T);
  }
  // The largest s in [-1, S] with start <= t (they ascend): the sequence of token t, or -1 / S for a token
  // before the first or behind the last one.
  __device__ __forceinline__ int of(int t) const {
    if (at == nullptr) return 0;
    int lo = -1, hi = S;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if ((*this)[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
};
// All threads call it; a barrier follows before the result is used.
__device__ __forceinline__ Starts stage_starts(const BalanceArgs& p, int32_t* smem) {
  if (p.offsets == nullptr || p.S + 1 > kStarts) return Starts{p.offsets, p.S, p.T};
  for (int i = threadIdx.x; i <= p.S; i += blockDim.x) smem[i] = p.offsets[i];
  return Starts{smem, p.S, p.T};
}

// How a token's E logits lie over lanes: LPR lanes to a row (32 / LPR rows to a warp), J logits to a lane; V
// consecutive ones load together.  Eight lanes with 32 logits each make 256 of them: a sum or maximum over the
// row is three shuffles for four rows, where a row to a warp takes five for each.
template <class T, int LPR, int J, int V>
struct RowMap {
  static constexpr int kRows = 32 / LPR;
  static __device__ __forceinline__ int expert(int lane, int j) {
    return V == 1 ? lane % LPR + LPR * j : V * (lane % LPR) + j % V + V * LPR * (j / V);
  }
  static __device__ __forceinline__ void load(const T* row, int E, int lane, bool live, float (&l)[J]) {
#pragma unroll
    for (int j = 0; j < J; j += V) {
      const int e = expert(lane, j);
      if constexpr (V == 4 && sizeof(T) == 4) {
        const float4 v = live && e < E ? *reinterpret_cast<const float4*>(row + e)
                                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        l[j] = v.x;
        l[j + 1] = v.y;
        l[j + 2] = v.z;
        l[j + 3] = v.w;
      } else if constexpr (V == 4) {
        const uint2 v = live && e < E ? *reinterpret_cast<const uint2*>(row + e) : make_uint2(0xFF80FF80u, 0xFF80FF80u);
        l[j] = __uint_as_float(v.x << 16);
        l[j + 1] = __uint_as_float(v.x & 0xFFFF0000u);
        l[j + 2] = __uint_as_float(v.y << 16);
        l[j + 3] = __uint_as_float(v.y & 0xFFFF0000u);
      } else if constexpr (sizeof(T) == 4) {
        l[j] = live && e < E ? row[e] : -INFINITY;
      } else {
        l[j] = live && e < E ? __bfloat162float(row[e]) : -INFINITY;
      }
    }
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(l - m) as 2^(l log2(e) - m log2(e)), one FMA: the rounding of m log2(e) is common to the row and cancels in the
// quotient, that of the result is at most that of l - m.  It has to be small for that: up to |m| = 1e6 it is at most
// 1/16 in the exponent, at 5e9 it takes every term to zero or infinity.  Rows above take the difference first.
constexpr float kFusedLogit = 1e6f;
template <int LPR, int J>
__device__ __forceinline__ void softmax_row(float (&l)[J]) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < J; ++j) m = fmaxf(m, l[j]);
  m = row_max<LPR>(m);
  float z = 0.f;
  if (__any_sync(0xffffffffu, fabsf(m) > kFusedLogit)) {   // far from zero, or nothing is finite
#pragma unroll
    for (int j = 0; j < J; ++j) {
      l[j] = l[j] == -INFINITY ? 0.f : expf(l[j] - m);
      z += l[j];
    }
  } else {
    const float ml = -m * kLog2e;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      l[j] = ex2(fmaf(l[j], kLog2e, ml));
      z += l[j];
    }
  }
  z = row_sum<LPR>(z);
  const float r = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
  for (int j = 0; j < J; ++j) l[j] *= r;
}

// Sigmoid scores from one exponential each: with s = min(largest logit of the row, 0), a = e^s and y = e^(s - l),
//   w = 1 / (a + y) = sigma(l) e^-s,   p = w / sum w,   sigma = a w,   1 - sigma = y w.
// Some w of a row is at least 1/2, however low its logits are, and 1 - sigma needs no difference where it is small.
// l: logits -> y, returns a.  A row without a finite logit, and a token that does not count (its logits read
// as -inf), have y = infinity throughout: zero scores.  All lanes of the warp call it.  Where every row has a logit
// above zero, s is 0 without a reduction.
template <int LPR, int J>
__device__ __forceinline__ float sigmoid_row(float (&l)[J]) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < J; ++j) m = fmaxf(m, l[j]);
  const uint32_t above = __ballot_sync(0xffffffffu, m >= 0.f), row = LPR == 32 ? 0xffffffffu : (1u << LPR) - 1;
  bool low = false;
#pragma unroll
  for (int i = 0; i < 32; i += LPR) low |= (above >> i & row) == 0;
  float s = 0.f;
  if (low) {                           // the whole warp
    m = row_max<LPR>(m);
    s = m == -INFINITY ? 0.f : fminf(m, 0.f);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) l[j] = ex2((s - l[j]) * kLog2e);
  return ex2(s * kLog2e);
}

// l: a token's logits -> its scores.  A row whose logits are all -inf has zero scores, and so has a token that does
// not count.  All lanes of the warp call it.
template <int LPR, int J>
__device__ __forceinline__ void scores(int score, float (&l)[J]) {
  if (score != MOE_SCORE_SIGMOID) {
    softmax_row<LPR, J>(l);
    return;
  }
  const float a = sigmoid_row<LPR, J>(l);
  float z = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    l[j] = rcp(a + l[j]);
    z += l[j];
  }
  z = row_sum<LPR>(z);
  const float r = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
  for (int j = 0; j < J; ++j) l[j] *= r;
}

// l: a token's logits -> its scores, with sigmoid scores times 1 - sigma; returns sum_j c_j p_j.
template <int LPR, int J>
__device__ __forceinline__ float weighted_scores(int score, const float (&c)[J], float (&l)[J]) {
  float mean = 0.f;
  if (score != MOE_SCORE_SIGMOID) {
    softmax_row<LPR, J>(l);
#pragma unroll
    for (int j = 0; j < J; ++j) mean = fmaf(c[j], l[j], mean);
    return row_sum<LPR>(mean);
  }
  const float a = sigmoid_row<LPR, J>(l);
  float z = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float w = rcp(a + l[j]);
    z += w;
    mean = fmaf(c[j], w, mean);
  }
  z = row_sum<LPR>(z);
  mean = row_sum<LPR>(mean);
  const float r = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float w = rcp(a + l[j]);
    l[j] = fminf(l[j], FLT_MAX) * w * (w * r);             // (1 - sigma) p; w is 0 where y is infinite
  }
  return mean * r;
}

// Sums over tokens [a, b) by one block: sum_s[warp][E] of scores, cnt_s[E] of choices, n_s tokens that count.  The
// next round's rows are on their way while one is computed.  A barrier stands at the end.
template <class T, int LPR, int J, int V, int U>
__device__ __forceinline__ void sum_tokens(const BalanceArgs& p, int a, int b, float* sum_s, int* cnt_s, int& n_s) {
  using Map = RowMap<T, LPR, J, V>;
  constexpr int kStep = kWarps * Map::kRows;                // tokens of the block a round of one row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kWarps * 32) cnt_s[e] = 0;
  if (threadIdx.x == 0) n_s = 0;
  float acc[J], l[U][J];
  bool live[U];
  int n = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) acc[j] = 0.f;
  auto load = [&](int r0, float (&x)[U][J], bool (&on)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = r0 + u * kStep + lane / LPR;
      on[u] = t < b && (p.mask == nullptr || p.mask[t] != 0);
      Map::load(static_cast<const T*>(p.logits) + (long)t * p.ldl, p.E, lane, on[u], x[u]);
    }
  };
  int r0 = a + warp * Map::kRows;
  if (r0 < b) load(r0, l, live);
  // choices of these tokens
  __syncthreads();
  const int32_t* ids = p.ids + (long)a * p.k;
  for (int i = threadIdx.x; i < (b - a) * p.k; i += kWarps * 32) {
    const int e = ids[i];
    if ((unsigned)e < (unsigned)p.E && (p.mask == nullptr || p.mask[a + i / p.k] != 0)) atomicAdd(&cnt_s[e], 1);
  }
  for (; r0 < b; r0 += U * kStep) {
    float next[U][J];
    bool on[U];
    load(r0 + U * kStep, next, on);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      n += live[u] && lane % LPR == 0;
      if (u == 0 || __any_sync(0xffffffffu, live[u])) {
        scores<LPR, J>(p.score, l[u]);
#pragma unroll
        for (int j = 0; j < J; ++j) acc[j] += l[u][j];
      }
#pragma unroll
      for (int j = 0; j < J; ++j) l[u][j] = next[u][j];
      live[u] = on[u];
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    const int e = Map::expert(lane, j);
    if (lane < LPR && e < p.E) sum_s[warp * p.E + e] = acc[j];
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0 && n > 0) atomicAdd(&n_s, n);
  __syncthreads();
}

__device__ __forceinline__ float warps_sum(const BalanceArgs& p, const float* sum_s, int e) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += sum_s[w * p.E + e];
  return v;
}

// Partial sums of one chunk of tokens, a slot per sequence that the chunk touches: (chunk, sequence)
// pairs ascend in both, so chunk + sequence numbers them without two sharing a number.
template <class T, int LPR, int J, int V, int U>
__global__ void __launch_bounds__(kWarps * 32, 2) balance_part_kernel(const BalanceArgs p) {
  extern __shared__ float sm[];
  float* sum_s = sm;                                        // [kWarps][E]
  int* cnt_s = reinterpret_cast<int*>(sm + kWarps * p.E);   // [E]
  __shared__ int n_s;
  __shared__ int32_t starts_s[kStarts];
  griddep_wait();
  griddep_launch_dependents();         // the join kernel's blocks wait on the device
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  const Starts start = stage_starts(p, starts_s);
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
  for (int s = max(0, start.of(t0)); s < p.S; ++s) {
    const int a = max(t0, start[s]), b = min(t1, start[s + 1]);
    if (start[s] >= t1) break;
    if (a >= b) continue;
    sum_tokens<T, LPR, J, V, U>(p, a, b, sum_s, cnt_s, n_s);
    const long slot = blockIdx.x + s;
    for (int e = threadIdx.x; e < p.E; e += kWarps * 32) {
      p.part_p[slot * p.E + e] = warps_sum(p, sum_s, e);
      p.part_c[slot * p.E + e] = cnt_s[e];
    }
    if (threadIdx.x == 0) p.part_n[slot] = n_s;
    __syncthreads();
  }
}

// Few tokens: the blocks of a cluster have a share of a sequence's tokens each, then of the experts, whose sums they
// add up in rank order through distributed shared memory.  One launch instead of two for one sequence.
constexpr int kCluster = 8;
constexpr int kClusterRounds = 4;      // rounds of rows (0.9 us each) a block of the cluster takes at most
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
template <class T, int LPR, int J, int V, int U>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kWarps * 32, 2)
    balance_cluster_kernel(const BalanceArgs p) {
  extern __shared__ float sm[];
  float* sum_s = sm;
  int* cnt_s = reinterpret_cast<int*>(sm + kWarps * p.E);
  __shared__ int n_s;
  __shared__ double part_s[kCluster];
  __shared__ double warp_s[kWarps];
  griddep_wait();
  griddep_launch_dependents();         // the total's block waits on the device
  const int rank = blockIdx.x % kCluster, s = blockIdx.x / kCluster, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Starts start{p.offsets, p.S, p.T};   // one look each
  const int first = start[s], len = max(0, start[s + 1] - first), chunk = (len + kCluster - 1) / kCluster;
  const int a = first + min(len, rank * chunk), b = first + min(len, (rank + 1) * chunk);
  sum_tokens<T, LPR, J, V, U>(p, a, b, sum_s, cnt_s, n_s);
  for (int e = threadIdx.x; e < p.E; e += kWarps * 32) sum_s[e] = warps_sum(p, sum_s, e);   // column e is this thread's
  __syncthreads();
  cluster_sync();
  int n = 0;
#pragma unroll
  for (int r = 0; r < kCluster; ++r) n += (int)ld_cluster(mapa_shared(&n_s, r));
  const float inv = n > 0 ? (float)n : 1.f;
  double v = 0.0;
  for (int e = rank + kCluster * threadIdx.x; e < p.E; e += kCluster * kWarps * 32) {
    float sum = 0.f;
    int c = 0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
      sum += __uint_as_float(ld_cluster(mapa_shared(sum_s + e, r)));
      c += (int)ld_cluster(mapa_shared(cnt_s + e, r));
    }
    const float mean = n > 0 ? sum / inv : 0.f;
    p.counts[(long)s * p.E + e] = c;
    p.probs[(long)s * p.E + e] = mean;
    v += (double)c * (double)mean;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) warp_s[warp] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += warp_s[w];
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(mapa_shared(part_s + rank, 0)), "d"(v) : "memory");
  }
  __syncthreads();
  cluster_sync();                      // no block leaves while another reads its sums
  if (rank == 0 && threadIdx.x == 0) {
    v = 0.0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) v += part_s[r];
    p.tokens[s] = n;
    if (p.S > 1) p.part_l[s] = n > 0 ? v / (double)n : 0.0;
    if (p.S == 1) *p.loss = n > 0 ? (float)(v * (double)p.coef * (double)p.E / ((double)p.k * (double)n)) : 0.f;
  }
}

// The loss from n terms of the sequences, in 64 bits and a fixed order, by the threads of one block of kTotal warps.
constexpr int kTotal = 8;
__device__ __forceinline__ void write_total(const BalanceArgs& p, int n) {
  __shared__ double v_s[kTotal];
  __shared__ int live_s[kTotal];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double v = 0.0;
  int live = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kTotal * 32) v += __ldcg(p.part_l + i);
#pragma unroll 4
  for (int i = threadIdx.x; i < p.S; i += kTotal * 32) live += __ldcg(p.tokens + i) > 0;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  live = __reduce_add_sync(0xffffffffu, live);
  if (lane == 0) {
    v_s[warp] = v;
    live_s[warp] = live;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.0;
    live = 0;
#pragma unroll
    for (int w = 0; w < kTotal; ++w) {
      v += v_s[w];
      live += live_s[w];
    }
    *p.loss = live > 0 ? (float)(v * (double)p.coef * (double)p.E / ((double)p.k * (double)live)) : 0.f;
  }
}
__global__ void __launch_bounds__(kTotal * 32) balance_total_kernel(const BalanceArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  write_total(p, p.S);
}

// One block per (sequence, 8 experts): the slots of the sequence, any number of them, added up in order, every 32nd by
// one thread.  Each addition's rounding is carried to the next one (Kahan), so that the number of slots does not count;
// in 64 bits, and one after the other at the end, 1.4 us more at 293 slots.
// The last block of the grid adds up the loss.
constexpr int kJoin = 32;
static_assert(kJoin * 8 == kTotal * 32, "the join kernel's last block writes the total");
__global__ void __launch_bounds__(kJoin * 8) balance_join_kernel(const BalanceArgs p) {
  __shared__ float fp[kJoin][8];
  __shared__ int fc[kJoin][8];
  __shared__ int fn[kJoin];
  __shared__ bool last;
  griddep_wait();
  griddep_launch_dependents();
  const int x = threadIdx.x & 7, w = threadIdx.x >> 3;
  const int s = blockIdx.x, e = blockIdx.y * 8 + x;
  const Starts start{p.offsets, p.S, p.T};
  const int a = start[s], b = start[s + 1];
  const int c0 = a / p.chunk, c1 = b > a ? (b - 1) / p.chunk + 1 : c0;   // chunks of the sequence
  float vp = 0.f, lost = 0.f;
  int vc = 0, vn = 0;
#pragma unroll 8
  for (int c = c0 + w; c < c1; c += kJoin) {
    const long slot = c + s;
    const float x = (e < p.E ? p.part_p[slot * p.E + e] : 0.f) - lost, sum = vp + x;
    vc += e < p.E ? p.part_c[slot * p.E + e] : 0;
    lost = (sum - vp) - x;
    vp = sum;
    vn += p.part_n[slot];
  }
  fp[w][x] = vp;
  fc[w][x] = vc;
  if (x == 0) fn[w] = vn;
  __syncthreads();
  if (threadIdx.x < 32) {              // lanes 8 and up repeat the first ones' experts
    float sums[kJoin];                 // in pairs, in pairs of pairs, ...
    vc = vn = 0;
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      sums[i] = fp[i][x];
      vc += fc[i][x];
      vn += fn[i];
    }
#pragma unroll
    for (int o = kJoin / 2; o >= 1; o /= 2)
#pragma unroll
      for (int i = 0; i < o; ++i) sums[i] += sums[i + o];
    vp = sums[0];
    const float mean = vn > 0 ? vp / (float)vn : 0.f;
    if (w == 0 && e < p.E) {
      p.counts[(long)s * p.E + e] = vc;
      p.probs[(long)s * p.E + e] = mean;
    }
    double r = e < p.E && vn > 0 ? (double)vc * (double)mean / (double)vn : 0.0;
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if (threadIdx.x == 0) {
      p.part_l[(long)s * gridDim.y + blockIdx.y] = r;
      if (blockIdx.y == 0) p.tokens[s] = vn;
      __threadfence();
      last = atomicAdd(p.ticket, 1u) == gridDim.x * gridDim.y - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!last) return;
  write_total(p, gridDim.x * gridDim.y);
}

// Tokens outside every sequence and masked tokens get zeros (or stay, accumulating).
template <class T, int LPR, int J, int V, int U>
__global__ void __launch_bounds__(kWarps * 32, 2) balance_grad_kernel(const BalanceArgs p) {
  using Map = RowMap<T, LPR, J, V>;
  __shared__ int live_s;
  __shared__ int32_t starts_s[kStarts];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Starts start = stage_starts(p, starts_s);
  const float grad_loss = *p.grad_loss;
  int live = 1;                        // sequences with tokens that count
  if (p.offsets != nullptr) {
    int alive = 0;
    for (int s = threadIdx.x; s < p.S; s += kWarps * 32) alive += p.tokens[s] > 0;
    if (threadIdx.x == 0) live_s = 0;
    __syncthreads();
    if (alive) atomicAdd(&live_s, alive);
    __syncthreads();
    live = max(1, live_s);
  }
  const int step = gridDim.x * kWarps * Map::kRows;
  int have = -1;                       // the sequence that c and g are of
  float c[J], g = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) c[j] = 0.f;
  float l[U][J];
  int seq[U];                          // -1: the token does not count
  auto load = [&](int r0, float (&x)[U][J], int (&of)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = r0 + u * step + lane / LPR;
      of[u] = -1;
      if (t < p.T && (p.mask == nullptr || p.mask[t] != 0)) {
        const int s = start.of(t);
        if (s >= 0 && s < p.S && t < start[s + 1]) of[u] = s;
      }
      Map::load(static_cast<const T*>(p.logits) + (long)t * p.ldl, p.E, lane, of[u] >= 0, x[u]);
    }
  };
  int r0 = (blockIdx.x * kWarps + warp) * Map::kRows;
  if (r0 < p.T) load(r0, l, seq);
  for (; r0 < p.T; r0 += U * step) {
    float next[U][J];                  // on their way while these are computed
    int of[U];
    load(r0 + U * step, next, of);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = r0 + u * step + lane / LPR;
      if (u > 0 && r0 + u * step >= p.T) break;            // the whole warp
      if (seq[u] >= 0 && seq[u] != have) {
        have = seq[u];
        // counts above the least one: the scores sum to 1, so a constant changes nothing, and what is subtracted
        // below is no larger than the counts themselves (equal counts: exactly zero)
        const int32_t* cs = p.counts + (long)have * p.E;
        const uint32_t row_lanes = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1) << (lane & ~(LPR - 1));
        int least = INT32_MAX;           // of a first reading: kept, the counts would not fit the registers
#pragma unroll 16
        for (int e = lane % LPR; e < p.E; e += LPR) least = min(least, cs[e]);
        least = __reduce_min_sync(row_lanes, least);       // the row's lanes are here together
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int e = Map::expert(lane, j);
          c[j] = e < p.E ? (float)(cs[e] - least) : 0.f;
        }
        const float n = (float)max(1, p.tokens[have]);
        g = grad_loss * p.coef * (float)p.E / ((float)p.k * (float)live) / n / n;
      }
      const float mean = weighted_scores<LPR, J>(p.score, c, l[u]);
      const bool write = t < p.T && (seq[u] >= 0 || !p.accumulate);
      T* out = static_cast<T*>(p.grad) + (long)t * p.ldg;
#pragma unroll
      for (int j = 0; j < J; j += V) {
        float d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          d[v] = g * l[u][j + v] * (c[j + v] - mean);
          if (seq[u] < 0) d[v] = 0.f;
        }
        const int e = Map::expert(lane, j);
        if (e >= p.E || !write) continue;
        if constexpr (V == 4) {
          if constexpr (sizeof(T) == 4) {
            float4* o = reinterpret_cast<float4*>(out + e);
            if (p.accumulate) {
              const float4 x = *o;
              *o = make_float4(x.x + d[0], x.y + d[1], x.z + d[2], x.w + d[3]);
            } else {
              *o = make_float4(d[0], d[1], d[2], d[3]);
            }
          } else {
            uint2* o = reinterpret_cast<uint2*>(out + e);
            if (p.accumulate) {
              const uint2 x = *o;
              d[0] += __uint_as_float(x.x << 16);
              d[1] += __uint_as_float(x.x & 0xFFFF0000u);
              d[2] += __uint_as_float(x.y << 16);
              d[3] += __uint_as_float(x.y & 0xFFFF0000u);
            }
            __nv_bfloat162 h[2] = {__floats2bfloat162_rn(d[0], d[1]), __floats2bfloat162_rn(d[2], d[3])};
            *o = *reinterpret_cast<const uint2*>(h);
          }
        } else if constexpr (sizeof(T) == 4) {
          out[e] = p.accumulate ? out[e] + d[0] : d[0];
        } else {
          out[e] = __float2bfloat16_rn(p.accumulate ? __bfloat162float(out[e]) + d[0] : d[0]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      seq[u] = of[u];
#pragma unroll
      for (int j = 0; j < J; ++j) l[u][j] = next[u][j];
    }
  }
}

// ------------------------------------------------------------------ host
size_t r256(size_t b) { return (b + 255) & ~size_t(255); }

struct Layout {
  int chunk, chunks;
  size_t part_p, part_c, part_n, part_l, ticket, total;
};

// About two blocks per SM (with four rows of 1 KB to a warp, 64 KB of logits in flight an SM), and a round of
// all warps at least.  At most 4096 tokens: a lane adds 128 scores of an expert then (E > 256: 256, E > 512: 512), and
// additions of like scores all round the same way, so that a chain is off by up to its length times 2^-24.  A block of
// 4096 tokens runs for about 100 us, beside which its start costs nothing.
constexpr int kChunk = 4096;
Layout layout(int T, int E, int S) {
  Layout L;
  const int chunk = ((T + 2 * 148 - 1) / (2 * 148) + 15) / 16 * 16;
  L.chunk = chunk < 32 ? 32 : chunk > kChunk ? kChunk : chunk;
  L.chunks = (T + L.chunk - 1) / L.chunk;
  const size_t slots = (size_t)L.chunks + (size_t)S;
  L.part_p = 0;
  L.part_c = L.part_p + r256(slots * E * 4);
  L.part_n = L.part_c + r256(slots * E * 4);
  L.part_l = L.part_n + r256(slots * 4);
  L.ticket = L.part_l + r256((size_t)S * ((E + 7) / 8) * 8);
  L.total = L.ticket + 256;
  return L;
}

bool shape_ok(int T, int E, int k, int S) {
  return T >= 0 && T <= (1 << 30) && E >= 1 && E <= 1024 && k >= 1 && k <= 16 && k <= E && S >= 1 && S <= (1 << 20);
}
bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <class T, int LPR, int J, int V, int U>
cudaError_t launch_as(BalanceArgs& a, bool grad, cudaStream_t s) {
  const int round = kWarps * 32 / LPR * U;                  // tokens of a block a round
  if (grad) {
    const int need = (a.T + kWarps * 32 / LPR - 1) / (kWarps * 32 / LPR);
    return launch_dependent(balance_grad_kernel<T, LPR, J, V, U>, dim3(need < 2 * 148 ? need : 2 * 148), kWarps * 32, 0, 1, s,
                            a);
  }
  const size_t smem = (size_t)(kWarps + 1) * a.E * 4;
  // One sequence: up to the rounds at which two launches, on all SMs, are as fast (T = 512: 7.3 us; 2048: 12.7, two
  // launches 8.5).  Several: a block of the two
  // launches takes about 4 us for each sequence of its chunk, one after the other; clusters take 5 us and 0.135 us
  // for each sequence over what fits the SMs (T = 16, S = 57: 79 us by chunks; T = 8191, S = 13: 22 us by chunks, 25
  // by clusters; 22.5 the whole step).
  a.clusters = a.S == 1 ? a.T <= kCluster * round * kClusterRounds
                        : 4.0 * a.chunk * a.S / a.T > 5.0 + 0.135 * a.S;
  return a.clusters
             ? launch_dependent(balance_cluster_kernel<T, LPR, J, V, U>, dim3(a.S * kCluster), kWarps * 32, smem, 1, s, a)
             : launch_dependent(balance_part_kernel<T, LPR, J, V, U>, dim3(a.chunks), kWarps * 32, smem, 1, s, a);
}
// vec: rows and pitches of whole groups of four logits
template <class T>
cudaError_t launch_any(BalanceArgs& a, bool vec, bool grad, cudaStream_t s) {
  if (a.E <= 8) return launch_as<T, 8, 1, 1, 4>(a, grad, s);
  if (a.E <= 32) return vec ? launch_as<T, 8, 4, 4, 4>(a, grad, s) : launch_as<T, 8, 4, 1, 4>(a, grad, s);
  if (a.E <= 64) return vec ? launch_as<T, 8, 8, 4, 2>(a, grad, s) : launch_as<T, 8, 8, 1, 2>(a, grad, s);
  if (a.E <= 128) return vec ? launch_as<T, 8, 16, 4, 2>(a, grad, s) : launch_as<T, 8, 16, 1, 2>(a, grad, s);
  if (a.E <= 256) return vec ? launch_as<T, 8, 32, 4, 1>(a, grad, s) : launch_as<T, 8, 32, 1, 1>(a, grad, s);
  if (a.E <= 512) return vec ? launch_as<T, 16, 32, 4, 1>(a, grad, s) : launch_as<T, 16, 32, 1, 1>(a, grad, s);
  return vec ? launch_as<T, 32, 32, 4, 1>(a, grad, s) : launch_as<T, 32, 32, 1, 1>(a, grad, s);
}
bool rows_of_four(const void* p, long long ld, int rows, int E, size_t size) {
  return E % 4 == 0 && aligned(p, 4 * size) && (rows <= 1 || ld % 4 == 0);
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(int T, int E, int S) {
  return shape_ok(T, E, 1, S) ? layout(T, E, S).total : 0;
}

int moe_balance_loss(int T, int E, int k, int S, const void* logits, long long ldl, int logits_type,
                     const int32_t* topk_ids, const int32_t* offsets, const uint8_t* mask, int score, float coef,
                     float* loss, int32_t* counts, float* probs, int32_t* tokens, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!shape_ok(T, E, k, S)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((logits_type != MOE_TYPE_FP32 && logits_type != MOE_TYPE_BF16) ||
      (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || !std::isfinite(coef))
    return MOE_ERR_INVALID_ARG;
  if ((T > 0 && (!aligned(logits, logits_type == MOE_TYPE_FP32 ? 4 : 2) || !aligned(topk_ids, 4))) ||
      (T > 1 && ldl < E) || (offsets == nullptr ? S != 1 : !aligned(offsets, 4)) || !aligned(loss, 4) || !aligned(counts, 4) ||
      !aligned(probs, 4) || !aligned(tokens, 4))
    return MOE_ERR_INVALID_ARG;
  const Layout L = layout(T, E, S);
  if (!aligned(workspace, 256) || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(loss, 0, 4, s) == cudaSuccess &&
                   cudaMemsetAsync(counts, 0, (size_t)S * E * 4, s) == cudaSuccess &&
                   cudaMemsetAsync(probs, 0, (size_t)S * E * 4, s) == cudaSuccess &&
                   cudaMemsetAsync(tokens, 0, (size_t)S * 4, s) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  BalanceArgs a{};
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.chunk = L.chunk;
  a.chunks = L.chunks;
  a.logits = logits;
  a.ldl = ldl;
  a.ids = topk_ids;
  a.offsets = offsets;
  a.mask = mask;
  a.coef = coef;
  a.score = score;
  a.part_p = reinterpret_cast<float*>(ws + L.part_p);
  a.part_c = reinterpret_cast<int32_t*>(ws + L.part_c);
  a.part_n = reinterpret_cast<int32_t*>(ws + L.part_n);
  a.part_l = reinterpret_cast<double*>(ws + L.part_l);
  a.ticket = reinterpret_cast<uint32_t*>(ws + L.ticket);
  a.loss = loss;
  a.counts = counts;
  a.probs = probs;
  a.tokens = tokens;
  const bool vec = rows_of_four(logits, ldl, T, E, logits_type == MOE_TYPE_FP32 ? 4 : 2);
  cudaError_t e = logits_type == MOE_TYPE_FP32 ? launch_any<float>(a, vec, false, s)
                                               : launch_any<__nv_bfloat16>(a, vec, false, s);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (a.clusters && S == 1) return MOE_OK;
  e = launch_dependent(a.clusters ? balance_total_kernel : balance_join_kernel, a.clusters ? dim3(1) : dim3(S, (E + 7) / 8),
                       kJoin * 8, 0, 1, s, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_balance_loss_backward(int T, int E, int k, int S, const float* grad_loss, const void* logits, long long ldl,
                              int logits_type, const int32_t* counts, const int32_t* tokens, const int32_t* offsets,
                              const uint8_t* mask, int score, float coef, void* grad_logits, long long ldg,
                              int accumulate, void* stream) {
  if (!shape_ok(T, E, k, S)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t es = logits_type == MOE_TYPE_FP32 ? 4 : 2;
  if ((logits_type != MOE_TYPE_FP32 && logits_type != MOE_TYPE_BF16) ||
      (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || !std::isfinite(coef))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!aligned(grad_loss, 4) || !aligned(logits, es) || (T > 1 && (ldl < E || ldg < E)) || !aligned(counts, 4) ||
      !aligned(tokens, 4) || (offsets == nullptr ? S != 1 : !aligned(offsets, 4)) || !aligned(grad_logits, es))
    return MOE_ERR_INVALID_ARG;
  BalanceArgs a{};
  a.T = T;
  a.E = E;
  a.k = k;
  a.S = S;
  a.logits = logits;
  a.ldl = ldl;
  a.offsets = offsets;
  a.mask = mask;
  a.coef = coef;
  a.score = score;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.grad_loss = grad_loss;
  a.grad = grad_logits;
  a.ldg = ldg;
  a.accumulate = accumulate != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = rows_of_four(logits, ldl, T, E, es) && rows_of_four(grad_logits, ldg, T, E, es);
  cudaError_t e = logits_type == MOE_TYPE_FP32 ? launch_any<float>(a, vec, true, s)
                                               : launch_any<__nv_bfloat16>(a, vec, true, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
