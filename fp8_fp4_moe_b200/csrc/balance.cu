// Balance loss of the router and its gradient (moe_balance_loss, moe_balance_loss_backward).
//
// Tokens t of sequence s (n_s of them count), scores p[t] = softmax(l[t]) or sigma(l[t]) / sum sigma(l[t]):
//   c[s,e] = number of choices of expert e,  P[s,e] = (1 / n_s) sum_t p[t,e],
//   L = coef / S' * sum_s E / (k n_s) * sum_e c[s,e] P[s,e],          S' = sequences with n_s > 0,
//   dL/dl[t,e] = w_s / n_s * p[t,e] * (c[s,e] - sum_j c[s,j] p[t,j])  [ * (1 - sigma(l[t,e])) ],
//   w_s = coef / S' * E / (k n_s).
// The loss reads the logits once; the gradient needs the counts of all tokens, so it reads them again.
// Sums over tokens run in a fixed order (per warp, per block, then over blocks), so results repeat bit
// for bit; counts are integers.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe_b200.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int kWarps = 8;

struct BalanceArgs {
  int T, E, k, S, chunk, chunks;
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

// First token of sequence s (0..S), inside [0, T] whatever the array holds.
__device__ __forceinline__ int seq_start(const BalanceArgs& p, int s) {
  if (p.offsets == nullptr) return s == 0 ? 0 : p.T;
  return min(max(p.offsets[s], 0), p.T);
}
// The largest s in [-1, S] with seq_start(s) <= t (offsets ascend): the sequence of token t, or -1 / S
// for a token before the first or behind the last one.
__device__ __forceinline__ int seq_of(const BalanceArgs& p, int t) {
  if (p.offsets == nullptr) return 0;
  int lo = -1, hi = p.S;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (seq_start(p, mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <class T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <int J>
__device__ __forceinline__ void softmax_row(float (&l)[J]) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < J; ++j) m = fmaxf(m, l[j]);
  m = warp_max(m);
  float z = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    l[j] = l[j] == -INFINITY ? 0.f : expf(l[j] - m);
    z += l[j];
  }
  z = warp_sum(z);
  const float r = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
  for (int j = 0; j < J; ++j) l[j] *= r;
}

// Scores of one token: lane holds experts lane + 32 j.  sg = sigma(l) (sigmoid scores).  A row whose
// logits are all -inf has zero scores.
template <int J, bool SIG>
__device__ __forceinline__ void scores(float (&l)[J], float (&sg)[J]) {
  if constexpr (SIG) {
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      sg[j] = 1.f / (1.f + expf(-l[j]));
      z += sg[j];
    }
    z = warp_sum(z);
    if (z < 1e-30f) {                  // every sigma underflows: the same scores from their logarithms
#pragma unroll
      for (int j = 0; j < J; ++j) l[j] = fminf(l[j], 0.f) - log1pf(expf(-fabsf(l[j])));
      softmax_row<J>(l);
      return;
    }
    const float r = 1.f / z;
#pragma unroll
    for (int j = 0; j < J; ++j) l[j] = sg[j] * r;
  } else {
    softmax_row<J>(l);
  }
}

template <class T, int J>
__device__ __forceinline__ void load_row(const BalanceArgs& p, int t, int lane, float (&l)[J]) {
  const T* row = static_cast<const T*>(p.logits) + (long)t * p.ldl;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < p.E ? load1<T>(row + e) : -INFINITY;
  }
}

// Partial sums of one chunk of tokens, a slot per sequence that the chunk touches: (chunk, sequence)
// pairs ascend in both, so chunk + sequence numbers them without gaps being shared.
template <class T, int J, bool SIG>
__global__ void __launch_bounds__(kWarps * 32) balance_part_kernel(const BalanceArgs p) {
  extern __shared__ float sm[];
  float* sum_s = sm;                                        // [kWarps][E]
  int* cnt_s = reinterpret_cast<int*>(sm + kWarps * p.E);   // [E]
  __shared__ int n_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
  int s = max(0, seq_of(p, t0));
  for (; s < p.S; ++s) {
    const int a = max(t0, seq_start(p, s)), b = min(t1, seq_start(p, s + 1));
    if (seq_start(p, s) >= t1) break;
    if (a >= b) continue;
    for (int e = threadIdx.x; e < p.E; e += kWarps * 32) cnt_s[e] = 0;
    if (threadIdx.x == 0) n_s = 0;
    __syncthreads();
    float acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = 0.f;
    int n = 0;
    for (int t = a + warp; t < b; t += kWarps) {
      if (p.mask != nullptr && p.mask[t] == 0) continue;
      ++n;
      float l[J], sg[J];
      load_row<T, J>(p, t, lane, l);
      for (int i = lane; i < p.k; i += 32) {
        const int e = p.ids[(long)t * p.k + i];
        if ((unsigned)e < (unsigned)p.E) atomicAdd(&cnt_s[e], 1);
      }
      scores<J, SIG>(l, sg);
#pragma unroll
      for (int j = 0; j < J; ++j) acc[j] += l[j];
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane + 32 * j < p.E) sum_s[warp * p.E + lane + 32 * j] = acc[j];
    if (lane == 0) atomicAdd(&n_s, n);
    __syncthreads();
    const long slot = blockIdx.x + s;
    for (int e = threadIdx.x; e < p.E; e += kWarps * 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += sum_s[w * p.E + e];
      p.part_p[slot * p.E + e] = v;
      p.part_c[slot * p.E + e] = cnt_s[e];
    }
    if (threadIdx.x == 0) p.part_n[slot] = n_s;
    __syncthreads();
  }
}

// One block per (sequence, 32 experts): the slots of the sequence added up in order.  The last block of
// the grid adds up the loss.
__global__ void __launch_bounds__(1024) balance_join_kernel(const BalanceArgs p) {
  __shared__ float fp[32][33];
  __shared__ int fc[32][33];
  __shared__ int fn[32];
  __shared__ bool last;
  griddep_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int s = blockIdx.x, e = blockIdx.y * 32 + lane;
  const int a = seq_start(p, s), b = seq_start(p, s + 1);
  const int c0 = a / p.chunk, c1 = b > a ? (b - 1) / p.chunk + 1 : c0;   // chunks of the sequence
  float vp = 0.f;
  int vc = 0, vn = 0;
  for (int c = c0 + w; c < c1; c += 32) {
    const long slot = c + s;
    if (e < p.E) {
      vp += p.part_p[slot * p.E + e];
      vc += p.part_c[slot * p.E + e];
    }
    if (lane == 0) vn += p.part_n[slot];
  }
  fp[w][lane] = vp;
  fc[w][lane] = vc;
  if (lane == 0) fn[w] = vn;
  __syncthreads();
  if (w == 0) {
    vp = 0.f;
    vc = vn = 0;
    for (int i = 0; i < 32; ++i) {
      vp += fp[i][lane];
      vc += fc[i][lane];
      vn += fn[i];
    }
    if (e < p.E) {
      p.counts[(long)s * p.E + e] = vc;
      p.probs[(long)s * p.E + e] = vn > 0 ? vp / (float)vn : 0.f;
    }
    if (blockIdx.y == 0 && lane == 0) p.tokens[s] = vn;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(p.ticket, 1u) == gridDim.x * gridDim.y - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  // 64-bit sums: S * E terms of one sign each
  double v = 0.0;
  int live = 0;
  for (int q = w; q < p.S; q += 32) {
    const int n = __ldcg(p.tokens + q);
    if (n <= 0) continue;
    live += lane == 0;
    double r = 0.0;
    for (int i = lane; i < p.E; i += 32)
      r += (double)__ldcg(p.counts + (long)q * p.E + i) * (double)__ldcg(p.probs + (long)q * p.E + i);
    v += r / (double)n;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __shared__ double lv[32];
  if (lane == 0) {
    lv[w] = v;
    fn[w] = live;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.0;
    live = 0;
    for (int i = 0; i < 32; ++i) {
      v += lv[i];
      live += fn[i];
    }
    *p.loss = live > 0 ? (float)(v * (double)p.coef * (double)p.E / ((double)p.k * (double)live)) : 0.f;
  }
}

template <class T>
__device__ __forceinline__ void put(T* p, float v, int accumulate);
template <>
__device__ __forceinline__ void put<float>(float* p, float v, int accumulate) { *p = accumulate ? *p + v : v; }
template <>
__device__ __forceinline__ void put<__nv_bfloat16>(__nv_bfloat16* p, float v, int accumulate) {
  *p = __float2bfloat16_rn(accumulate ? __bfloat162float(*p) + v : v);
}

// A warp per token.  Tokens outside every sequence and masked tokens get zeros (or stay, accumulating).
template <class T, int J, bool SIG>
__global__ void __launch_bounds__(kWarps * 32) balance_grad_kernel(const BalanceArgs p) {
  __shared__ int live_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) live_s = 0;
  __syncthreads();
  int live = 0;
  for (int s = threadIdx.x; s < p.S; s += kWarps * 32) live += p.tokens[s] > 0;
  if (live) atomicAdd(&live_s, live);
  __syncthreads();
  const float base = *p.grad_loss * p.coef * (float)p.E / ((float)p.k * (float)max(1, live_s));
  for (int t = blockIdx.x * kWarps + warp; t < p.T; t += gridDim.x * kWarps) {
    const int s = seq_of(p, t);
    T* out = static_cast<T*>(p.grad) + (long)t * p.ldg;
    if (s < 0 || s >= p.S || t >= seq_start(p, s + 1) || (p.mask != nullptr && p.mask[t] == 0) || p.tokens[s] <= 0) {
      if (!p.accumulate) {
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (lane + 32 * j < p.E) put<T>(out + lane + 32 * j, 0.f, 0);
      }
      continue;
    }
    float l[J], sg[J], c[J];
    load_row<T, J>(p, t, lane, l);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = lane + 32 * j;
      c[j] = e < p.E ? (float)__ldg(p.counts + (long)s * p.E + e) : 0.f;
    }
    scores<J, SIG>(l, sg);
    float mean = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) mean += c[j] * l[j];
    mean = warp_sum(mean);
    const float n = (float)p.tokens[s];
    const float g = base / n / n;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float d = g * l[j] * (c[j] - mean);
      if constexpr (SIG) d *= 1.f - sg[j];
      if (lane + 32 * j < p.E) put<T>(out + lane + 32 * j, d, p.accumulate);
    }
  }
}

// ------------------------------------------------------------------ host
size_t r256(size_t b) { return (b + 255) & ~size_t(255); }

struct Layout {
  int chunk, chunks;
  size_t part_p, part_c, part_n, ticket, total;
};

// About two blocks per SM, and chunks of a multiple of the warps.
Layout layout(int T, int E, int S) {
  Layout L;
  int chunk = (T + 2 * 148 - 1) / (2 * 148);
  chunk = (chunk + kWarps - 1) / kWarps * kWarps;
  L.chunk = chunk < kWarps ? kWarps : chunk;
  L.chunks = (T + L.chunk - 1) / L.chunk;
  const size_t slots = (size_t)L.chunks + (size_t)S;
  L.part_p = 0;
  L.part_c = L.part_p + r256(slots * E * 4);
  L.part_n = L.part_c + r256(slots * E * 4);
  L.ticket = L.part_n + r256(slots * 4);
  L.total = L.ticket + 256;
  return L;
}

bool shape_ok(int T, int E, int k, int S) {
  return T >= 0 && E >= 1 && E <= 1024 && k >= 1 && k <= 16 && k <= E && S >= 1 && S <= (1 << 20);
}
bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <class T, int J>
cudaError_t launch_part(const BalanceArgs& a, int score, cudaStream_t s) {
  const size_t smem = (size_t)(kWarps + 1) * a.E * 4;
  auto f = score == MOE_SCORE_SIGMOID ? balance_part_kernel<T, J, true> : balance_part_kernel<T, J, false>;
  f<<<a.chunks, kWarps * 32, smem, s>>>(a);
  return cudaGetLastError();
}
template <class T, int J>
cudaError_t launch_grad(const BalanceArgs& a, int score, cudaStream_t s) {
  const int need = (a.T + kWarps - 1) / kWarps, grid = need < 148 * 8 ? need : 148 * 8;
  auto f = score == MOE_SCORE_SIGMOID ? balance_grad_kernel<T, J, true> : balance_grad_kernel<T, J, false>;
  f<<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}
template <class T>
cudaError_t launch_any(const BalanceArgs& a, int score, bool grad, cudaStream_t s) {
  const int j = (a.E + 31) / 32;
#define MOE_J(N) (grad ? launch_grad<T, N>(a, score, s) : launch_part<T, N>(a, score, s))
  return j <= 1 ? MOE_J(1) : j <= 2 ? MOE_J(2) : j <= 4 ? MOE_J(4) : j <= 8 ? MOE_J(8) : j <= 16 ? MOE_J(16) : MOE_J(32);
#undef MOE_J
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
  a.part_p = reinterpret_cast<float*>(ws + L.part_p);
  a.part_c = reinterpret_cast<int32_t*>(ws + L.part_c);
  a.part_n = reinterpret_cast<int32_t*>(ws + L.part_n);
  a.ticket = reinterpret_cast<uint32_t*>(ws + L.ticket);
  a.loss = loss;
  a.counts = counts;
  a.probs = probs;
  a.tokens = tokens;
  cudaError_t e = logits_type == MOE_TYPE_FP32 ? launch_any<float>(a, score, false, s)
                                               : launch_any<__nv_bfloat16>(a, score, false, s);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  balance_join_kernel<<<dim3(S, (E + 31) / 32), 1024, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.grad_loss = grad_loss;
  a.grad = grad_logits;
  a.ldg = ldg;
  a.accumulate = accumulate != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = logits_type == MOE_TYPE_FP32 ? launch_any<float>(a, score, true, s)
                                               : launch_any<__nv_bfloat16>(a, score, true, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
