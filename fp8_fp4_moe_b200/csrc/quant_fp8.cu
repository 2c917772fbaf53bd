// Block quantisation to FP8 with power-of-two scales (moe_quant_fp8).
//
// For every block (1 x 128 along a row, 128 x 1 along a column of the transposed copy, or 128 x 128):
//   p = the smallest integer >= -126 with amax <= MAX * 2^p (0 for an all-zero block),
//   code = rne_fp8(x * 2^-p), MAX = 448 (E4M3) or 57344 (E5M2), scale = 2^p (fp32 or UE8M0 code p + 127)
// -- the layer's own activation rule, so x * 2^-p is exact and the codes do not depend on how they are
// computed.  Both kernels read x once and are bound by memory traffic.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/moe_b200.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

struct QuantArgs {
  int M, K;
  const void* x;
  long ldx;
  uint8_t* q;
  long ldq;
  void* s;
  long s_row, s_blk;     // strides of the scales in elements: row (or row block), K block
  uint8_t* qt;
  long ldqt;
  void* st;
  long st_row, st_blk;   // column (or column block), row block
  int ue8m0;             // scale type
  int x_vec;             // 16-byte loads of x are allowed
};

// ------------------------------------------------------------------ elements
template <class T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }

// 8 consecutive elements of one row, as they are stored
template <class T>
struct Vec8 {
  static constexpr int kWords = sizeof(T) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint16_t h = (uint16_t)(w[i >> 1] >> ((i & 1) * 16));
      return to_float<T>(*reinterpret_cast<const T*>(&h));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // elements [0, n) of p (n <= 0: none), the rest zero
  __device__ __forceinline__ void load(const T* p, int n, bool vec) {
    if (vec && n >= 8) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
      return;
    }
    zero();
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i] = __float_as_uint(p[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << ((i & 1) * 16);
    }
  }
};

// E5 = E5M2 (largest value 1.75 * 2^15), else E4M3 (1.75 * 2^8): the exponent rule is the same one
// shifted by the difference of the two largest exponents.  A subnormal amax ends at the least exponent.
template <bool E5>
__device__ __forceinline__ int block_exp(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int p = (int)(bits >> 23) - 127 - (E5 ? 15 : 8) + ((bits & 0x7FFFFF) > 0x600000u ? 1 : 0);
  return amax > 0.f ? max(p, -126) : 0;
}

template <bool E5>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  if constexpr (E5) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %2, %1;" : "=h"(lo) : "f"(a), "f"(b));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %2, %1;" : "=h"(hi) : "f"(c), "f"(d));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  } else {
    return pack_e4m3x4(a, b, c, d);
  }
}

__device__ __forceinline__ void store_scale(void* s, long at, int p, int ue8m0) {
  if (ue8m0)
    static_cast<uint8_t*>(s)[at] = (uint8_t)(p + 127);
  else
    static_cast<float*>(s)[at] = __uint_as_float((uint32_t)(p + 127) << 23);
}

__device__ __forceinline__ void store_codes8(uint8_t* dst, uint2 v, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(dst) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) dst[i] = (uint8_t)((i < 4 ? v.x : v.y) >> ((i & 3) * 8));
}

// Scales as the elements are multiplied: bf16 in pairs as they are stored (a power of two changes the exponent
// alone; what becomes subnormal is far below FP8's least value), the other types in fp32.
struct Scale {
  float f;
  uint32_t h;                        // bf16 bits
  __device__ __forceinline__ explicit Scale(int p = 0) : f(exp2_neg(p)), h((uint32_t)(127 - p) << 7) {}
};
// Words of two values a (first half) and b.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t v, uint32_t s) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&s));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <class T, bool E5>
__device__ __forceinline__ uint2 encode8(const Vec8<T>& v, const Scale& sc) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = mul_bf16x2(v.w[i], sc.h * 0x10001u);
    return make_uint2(pack4<E5>(low(w[0]), high(w[0]), low(w[1]), high(w[1])),
                      pack4<E5>(low(w[2]), high(w[2]), low(w[3]), high(w[3])));
  } else {
    return make_uint2(pack4<E5>(v.get(0) * sc.f, v.get(1) * sc.f, v.get(2) * sc.f, v.get(3) * sc.f),
                      pack4<E5>(v.get(4) * sc.f, v.get(5) * sc.f, v.get(6) * sc.f, v.get(7) * sc.f));
  }
}
// Columns 2 j and 2 j + 1 of 8 rows, each with its scale.
template <class T, bool E5>
__device__ __forceinline__ void encode_columns(const Vec8<T> (&v)[8], int j, const Scale& a, const Scale& b, uint2 (&out)[2]) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = mul_bf16x2(v[i].w[j], a.h | b.h << 16);
    out[0] = make_uint2(pack4<E5>(low(w[0]), low(w[1]), low(w[2]), low(w[3])),
                        pack4<E5>(low(w[4]), low(w[5]), low(w[6]), low(w[7])));
    out[1] = make_uint2(pack4<E5>(high(w[0]), high(w[1]), high(w[2]), high(w[3])),
                        pack4<E5>(high(w[4]), high(w[5]), high(w[6]), high(w[7])));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float s = h ? b.f : a.f;
      const int c = 2 * j + h;
      out[h] = make_uint2(pack4<E5>(v[0].get(c) * s, v[1].get(c) * s, v[2].get(c) * s, v[3].get(c) * s),
                          pack4<E5>(v[4].get(c) * s, v[5].get(c) * s, v[6].get(c) * s, v[7].get(c) * s));
    }
  }
}

// Largest magnitudes; a NaN is passed over.  Two 16-bit values share an instruction: their magnitudes, with the
// sign bits cleared, are in the order of the numbers.
template <class T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
};
template <>
struct Pair<__half> {
  using type = __half2;
};
template <class T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {   // b any, a without signs
  using P = typename Pair<T>::type;
  b &= 0x7FFF7FFFu;
  const P m = __hmax2(*reinterpret_cast<const P*>(&a), *reinterpret_cast<const P*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
template <class T>
__device__ __forceinline__ float half_of(uint32_t w, int i) {
  const uint16_t h = (uint16_t)(w >> (16 * i));
  return to_float<T>(*reinterpret_cast<const T*>(&h));
}
template <class T>
__device__ __forceinline__ float amax8(const Vec8<T>& v) {
  if constexpr (sizeof(T) == 4) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v.get(i)));
    return a;
  } else {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = max2<T>(a, v.w[i]);
    return fmaxf(half_of<T>(a, 0), half_of<T>(a, 1));
  }
}
// of the 8 rows, over the 16 lanes that share them
template <class T>
__device__ __forceinline__ void row_amax(const Vec8<T> (&v)[8], float (&a)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = amax8(v[i]);
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) a[i] = fmaxf(a[i], __shfl_xor_sync(0xffffffffu, a[i], o));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {           // two rows to a word
      uint32_t m[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[h] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m[h] = max2<T>(m[h], v[i + h].w[j]);
      }
      uint32_t w = max2<T>(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) w = max2<T>(w, __shfl_xor_sync(0xffffffffu, w, o));
      a[i] = half_of<T>(w, 0);
      a[i + 1] = half_of<T>(w, 1);
    }
  }
}
// of each of the 8 columns of 8 rows
template <class T>
__device__ __forceinline__ void column_amax(const Vec8<T> (&v)[8], float (&a)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a[j] = fmaxf(a[j], fabsf(v[i].get(j)));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max2<T>(m, v[i].w[j]);
      a[2 * j] = half_of<T>(m, 0);
      a[2 * j + 1] = half_of<T>(m, 1);
    }
  }
}

// ------------------------------------------------------------------ rows only
// 16 lanes per 1 x 128 block, 8 elements a lane: no shared memory, one block per half-warp, so that a
// single row of activations already spreads over many SMs.  64 x 7168 bf16: 1.8 us, the time of a launch.
template <class T, bool E5>
__global__ void __launch_bounds__(256) quant_rows_kernel(const QuantArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const int kb = (p.K + 127) / 128;
  const long blocks = (long)p.M * kb;
  const int l16 = threadIdx.x & 15;
  for (long b = (long)blockIdx.x * 16 + (threadIdx.x >> 4); b - (threadIdx.x >> 4) % 2 < blocks;
       b += (long)gridDim.x * 16) {
    const bool live = b < blocks;      // both half-warps stay for the shuffles
    const long row = live ? b / kb : 0;
    const int blk = live ? (int)(b - row * kb) : 0;
    const int k0 = blk * 128 + l16 * 8;
    const int n = live ? p.K - k0 : 0;
    Vec8<T> v;
    v.load(static_cast<const T*>(p.x) + row * p.ldx + k0, n, p.x_vec);
    float a = amax8(v);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const int e = block_exp<E5>(a);
    store_codes8(p.q + row * p.ldq + k0, encode8<T, E5>(v, Scale(e)), n);
    if (live && l16 == 0) store_scale(p.s, row * p.s_row + blk * p.s_blk, e, p.ue8m0);
  }
}

// ------------------------------------------------------------------ 128 x 128 tiles
// One tile of x per block, held in registers: thread (g, c) = (tid / 16, tid % 16) has rows 8 g .. 8 g + 7
// and columns 8 c .. 8 c + 7, so a row's 16 lanes sit in one half-warp and a column's 8 rows make 8
// consecutive bytes of the transposed copy, which goes out through shared memory in whole rows.
// Four blocks of 16-bit elements fit an SM, three of fp32.  Two directions of bf16 at 8192 x 7168: 45 us, 5.3 TB/s (57
// with three blocks and every value widened to fp32 before maxima and scaling); fp32 weights of 4096 x 7168 in
// 128 x 128 blocks, both directions: 29 us, 6.1 TB/s.
template <class T, bool E5, bool TILE>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 3 : 4) quant_tile_kernel(const QuantArgs p) {
  __shared__ __align__(16) uint8_t tr[128 * 128];   // transposed codes, 8-byte pieces XOR-swizzled
  __shared__ __align__(16) float cmax[8][128];      // of each warp's 16 rows
  __shared__ int cexp[128];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, g = tid >> 4, c = tid & 15, lane = tid & 31;
  const int k0 = blockIdx.x * 128, m0 = blockIdx.y * 128;
  const int kc = k0 + c * 8;
  const int nk = p.K - kc;                          // columns of this thread inside x
  Vec8<T> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + g * 8 + i;
    v[i].load(static_cast<const T*>(p.x) + (long)m * p.ldx + kc, m < p.M ? nk : 0, p.x_vec);
  }
  Scale sc_tile;
  if constexpr (TILE) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, amax8(v[i]));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (lane == 0) cmax[0][tid >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) a = fmaxf(a, cmax[0][w]);
    const int e = block_exp<E5>(a);
    sc_tile = Scale(e);
    if (tid == 0) {
      if (p.q) store_scale(p.s, blockIdx.y * p.s_row + blockIdx.x * p.s_blk, e, p.ue8m0);
      if (p.qt) store_scale(p.st, blockIdx.x * p.st_row + blockIdx.y * p.st_blk, e, p.ue8m0);
    }
  }
  if (p.q) {
    float a[8];
    if constexpr (!TILE) row_amax<T>(v, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = m0 + g * 8 + i;
      Scale sc = sc_tile;
      if constexpr (!TILE) {
        const int e = block_exp<E5>(a[i]);
        sc = Scale(e);
        if (c == i && m < p.M) store_scale(p.s, (long)m * p.s_row + blockIdx.x * p.s_blk, e, p.ue8m0);
      }
      if (m < p.M) store_codes8(p.q + (long)m * p.ldq + kc, encode8<T, E5>(v[i], sc), nk);
    }
  }
  if (!p.qt) return;
  Scale sc[8];
  if constexpr (TILE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sc[j] = sc_tile;
  } else {
    float m[8];
    column_amax<T>(v, m);
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
    if (lane < 16) {
      float4* d = reinterpret_cast<float4*>(&cmax[tid >> 5][c * 8]);
      d[0] = make_float4(m[0], m[1], m[2], m[3]);
      d[1] = make_float4(m[4], m[5], m[6], m[7]);
    }
    __syncthreads();
    if (tid < 128) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) a = fmaxf(a, cmax[w][tid]);
      const int e = block_exp<E5>(a);
      cexp[tid] = e;
      if (k0 + tid < p.K) store_scale(p.st, (long)(k0 + tid) * p.st_row + blockIdx.y * p.st_blk, e, p.ue8m0);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) sc[j] = Scale(cexp[c * 8 + j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint2 w[2];
    encode_columns<T, E5>(v, j, sc[2 * j], sc[2 * j + 1], w);
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<uint2*>(tr + (c * 8 + 2 * j + h) * 128 + ((g ^ c) & 15) * 8) = w[h];
  }
  __syncthreads();
  // 16 lanes per transposed row, 8 bytes each; piece h of row `col` sits at h ^ (col / 8)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int col = i * 16 + g, h = c;
    const uint2 w = *reinterpret_cast<const uint2*>(tr + col * 128 + ((h ^ (col >> 3)) & 15) * 8);
    const int m = m0 + h * 8;
    if (k0 + col < p.K) store_codes8(p.qt + (long)(k0 + col) * p.ldqt + m, w, p.M - m);
  }
}

template <class T, bool E5>
cudaError_t launch_quant(const QuantArgs& a, bool tile, cudaStream_t s, int sms) {
  const int kb = (a.K + 127) / 128, mb = (a.M + 127) / 128;
  if (!tile && a.qt == nullptr) {
    const long blocks = (long)a.M * kb, need = (blocks + 15) / 16;
    const int grid = (int)(need < 16l * sms ? need : 16l * sms);
    return launch_dependent(quant_rows_kernel<T, E5>, dim3(grid), 256, 0, 1, s, a);
  }
  return launch_dependent(tile ? quant_tile_kernel<T, E5, true> : quant_tile_kernel<T, E5, false>, dim3(kb, mb), 256, 0, 1,
                          s, a);
}

template <class T>
cudaError_t launch_fmt(const QuantArgs& a, int fmt, bool tile, cudaStream_t s, int sms) {
  return fmt == MOE_FP8_E5M2 ? launch_quant<T, true>(a, tile, s, sms) : launch_quant<T, false>(a, tile, s, sms);
}

bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Whether scales of `rows` x `blocks` have a place each: the strides of one index step over all of the other.
bool distinct(long long rows, long long row_stride, long long blocks, long long block_stride) {
  if (row_stride < 0 || block_stride < 0 || (rows > 1 && row_stride == 0) || (blocks > 1 && block_stride == 0)) return false;
  return rows == 1 || blocks == 1 || (row_stride - 1) / (blocks - 1) >= block_stride ||
         (block_stride - 1) / (rows - 1) >= row_stride;
}

}  // namespace

extern "C" int moe_quant_fp8(int M, int K, const void* x, long long ldx, int x_type, int block, int format,
                             int scale_type, void* q, long long ldq, void* scales, long long s_row_stride,
                             long long s_block_stride, void* qt, long long ldqt, void* scales_t,
                             long long st_row_stride, long long st_block_stride, void* stream) {
  if (M < 0 || K < 0 || M > (1 << 30) || K > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((x_type != MOE_TYPE_BF16 && x_type != MOE_TYPE_FP16 && x_type != MOE_TYPE_FP32) ||
      (block != MOE_BLOCK_ROW && block != MOE_BLOCK_TILE) || (format != MOE_FP8_E4M3 && format != MOE_FP8_E5M2) ||
      (scale_type != MOE_SCALE_FP32 && scale_type != MOE_SCALE_UE8M0))
    return MOE_ERR_INVALID_ARG;
  if (M == 0 || K == 0) return MOE_OK;
  if (q == nullptr && qt == nullptr) return MOE_ERR_INVALID_ARG;
  const uintptr_t esize = x_type == MOE_TYPE_FP32 ? 4 : 2, ssize = scale_type == MOE_SCALE_FP32 ? 4 : 1;
  if (!aligned(x, esize) || (M > 1 && ldx < K)) return MOE_ERR_INVALID_ARG;
  const int mb = (M + 127) / 128, kb = (K + 127) / 128;
  const bool tiles = block == MOE_BLOCK_TILE;
  if ((tiles || qt) && mb > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (q && (!aligned(q, 16) || !aligned(scales, ssize) || (M > 1 && (ldq < K || ldq % 16)) ||
            !distinct(tiles ? mb : M, s_row_stride, kb, s_block_stride)))
    return MOE_ERR_INVALID_ARG;
  if (qt && (!aligned(qt, 16) || !aligned(scales_t, ssize) || (K > 1 && (ldqt < M || ldqt % 16)) ||
             !distinct(tiles ? kb : K, st_row_stride, mb, st_block_stride)))
    return MOE_ERR_INVALID_ARG;
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  QuantArgs a{};
  a.M = M;
  a.K = K;
  a.x = x;
  a.ldx = ldx;
  a.q = static_cast<uint8_t*>(q);
  a.ldq = ldq;
  a.s = scales;
  a.s_row = s_row_stride;
  a.s_blk = s_block_stride;
  a.qt = static_cast<uint8_t*>(qt);
  a.ldqt = ldqt;
  a.st = scales_t;
  a.st_row = st_row_stride;
  a.st_blk = st_block_stride;
  a.ue8m0 = scale_type == MOE_SCALE_UE8M0;
  a.x_vec = aligned(x, 16) && (M == 1 || ldx * (long long)esize % 16 == 0);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = x_type == MOE_TYPE_BF16   ? launch_fmt<__nv_bfloat16>(a, format, tiles, s, sms)
                  : x_type == MOE_TYPE_FP16 ? launch_fmt<__half>(a, format, tiles, s, sms)
                                            : launch_fmt<float>(a, format, tiles, s, sms);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
