// Block-scaled FP8 x FP8 matrix product (moe_gemm_fp8) on tcgen05.
//
//   out[m][n] (+)= sum_b sA(m, b) sB(n, b) sum_{k in block b of 128} A[m][k] B[n][k]
//
// One operand ("P") is the MMA's row side, the other ("Q") its column side.  With many tokens P = A; with
// few (M <= 128) the roles swap, P = B: the weight rows fill the 128 lanes and the columns shrink to the
// tokens, so that each weight byte is read once and little is multiplied by padding.
//
//   warp 0      TMA producer: per 128-deep K block the P tile (128 x 128 B) and the Q tile, 128-byte swizzle;
//               codes past the matrix arrive as zeros
//   warp 1      MMA issuer
//   one warp    scales
//   eight warps epilogue: TMEM lane quarter warp % 4, a half of the columns each
// UE8M0 scales (MX): the scale warp writes each stage's scale atoms, tcgen05.mma.kind::mxf8f6f4 applies them and
// the accumulator stays in TMEM over the whole K loop.  fp32 scales: each K block is one kind::f8f6f4
// product into a TMEM buffer of its own, and the epilogue warps add it, scaled, to accumulators in
// registers while the next block's MMAs run.
// Two kernels:
//   pair    two CTAs share each M = 256 MMA (cta_group::2), each holding 128 P rows and half of the Q rows.
//           A single CTA's 128 x 256 tile reads and writes 96 KB of shared memory per K block, 768
//           clocks at 128 B each for 512 clocks of MMA; in the pair the Q half brings that to 64 KB.
//           Persistent, up to 256 columns.
//   small   one CTA per tile of up to 128 columns; where the tiles do not fill the SMs the K loop is split
//           over the CTAs of a cluster, which add up their parts in rank order through distributed shared
//           memory: no workspace, no atomics.
// Every wait is bounded (WaitCtl); on a timeout the CTA records MOE_ERR_DEVICE_TIMEOUT, drains its own
// copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "../../include/moe_b200.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int BM = 128, BK = 128;
constexpr int kPairThreads = 384;             // three warpgroups: TMA, MMA, scales; 2 x epilogue
constexpr int kSmallThreads = 352;            // TMA, MMA, 8 x epilogue, scales
constexpr int kSfSlots = 2;                   // groups of four K blocks whose scales are in flight
constexpr uint32_t kPBytes = BM * BK;
enum : uint32_t { kWhereProducer = 0xB00, kWhereMma = 0xB10, kWhereEpilogue = 0xB20, kWhereScales = 0xB30,
                  kWhereDrain = 0xB40 };

struct Fp8Args {
  int p_rows, q_rows, KB;
  int tiles_p, tiles_q, splits;
  int bn;                            // columns of a tile (pair kernel)
  const void *sp, *sq;               // scales of P and Q
  long sp_row, sp_blk, sq_row, sq_blk;
  int sp_shift, sq_shift;            // 0: per row, 7: per 128 rows
  int sp_quad, sq_quad;              // the scales of four K blocks of a row are one aligned load
  void* out;
  long ldo;
  int out_fp32, accumulate, swap, vec;
  uint32_t idesc;                    // formats and shape of the MMA
  uint32_t* status;
  uint64_t timeout_ns;
};

template <int BN, bool MX>
struct Cfg {
  static constexpr int kStages = BN == 128 ? 6 : BN == 64 ? 8 : BN == 32 ? 9 : 10;
  static constexpr int kCols = BN / 2;                           // columns per epilogue thread
  static constexpr int kAcc = MX ? 2 : 4;                        // TMEM accumulators
  static constexpr uint32_t kSfCol = kAcc * BN;                  // MX: scale columns (P 4, Q 4; 16 a slot)
  static constexpr uint32_t kTmem = (kAcc * BN + (MX ? 32 : 0)) <= 64 ? 64
                                    : (kAcc * BN + (MX ? 32 : 0)) <= 128 ? 128
                                    : (kAcc * BN + (MX ? 32 : 0)) <= 256 ? 256 : 512;
  static constexpr uint32_t kQBytes = BN * BK;
  static constexpr uint32_t kSfq = 512;                          // Q scale atoms of a slot
  static constexpr uint32_t p = 0;
  static constexpr uint32_t q = p + kStages * kPBytes;
  static constexpr uint32_t sfp = q + kStages * kQBytes;
  static constexpr uint32_t sfq = sfp + (MX ? kSfSlots * 512 : 0);
  static constexpr uint32_t ring = sfq + (MX ? kSfSlots * kSfq : 0);
  static constexpr uint32_t kRowBytes = (BM + (BN < 32 ? 32 : BN)) * 4;   // fp32 scales of a K block; whole warps write
  static constexpr uint32_t staging = ring + (MX ? 0 : kSfSlots * 4 * kRowBytes);
  static constexpr uint32_t bars = staging + 8 * 2048;
  static constexpr int kBars = 2 * kStages + 2 * kAcc + 2 * kSfSlots + 1;
  static constexpr uint32_t misc = bars + kBars * 8;
  static constexpr uint32_t total = misc + 16;
  static constexpr uint32_t bytes = total + 1024;                // 1024-byte alignment of the stages
  static_assert(bytes <= 232448, "shared memory");
  // a split tile's partial sums [outer][inner + 4], over the stages (inner: the output's contiguous side)
  static_assert(BM * (BN + 4) * 4 <= sfp && BN * (BM + 4) * 4 <= sfp, "a partial tile fits over the stages");
};

// The pair kernel: each CTA 128 P rows and half of up to 256 Q rows.
template <bool MX>
struct PairCfg {
  static constexpr int kStages = 6;
  static constexpr uint32_t kQBytes = 128 * BK;
  static constexpr uint32_t kSfq = 1024;                         // both CTAs hold the scales of all columns
  static constexpr uint32_t p = 0;
  static constexpr uint32_t q = p + kStages * kPBytes;
  static constexpr uint32_t sfp = q + kStages * kQBytes;
  static constexpr uint32_t sfq = sfp + (MX ? kSfSlots * 512 : 0);
  static constexpr uint32_t ring = sfq + (MX ? kSfSlots * kSfq : 0);
  static constexpr uint32_t kRowBytes = (BM + 256) * 4;            // fp32 scales of a K block
  static constexpr uint32_t staging = ring + (MX ? 0 : kSfSlots * 4 * kRowBytes);
  static constexpr uint32_t bars = staging + 8 * 2048;
  static constexpr int kBars = 2 * kStages + 8 + 2 * kSfSlots + 1;
  static constexpr uint32_t misc = bars + kBars * 8;
  static constexpr uint32_t bytes = misc + 16 + 1024;
  static_assert(bytes <= 232448, "shared memory");
};

__device__ __forceinline__ void tc_mma_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f8f6f4: fp32 accumulator, formats 0 = E4M3, 1 = E5M2, both K-major
__host__ __device__ constexpr uint32_t idesc_f8f6f4(int M, int N, uint32_t a_fmt, uint32_t b_fmt) {
  return (1u << 4) | (a_fmt << 7) | (b_fmt << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint64_t sw128(uint32_t saddr) { return smem_desc(saddr, 16, 1024, kLayoutSwizzle128B); }
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) { return smem_desc(saddr, 16, 128, kLayoutNoSwizzle); }

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if constexpr (N == 32) {
    tmem_ld_32x32b_x32(taddr, *reinterpret_cast<uint32_t(*)[32]>(r));
  } else if constexpr (N == 16) {
    tmem_ld_32x32b_x16(taddr, r);
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  }
}

// 16 lanes x 32 columns as matrix fragments: r[4 i + 2 j + e] is TMEM lane 8 j + lane / 4, column
// 8 i + 2 (lane % 4) + e.  A thread gets 8 columns of several rows instead of all columns of one.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// ... x 16 columns: r[0..7]
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr) : "memory");
  return v;
}
// mbar_wait with the abort flag and the clock looked at once in 64 tries: each look costs more than a K block's
// MMAs, and most waits here end within a few tries.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const WaitCtl& ctl, uint32_t where) {
  uint64_t t0 = 0;
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if ((n & 63) != 0) continue;
    if (*ctl.abort_flag) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > ctl.timeout_ns) {
      report_status(ctl.status, kStatusTimeout, where, parity);
      *ctl.abort_flag = 1;
      __threadfence_block();
      return false;
    }
  }
  return true;
}
// Arrivals on the same barrier of CTA 0 of the pair.  A release at cluster scope costs a memory barrier of
// about 0.7 us, more than a K block's MMAs (8192 x 4096 x 7168: 208 us instead of 168).  arrive_first hands scale atoms in
// this CTA's shared memory over, to be copied to TMEM by CTA 0's thread after see_first: a release and an acquire between
// the CTAs of the cluster that are restricted to shared memory, at no measurable cost.  hand_back returns an
// accumulator: tcgen05.fence::before_thread_sync orders the loads from it, no other memory is passed on.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t"
               "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(bar, 0)) : "memory");
}
__device__ __forceinline__ void see_first() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
__device__ __forceinline__ void hand_back(uint32_t bar_cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster_addr) : "memory");
}

// One thread of the converged warp.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tc_mma_f8f6f4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Tile order: bands of 8 P tiles, every Q tile of a band before the next band, so that what the grid
// works on at a time shares rows of both operands in L2.
__device__ __forceinline__ void tile_coord(const Fp8Args& p, int tile, int& tp, int& tq) {
  constexpr int kBand = 8;
  const int band = tile / (kBand * p.tiles_q), rem = tile - band * kBand * p.tiles_q;
  const int h = min(kBand, p.tiles_p - band * kBand);
  tq = rem / h;
  tp = band * kBand + (rem - tq * h);
}

// One addition per element and call, so their order is fixed; as a reduction it does not wait for the old value.
__device__ __forceinline__ void add_to(float* p, float v) {
  asm volatile("red.global.add.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}
__device__ __forceinline__ void put_out(const Fp8Args& p, long m, long n, float v) {
  if (p.out_fp32) {
    float* o = static_cast<float*>(p.out) + m * p.ldo + n;
    if (p.accumulate)
      add_to(o, v);
    else
      *o = v;
  } else {
    static_cast<__nv_bfloat16*>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
  }
}

// four consecutive columns of a row; columns from n_end on are not written
__device__ __forceinline__ void put_out4(const Fp8Args& p, long m, long n, float4 v, long n_end) {
  if (p.vec && n + 4 <= n_end && !p.accumulate) {
    if (p.out_fp32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + m * p.ldo + n) = v;
    } else {
      __nv_bfloat162 b[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + m * p.ldo + n) = *reinterpret_cast<const uint2*>(b);
    }
    return;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
  if (p.out_fp32 && !p.accumulate) {   // one look at the kind of output for all four
    float* o = static_cast<float*>(p.out) + m * p.ldo + n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < n_end) o[i] = f[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < n_end) put_out(p, m, n + i, f[i]);
}

// 64 bytes of each of the warp's 32 rows from its 2 KB buffer to global memory, so that stores cover whole
// sectors: 16-byte pieces, 4 lanes to a row, where the row pitch and the columns allow it, else element by
// element.  Piece c of row r lies at piece c ^ (r / 2 % 4).  row0, col0: first row and column; cols: columns
// of the matrix from col0 on.
__device__ __forceinline__ uint8_t* piece_at(uint8_t* buf, int r, int c) {
  return buf + r * 64 + ((c ^ ((r >> 1) & 3)) * 16);
}
__device__ __forceinline__ void flush_64b(const Fp8Args& p, uint8_t* buf, long row0, long col0, int rows, int cols, int lane) {
  __syncwarp();
  const int esize = p.out_fp32 ? 4 : 2, n = 64 / esize;
  if (p.vec && cols >= n) {
    uint8_t* dst = static_cast<uint8_t*>(p.out) + (row0 * p.ldo + col0) * esize;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int r = it * 8 + (lane >> 2), c = lane & 3;
      const uint4 w = *reinterpret_cast<const uint4*>(piece_at(buf, r, c));
      if (r < rows) {
        uint8_t* d = dst + (long)r * p.ldo * esize + c * 16;
        if (p.accumulate)
          asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(d), "f"(__uint_as_float(w.x)),
                       "f"(__uint_as_float(w.y)), "f"(__uint_as_float(w.z)), "f"(__uint_as_float(w.w))
                       : "memory");
        else
          *reinterpret_cast<uint4*>(d) = w;
      }
    }
  } else {
    // a lane keeps its column; not unrolled, which costs every call registers and these rows more than it saves
    // (4001 x 2049 x 1000 bf16: 39 instead of 26 us)
    const int c = lane & (n - 1), byte = c * esize;
    const int last = c < cols ? min(rows, 32) : 0;
#pragma unroll 1
    for (int r = lane / n; r < last; r += 32 / n) {
      const uint8_t* at = piece_at(buf, r, byte >> 4) + (byte & 15);
      const long o = (row0 + r) * p.ldo + col0 + c;
      if (p.out_fp32) {
        float* d = static_cast<float*>(p.out) + o;
        const float x = *reinterpret_cast<const float*>(at);
        if (p.accumulate)
          add_to(d, x);
        else
          *d = x;
      } else {
        static_cast<uint16_t*>(p.out)[o] = *reinterpret_cast<const uint16_t*>(at);
      }
    }
  }
  __syncwarp();
}
// 32 columns of the warp's rows, lane = row
__device__ __forceinline__ void store_rows(const Fp8Args& p, uint8_t* buf, const float* v, long row0, long col0, int rows,
                                           int cols, int lane) {
  if (p.out_fp32) {
#pragma unroll
    for (int s = 0; s < 32; s += 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(piece_at(buf, lane, i)) =
            make_float4(v[s + 4 * i], v[s + 4 * i + 1], v[s + 4 * i + 2], v[s + 4 * i + 3]);
      flush_64b(p, buf, row0, col0 + s, rows, cols - s, lane);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
      *reinterpret_cast<uint4*>(piece_at(buf, lane, i)) = *reinterpret_cast<const uint4*>(b);
    }
    flush_64b(p, buf, row0, col0, rows, cols, lane);
  }
}
// 32 columns of the warp's rows as fragments (see tmem_ld_frag): v[h * 16 + 4 i + 2 j + e] is row
// 16 h + 8 j + lane / 4, column 8 i + 2 (lane % 4) + e
__device__ __forceinline__ void store_frags(const Fp8Args& p, uint8_t* buf, const float* v, long row0, long col0, int rows,
                                            int cols, int lane) {
  const int quad = lane & 3, r0 = lane >> 2;
  if (p.out_fp32) {
#pragma unroll
    for (int s = 0; s < 4; s += 2) {           // two groups of 8 columns: 64 bytes
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h)
          *reinterpret_cast<float2*>(piece_at(buf, 8 * h + r0, 2 * i + (quad >> 1)) + (quad & 1) * 8) =
              make_float2(v[(h >> 1) * 16 + 4 * (s + i) + 2 * (h & 1)], v[(h >> 1) * 16 + 4 * (s + i) + 2 * (h & 1) + 1]);
      flush_64b(p, buf, row0, col0 + 8 * s, rows, cols - 8 * s, lane);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        *reinterpret_cast<__nv_bfloat162*>(piece_at(buf, 8 * h + r0, i) + quad * 4) =
            __floats2bfloat162_rn(v[(h >> 1) * 16 + 4 * i + 2 * (h & 1)], v[(h >> 1) * 16 + 4 * i + 2 * (h & 1) + 1]);
    flush_64b(p, buf, row0, col0, rows, cols, lane);
  }
}

// fp32 scales may have any finite value.  Two of magnitudes in [2^-62, 2^63), or zero, have a product that is normal or
// zero, and a block sum takes it in one FMA.  In a group of four K blocks with others (a byte per slot and scale
// warp tells the epilogue) the two are applied one after the other where need be (add_scaled).  That loop holds its sums in
// local memory and looks at few columns at a time, so that the ordinary one keeps its registers: with both additions in
// one loop 8192 x 4096 x 7168 took 265 us, not 227, column scales 453 at 4096 x 7168 x 8191, not 336.
__device__ __forceinline__ bool plain_scale(uint32_t bits) {
  constexpr uint32_t lo = (127u - 62) << 23, hi = (127u + 63) << 23;
  const uint32_t u = bits & 0x7FFFFFFFu;
  return u - lo < hi - lo || u == 0;
}
__device__ __forceinline__ bool any_wide(const uint8_t* wide, int slot) {
  return *reinterpret_cast<const volatile uint16_t*>(wide + slot * 2) != 0;
}
// a + v p q, |v| zero or in [2^-32, 2^39).  Unless p q is normal, v takes one scale after the other, in the order that
// stays in range wherever the result does.  A product beyond the largest value: the smaller scale is 1 at least, so v
// times it does not underflow, and overflows only with the result.  A product below the normal range: one scale is
// below 2^-63 and the other below 2^23, whose product with v is in range, or it is below 2^-126 and the result below 2^-189.
// A zero goes first.
__device__ __forceinline__ float add_scaled(float v, float p, float q, float a) {
  constexpr float kLeast = 1.17549435e-38f, kLargest = 3.402823466e38f;   // normal numbers
  const float s = p * q, mag = fabsf(s);
  if (mag >= kLeast && mag <= kLargest) return fmaf(v, s, a);
  const bool p_larger = fabsf(p) >= fabsf(q);
  const float big = p_larger ? p : q, small = p_larger ? q : p;
  return mag < kLeast && small != 0.f ? fmaf(v * big, small, a) : fmaf(v * small, big, a);
}

// Scales of a tile on their way into shared memory, four K blocks at a time; rows l, l + 32, l + 64, l + 96
// of P are lane l's items 0 to 3, its rows of Q the items from 4 on (fp32 with one scale per 128 columns: row
// 128 l); a warp has the items [FIRST, FIRST + NR).  The next four blocks are in flight
// while the current ones wait for their slot.
// UE8M0: an atom's word holds a row's scales of the four blocks; the MMAs of block j take byte j of it for all of
// their 32-K steps, so that one copy to TMEM serves four blocks.  fp32: per block, [128] of P, then of Q.
// The addresses are kept and advanced: worked out anew for each group, they took one warp longer than the group's
// MMAs.
template <bool MX, int FIRST, int NR, bool QROW>
struct ScaleLoader {
  using Word = std::conditional_t<MX, uint8_t, uint32_t>;
  const Word* at[NR];                // scales of the next four blocks
  uint32_t live;                     // items inside the matrix
  bool quad[2];                      // P, Q: one load for four blocks (MX: v[i][0] is the atom's word then)
  bool quads;                        // ... in what v holds
  uint32_t v[NR][4];
  static __device__ __forceinline__ constexpr bool is_p(int i) { return FIRST + i < 4; }
  __device__ __forceinline__ void begin(const Fp8Args& p, int p_row, int q_row, int q_n, int lane, int kb) {
    live = 0;
    quad[0] = p.sp_quad;
    quad[1] = p.sq_quad;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int in = is_p(i) ? lane + 32 * (FIRST + i) : QROW ? lane + 32 * (FIRST + i - 4) : lane * 128;
      const int row = (is_p(i) ? p_row : q_row) + in;
      const bool on = is_p(i) ? row < p.p_rows : in < q_n && row < p.q_rows;
      const long o = is_p(i) ? (long)(row >> p.sp_shift) * p.sp_row + kb * p.sp_blk
                             : (long)(row >> p.sq_shift) * p.sq_row + kb * p.sq_blk;
      at[i] = static_cast<const Word*>(is_p(i) ? p.sp : p.sq) + (on ? o : 0);
      live |= (uint32_t)on << i;
    }
  }
  // the next n blocks (n <= 0: none), and on to the four after them
  __device__ __forceinline__ void load(const Fp8Args& p, int n) {
    constexpr uint32_t kNone = MX ? 127u : 0u;   // past the matrix
    quads = n >= 4;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const bool on = live >> i & 1;
      const long blk = is_p(i) ? p.sp_blk : p.sq_blk;
      if (quads && quad[is_p(i) ? 0 : 1]) {
        if constexpr (MX) {
          v[i][0] = on ? *reinterpret_cast<const uint32_t*>(at[i]) : 0x7F7F7F7Fu;
        } else {
          const uint4 w = on ? *reinterpret_cast<const uint4*>(at[i]) : make_uint4(0, 0, 0, 0);
          v[i][0] = w.x;
          v[i][1] = w.y;
          v[i][2] = w.z;
          v[i][3] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = on && j < n ? at[i][j * blk] : kNone;
      }
      if (on) at[i] += 4 * blk;
    }
  }
  __device__ __forceinline__ void store_atoms(uint8_t* sfp, uint8_t* sfq, int lane) {
#pragma unroll
    for (int i = 0; i < NR; i += 4) {
      uint32_t w[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        w[r] = quads && quad[i < 4 ? 0 : 1] ? v[i + r][0] : v[i + r][0] | v[i + r][1] << 8 | v[i + r][2] << 16 | v[i + r][3] << 24;
      *reinterpret_cast<uint4*>((i < 4 ? sfp : sfq + (i - 4) * 128) + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
  }
  // wide: the slot's byte of this warp, whether one of its scales is outside the range of plain_scale
  __device__ __forceinline__ void store_rows(uint8_t* slot, uint32_t row_bytes, uint8_t* wide, int lane) {
    bool out = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t* d = reinterpret_cast<uint32_t*>(slot + j * row_bytes);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        if (FIRST + i < 4 || QROW || lane < 2) d[lane + 32 * (FIRST + i)] = v[i][j];
        out |= !plain_scale(v[i][j]);
      }
    }
    out = __any_sync(0xffffffffu, out);
    if (lane == 0) *wide = out;
    __syncwarp();
  }
};
// idesc with the scale byte of both operands
__device__ __forceinline__ uint32_t with_byte(uint32_t idesc, int j) { return idesc | (uint32_t)j << 4 | (uint32_t)j << 29; }

// ------------------------------------------------------------------ pair kernel
// What bounds it (8192 x 4096 x 7168, 481 GFLOP): UE8M0 170 us, 2.8 PFLOP/s -- the power limit, under which the SM clock
// falls to about 1.4 GHz, and the last wave of tiles; tensor pipe busy three quarters of the cycles at 2048 rows.
// fp32 scales 227 us, 2.1 PFLOP/s: the epilogue warps' TMEM reads and one FMA per element and K block beside the
// MMAs.  No unit is full (2048 rows: tensor pipe 51 %, FMA pipe 30 %, issue slots 48 %): buffers go back and
// forth between MMAs and additions, two of 256 columns, and each side waits for the other.  QROW 336 us at 4096 x 7168 x
// 8191, 1.4 PFLOP/s: a second fp32 operation per element and the column scales' shared-memory reads (tensor pipe 33 %, FMA
// pipe 37 %, issue slots 54 %).
// QROW (fp32 scales only): Q's scales differ by column; otherwise one per 128 columns, and every tile
// starts at a multiple of 128.  NC: columns of an epilogue thread; with fp32 scales bn = 2 NC, known to the
// compiler so that it can move loads and additions of different columns past each other (NC = 112: the
// last 16 of them by themselves); UE8M0: up to NC.
template <bool MX, bool QROW, int NC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                         const Fp8Args p) {
  using C = PairCfg<MX>;
  constexpr int ST = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the same offset in both CTAs: dynamic shared memory starts at one address everywhere
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);   // rank 0's count for both
  uint64_t* empty = full + ST;
  uint64_t* accf = empty + ST;
  uint64_t* acce = accf + 4;                                      // rank 0's
  uint64_t* sfull = acce + 4;                                     // UE8M0: rank 0's
  uint64_t* sempty = sfull + kSfSlots;
  uint64_t* drain = sempty + kSfSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc + 4);
  uint8_t* wide = smem + C::misc + 8;                             // fp32 scales: [slot][scale warp]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const WaitCtl ctl{abort_flag, p.status, p.timeout_ns};

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);          // rank 0's producer; the bytes of both CTAs
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 16);
    }
    for (int i = 0; i < kSfSlots; ++i) {
      mbar_init(&sfull[i], MX || QROW ? 2 : 1);   // UE8M0: the scale warps of both CTAs; QROW: two warps
      mbar_init(&sempty[i], MX ? 1 : 8);   // the copies to TMEM, or the epilogue warps
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *reinterpret_cast<uint32_t*>(wide) = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  griddep_wait();                      // nothing above touches global memory
  // TMEM only now: a block that held some while it waits for a kernel that has not allocated its own yet would
  // keep that kernel from ending, on an SM that has room for both
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  if (blockIdx.x == 0 && threadIdx.x < 4) p.status[threadIdx.x] = 0;   // long before any wait can expire
  __syncthreads();
  griddep_launch_dependents();         // after the allocation, for the same reason
  cluster_sync();                      // the peer's barriers are initialised before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int KB = p.KB, bn = MX ? p.bn : 2 * NC;
  const int tiles = p.tiles_p * p.tiles_q, first = blockIdx.x >> 1, step = gridDim.x >> 1;
  // UE8M0: two accumulators where two of bn columns and the scales behind the first fit, else one.  fp32
  // scales: as many as fit, up to four: from the end of a block's MMAs to the next use of its buffer lie about
  // 900 clocks of commits, waits and the arrival at the other CTA, which only other buffers' MMAs fill
  const int na = MX ? (bn > 224 ? 1 : 2) : min(4, 512 / bn);
  const uint32_t acc_cols = MX || bn > 128 ? 256 : bn;
  const uint32_t sf_col = bn > 224 ? 256 : 224;

  // fp32 scales: the epilogue warps hold 128 accumulators each, beyond the 168 registers a thread of 12
  // warps; the first warpgroup gives up what they need: 128 x 72 + 256 x 216 = 384 x 168
  if (warp < 4) {
    if constexpr (!MX) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0, fills = 0;
        const uint32_t q_bytes = (uint32_t)bn / 2 * BK, full0 = mapa_shared(full, 0);
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
          int tp, tq;
          tile_coord(p, tile, tp, tq);
          for (int kb = 0; kb < KB; ++kb) {
            ok = wait_for(&empty[stage], phase ^ 1, ctl, kWhereProducer);
            if (!ok) break;
            const uint32_t fb = full0 + stage * 8;
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (kPBytes + q_bytes));
            tma_load_2d_pair(smem + C::p + stage * kPBytes, &tmP, kb * BK, tp * 256 + rank * BM, fb);
            tma_load_2d_pair(smem + C::q + stage * C::kQBytes, &tmQ, kb * BK, tq * bn + rank * (bn / 2), fb);
            ++fills;
            if (++stage == ST) { stage = 0; phase ^= 1; }
          }
        }
        // rank 0's stage barriers count both CTAs' copies: waiting for them covers the peer too
        if (rank == 0)
          for (int s = 0; s < ST; ++s) {
            const uint32_t n = (fills + ST - 1 - s) / ST;
            if (n > 0 && !mbar_wait_drain(&full[s], (n - 1) & 1, p.timeout_ns))
              report_status(p.status, kStatusTimeout, kWhereDrain, s);
          }
      }
    } else if (warp == 1) {
      if (rank == 0 && elect()) {      // one thread; elected, so that the compiler keeps the operands uniform
        const uint64_t dp0 = sw128(smem_u32(smem + C::p)), dq0 = sw128(smem_u32(smem + C::q));
        const uint64_t sp0 = sf_desc(smem_u32(smem + C::sfp)), sq0 = sf_desc(smem_u32(smem + C::sfq));
        int stage = 0, buf = 0, sf = 0;
        uint32_t phase = 0, aphase = 0, sphase = 0, tsp = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
          for (int kb = 0; kb < KB; ++kb) {
            if ((!MX || kb == 0) && !wait_for(&acce[buf], aphase ^ 1, ctl, kWhereMma)) { ok = false; break; }
            if (MX && (kb & 3) == 0) {
              if (!wait_for(&sfull[sf], sphase, ctl, kWhereMma + 2)) { ok = false; break; }
              see_first();
              tc_fence_after();
              tsp = tmem + sf_col + sf * 16;     // the slots' columns alternate as well
              const uint64_t sp = sp0 + sf * (512 >> 4), sq = sq0 + sf * (C::kSfq >> 4);
              tc_cp_32x128b_warpx4_pair(tsp, sp);
              tc_cp_32x128b_warpx4_pair(tsp + 4, sq);
              tc_cp_32x128b_warpx4_pair(tsp + 8, sq + 32);
              tc_commit_pair(&sempty[sf], 0x3);
              if (++sf == kSfSlots) { sf = 0; sphase ^= 1; }
            }
            if (!wait_for(&full[stage], phase, ctl, kWhereMma + 1)) { ok = false; break; }
            tc_fence_after();
            const uint32_t acc = tmem + buf * acc_cols;
            const uint64_t dp = dp0 + stage * (kPBytes >> 4), dq = dq0 + stage * (C::kQBytes >> 4);
            if constexpr (MX) {
              const uint32_t id = with_byte(p.idesc, kb & 3);
#pragma unroll
              for (int i = 0; i < 4; ++i) tc_mma_mxf8f6f4_pair(acc, dp + 2 * i, dq + 2 * i, id, tsp, tsp + 4, kb | i);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) tc_mma_f8f6f4_pair(acc, dp + 2 * i, dq + 2 * i, p.idesc, i);
            }
            tc_commit_pair(&empty[stage], 0x3);
            if (!MX || kb == KB - 1) {
              tc_commit_pair(&accf[buf], 0x3);
              if (++buf == na) { buf = 0; aphase ^= 1; }
            }
            if (++stage == ST) { stage = 0; phase ^= 1; }
          }
        }
        tc_commit_pair(drain, 0x1);
        if (!mbar_wait_drain(drain, 0, p.timeout_ns)) report_status(p.status, kStatusTimeout, kWhereDrain, 99);
      }
    } else {
      auto feed = [&](auto sf) {
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
          int tp, tq;
          tile_coord(p, tile, tp, tq);
          const int p_row = tp * 256 + rank * BM, q_row = tq * bn;
          sf.begin(p, p_row, q_row, bn, lane, 0);
          sf.load(p, KB);
          for (int kb = 0; kb < KB; kb += 4) {
            ok = __all_sync(0xffffffffu, wait_for(&sempty[slot], phase ^ 1, ctl, kWhereScales));
            if (!ok) break;
            if constexpr (MX) {
              sf.store_atoms(smem + C::sfp + slot * 512, smem + C::sfq + slot * C::kSfq, lane);
              if (lane == 0) arrive_first(&sfull[slot]);
            } else {
              sf.store_rows(smem + C::ring + slot * 4 * C::kRowBytes, C::kRowBytes, wide + slot * 2 + warp - 2, lane);
              if (lane == 0) mbar_arrive(&sfull[slot]);
            }
            sf.load(p, KB - kb - 4);
            if (++slot == kSfSlots) { slot = 0; phase ^= 1; }
          }
        }
      };
      constexpr int kItems = 4 + NC / 16, kHalf = (kItems + 1) / 2;   // QROW: the items of two warps, which have 72 registers
      if (warp == 2) {
        if constexpr (MX)
          feed(ScaleLoader<true, 0, 12, true>());
        else if constexpr (QROW)
          feed(ScaleLoader<false, 0, kHalf, true>());
        else
          feed(ScaleLoader<false, 0, 5, false>());
      } else if constexpr (!MX && QROW) {
        feed(ScaleLoader<false, kHalf, kItems - kHalf, true>());
      }
    }
  } else {
    if constexpr (!MX) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ------------------------------------------------------------ epilogue (warps 4..11, both CTAs)
    const int q = warp & 3, half = (warp - 4) >> 2;
    uint8_t* obuf = smem + C::staging + (warp - 4) * 2048;
    // columns [0, h) and [h, bn), UE8M0: h a multiple of 32; both kinds of warp sit on every scheduler
    const int h = MX ? (bn / 2 + 31) & ~31 : NC, c0 = half ? h : 0, nc = half ? bn - h : h;
    const uint32_t t_acc = tmem + c0 + ((uint32_t)(q * 32) << 16), acce0 = mapa_shared(acce, 0);
    int buf = 0, slot = 0;
    uint32_t aphase = 0, rphase = 0;
    bool ok = true;
    for (int tile = first; tile < tiles; tile += step) {
      int tp, tq;
      tile_coord(p, tile, tp, tq);
      float acc[(NC + 31) / 32 * 32];
      if constexpr (MX) {
        ok = __all_sync(0xffffffffu, wait_for(&accf[buf], aphase, ctl, kWhereEpilogue));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NC; c += 32)
          if (c < nc) tmem_ld<32>(t_acc + buf * acc_cols + c, reinterpret_cast<uint32_t*>(acc + c));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) hand_back(acce0 + buf * 8);
        if (++buf == na) { buf = 0; aphase ^= 1; }
      } else {
#pragma unroll
        for (int c = 0; c < (NC + 31) / 32 * 32; ++c) acc[c] = 0.f;
        // 32 columns at a time, the next ones on their way from TMEM while these are added
        auto load = [&](int c, uint32_t* r) {
          const uint32_t t = t_acc + buf * acc_cols + c;
          if constexpr (QROW) {
            if (c + 32 <= NC) {
              tmem_ld_frag(t, r);
              tmem_ld_frag(t + (16u << 16), r + 16);
            } else {
              tmem_ld_frag16(t, r);
              tmem_ld_frag16(t + (16u << 16), r + 16);
            }
          } else {
            tmem_ld<32>(t, r);
          }
        };
        for (int g = 0; g < KB; g += 4) {                // groups of four K blocks, whose scales came together
          const int end = min(g + 4, KB);
          ok = __all_sync(0xffffffffu, wait_for(&sfull[slot], rphase, ctl, kWhereEpilogue));
          if (!ok) break;
          if (any_wide(wide, slot)) {                    // 16 columns at a time
            float sum[(NC + 31) / 32 * 32];
#pragma unroll
            for (int c = 0; c < (NC + 31) / 32 * 32; ++c) sum[c] = acc[c];
            for (int kb = g; kb < end; ++kb) {
              ok = __all_sync(0xffffffffu, wait_for(&accf[buf], aphase, ctl, kWhereEpilogue + 1));
              if (!ok) break;
              tc_fence_after();
              const float* sc = reinterpret_cast<const float*>(smem + C::ring + (slot * 4 + kb - g) * C::kRowBytes);
#pragma unroll 1
              for (int c = 0; c < NC; c += 16) {
                const uint32_t t = t_acc + buf * acc_cols + c;
                uint32_t r[16];
                if constexpr (QROW) {
                  tmem_ld_frag16(t, r);
                  tmem_ld_frag16(t + (16u << 16), r + 8);
                } else {
                  tmem_ld<16>(t, r);
                }
                tmem_ld_wait();
                if (c + 16 == NC) {
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) hand_back(acce0 + buf * 8);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float sp, sq;
                  int at;                // in sum, as the ordinary loop has its columns in acc
                  if constexpr (QROW) {  // i = 8 (row / 16) + 4 (column / 8) + 2 (row / 8 % 2) + column % 2
                    const int col = c + (i >> 2 & 1) * 8 + 2 * (lane & 3) + (i & 1);
                    sp = sc[q * 32 + (i >> 3) * 16 + (i >> 1 & 1) * 8 + (lane >> 2)];
                    sq = sc[BM + c0 + col];
                    at = (c & ~31) + (i >> 3) * 16 + (c & 16) / 2 + (i & 7);
                  } else {
                    sp = sc[q * 32 + lane];
                    sq = sc[BM + (c0 >> 7)];
                    at = c + i;
                  }
                  sum[at] = add_scaled(__uint_as_float(r[i]), sp, sq, sum[at]);
                }
              }
              if (++buf == na) { buf = 0; aphase ^= 1; }
            }
#pragma unroll
            for (int c = 0; c < (NC + 31) / 32 * 32; ++c) acc[c] = sum[c];
          } else {
            for (int kb = g; kb < end; ++kb) {
              const float* sc = reinterpret_cast<const float*>(smem + C::ring + (slot * 4 + kb - g) * C::kRowBytes);
              float sp[QROW ? 4 : 1];
              if constexpr (QROW) {
#pragma unroll
                for (int h = 0; h < 4; ++h) sp[h] = sc[q * 32 + 8 * h + (lane >> 2)];
              } else {
                sp[0] = sc[q * 32 + lane] * sc[BM + (c0 >> 7)];   // bn is 128 or 256: one block of 128 columns
              }
              ok = __all_sync(0xffffffffu, wait_for(&accf[buf], aphase, ctl, kWhereEpilogue + 1));
              if (!ok) break;
              tc_fence_after();
              uint32_t r[2][32];
              load(0, r[0]);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < (NC + 31) / 32; ++i) {
                if (i + 1 < (NC + 31) / 32) {
                  load((i + 1) * 32, r[(i + 1) & 1]);
                } else {                             // everything is read: the buffer may be overwritten
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) hand_back(acce0 + buf * 8);
                }
                const uint32_t(&v)[32] = r[i & 1];
                float* a = acc + i * 32;
                if constexpr (QROW) {
                  // 8 bytes of column scales serve four rows: with a row to a lane, every lane would read all
                  // columns' scales, and shared memory returns 128 bytes a clock whether they differ or not
#pragma unroll
                  for (int j = 0; j < (i * 32 + 32 <= NC ? 4 : 2); ++j) {
                    const float2 sq = *reinterpret_cast<const float2*>(sc + BM + c0 + i * 32 + 8 * j + 2 * (lane & 3));
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                      const int e = (h >> 1) * 16 + 4 * j + 2 * (h & 1);
                      a[e] = fmaf(__uint_as_float(v[e]), sp[h] * sq.x, a[e]);
                      a[e + 1] = fmaf(__uint_as_float(v[e + 1]), sp[h] * sq.y, a[e + 1]);
                    }
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 32; ++j) a[j] = fmaf(__uint_as_float(v[j]), sp[0], a[j]);
                }
                if (i + 1 < (NC + 31) / 32) tmem_ld_wait();
              }
              if (++buf == na) { buf = 0; aphase ^= 1; }
            }
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[slot]);
          if (++slot == kSfSlots) { slot = 0; rphase ^= 1; }
        }
        if (!ok) break;
      }
      const int row = tp * 256 + rank * BM + q * 32, col = tq * bn + c0;   // P row of lane 0, Q row of column 0
      const int rows = p.p_rows - row;
#pragma unroll
      for (int c = 0; c < NC; c += 32) {
        const int cols = min(nc - c, p.q_rows - col - c);
        if (cols > 0) {
          if constexpr (!MX && QROW)
            store_frags(p, obuf, acc + c, row, col + c, rows, cols, lane);
          else
            store_rows(p, obuf, acc + c, row, col + c, rows, cols, lane);
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  cluster_sync();                      // no CTA leaves while its peer may still touch its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ small kernel
// What bounds it: 1 x 7168 x 2048 6.9 us, of which 2.3 are the weights at full bandwidth; the rest is the launch, the first
// loads' latency and adding up the split.  1 x 7168 x 7168 12.5 us, 4.1 TB/s.  512 x 4096 x 7168 UE8M0 18.7 us, 1.6
// PFLOP/s: a 128 x 128 tile moves 64 KB through shared memory per K block, as long as its MMAs take, on 128 of the SMs.
template <int BN, bool MX>
__global__ void __launch_bounds__(kSmallThreads, 1)
    gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                          const Fp8Args p) {
  using C = Cfg<BN, MX>;
  constexpr int ST = C::kStages, NA = C::kAcc, COLS = C::kCols, CH = COLS < 32 ? COLS : 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the same offset in every CTA of a cluster: dynamic shared memory starts at one address everywhere
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::bars);
  uint64_t* empty = full + ST;
  uint64_t* accf = empty + ST;
  uint64_t* acce = accf + NA;
  uint64_t* sfull = acce + NA;
  uint64_t* sempty = sfull + kSfSlots;
  uint64_t* drain = sempty + kSfSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc + 4);
  uint8_t* wide = smem + C::misc + 8;                             // fp32 scales: [slot][scale warp]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl ctl{abort_flag, p.status, p.timeout_ns};

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NA; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 8);
    }
    for (int i = 0; i < kSfSlots; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], MX ? 1 : 8);   // the copies to TMEM, or the epilogue warps
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *reinterpret_cast<uint32_t*>(wide) = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  griddep_wait();                      // nothing above touches global memory
  if (warp == 1) {                     // TMEM after the wait, the trigger after both, as in the pair kernel
    tmem_alloc(tmem_slot, C::kTmem);
    tmem_relinquish();
    tc_fence_before();
  }
  if (blockIdx.x == 0 && threadIdx.x < 4) p.status[threadIdx.x] = 0;   // long before any wait can expire
  __syncthreads();
  griddep_launch_dependents();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int S = p.splits, rank = blockIdx.x % S;
  const int tiles = p.tiles_p * p.tiles_q, step = gridDim.x / S;
  // this CTA's K blocks: whole groups of four, whose scales load together
  const int groups = (p.KB + 3) / 4;
  const int kb0 = groups * rank / S * 4, kb1 = min(p.KB, groups * (rank + 1) / S * 4);

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, fills = 0;
      bool ok = true;
      for (int tile = blockIdx.x / S; tile < tiles && ok; tile += step) {
        int tp, tq;
        tile_coord(p, tile, tp, tq);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait_for(&empty[stage], phase ^ 1, ctl, kWhereProducer);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[stage], kPBytes + C::kQBytes);
          tma_load_2d(smem + C::p + stage * kPBytes, &tmP, kb * BK, tp * BM, &full[stage]);
          tma_load_2d(smem + C::q + stage * C::kQBytes, &tmQ, kb * BK, tq * BN, &full[stage]);
          ++fills;
          if (++stage == ST) { stage = 0; phase ^= 1; }
        }
      }
      for (int s = 0; s < ST; ++s) {   // our own copies, before the CTA may exit (complete unless aborted)
        const uint32_t n = (fills + ST - 1 - s) / ST;
        if (n > 0 && !mbar_wait_drain(&full[s], (n - 1) & 1, p.timeout_ns))
          report_status(p.status, kStatusTimeout, kWhereDrain, s);
      }
    }
  } else if (warp == 1) {
    if (elect()) {                     // one thread; elected, so that the compiler keeps the operands uniform
      const uint64_t dp0 = sw128(smem_u32(smem + C::p)), dq0 = sw128(smem_u32(smem + C::q));
      const uint64_t sp0 = sf_desc(smem_u32(smem + C::sfp)), sq0 = sf_desc(smem_u32(smem + C::sfq));
      int stage = 0, buf = 0, sf = 0;
      uint32_t phase = 0, aphase = 0, sphase = 0, tsp = 0;
      bool ok = true;
      for (int tile = blockIdx.x / S; tile < tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          const int j = kb & 3;                  // kb0 is a multiple of four
          if ((!MX || kb == kb0) && !wait_for(&acce[buf], aphase ^ 1, ctl, kWhereMma)) { ok = false; break; }
          if (MX && j == 0) {
            if (!wait_for(&sfull[sf], sphase, ctl, kWhereMma + 2)) { ok = false; break; }
            tc_fence_after();
            tsp = tmem + C::kSfCol + sf * 16;    // the slots' columns alternate as well
            tc_cp_32x128b_warpx4(tsp, sp0 + sf * (512 >> 4));
            tc_cp_32x128b_warpx4(tsp + 4, sq0 + sf * (C::kSfq >> 4));
            tc_commit(&sempty[sf]);
            if (++sf == kSfSlots) { sf = 0; sphase ^= 1; }
          }
          if (!wait_for(&full[stage], phase, ctl, kWhereMma + 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t acc = tmem + buf * BN;
          const uint64_t dp = dp0 + stage * (kPBytes >> 4), dq = dq0 + stage * (C::kQBytes >> 4);
          if constexpr (MX) {
            const uint32_t id = with_byte(p.idesc, j);
#pragma unroll
            for (int i = 0; i < 4; ++i) tc_mma_mxf8f6f4(acc, dp + 2 * i, dq + 2 * i, id, tsp, tsp + 4, (kb > kb0) | i);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) tc_mma_f8f6f4(acc, dp + 2 * i, dq + 2 * i, p.idesc, i);
          }
          tc_commit(&empty[stage]);
          if (!MX || kb == kb1 - 1) {
            tc_commit(&accf[buf]);
            if (++buf == NA) { buf = 0; aphase ^= 1; }
          }
          if (++stage == ST) { stage = 0; phase ^= 1; }
        }
      }
      tc_commit(drain);
      if (!mbar_wait_drain(drain, 0, p.timeout_ns)) report_status(p.status, kStatusTimeout, kWhereDrain, 99);
    }
  } else if (warp == 10) {
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x / S; tile < tiles && ok; tile += step) {
      int tp, tq;
      tile_coord(p, tile, tp, tq);
      ScaleLoader<MX, 0, MX ? 8 : 4 + (BN + 31) / 32, true> sf;
      sf.begin(p, tp * BM, tq * BN, BN, lane, kb0);
      sf.load(p, kb1 - kb0);
      for (int kb = kb0; kb < kb1; kb += 4) {
        ok = __all_sync(0xffffffffu, wait_for(&sempty[slot], phase ^ 1, ctl, kWhereScales));
        if (!ok) break;
        if constexpr (MX)
          sf.store_atoms(smem + C::sfp + slot * 512, smem + C::sfq + slot * C::kSfq, lane);
        else
          sf.store_rows(smem + C::ring + slot * 4 * C::kRowBytes, C::kRowBytes, wide + slot * 2, lane);
        if (lane == 0) mbar_arrive(&sfull[slot]);
        sf.load(p, kb1 - kb - 4);
        if (++slot == kSfSlots) { slot = 0; phase ^= 1; }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..9)
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* obuf = smem + C::staging + (warp - 2) * 2048;
    const uint32_t t_acc = tmem + half * COLS + ((uint32_t)(q * 32) << 16);
    int buf = 0, slot = 0;
    uint32_t aphase = 0, rphase = 0;
    bool ok = true;
    for (int tile = blockIdx.x / S; tile < tiles; tile += step) {
      int tp, tq;
      tile_coord(p, tile, tp, tq);
      float acc[COLS];
      if constexpr (MX) {
        ok = __all_sync(0xffffffffu, wait_for(&accf[buf], aphase, ctl, kWhereEpilogue));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < COLS; c += CH)
          tmem_ld<CH>(t_acc + buf * BN + c, reinterpret_cast<uint32_t*>(acc + c));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acce[buf]);
        if (++buf == NA) { buf = 0; aphase ^= 1; }
      } else {
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[c] = 0.f;
        for (int g = kb0; g < kb1; g += 4) {             // groups of four K blocks, whose scales came together
          const int end = min(g + 4, kb1);
          ok = __all_sync(0xffffffffu, wait_for(&sfull[slot], rphase, ctl, kWhereEpilogue));
          if (!ok) break;
          if (any_wide(wide, slot)) {                    // 8 columns at a time
            float sum[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) sum[c] = acc[c];
            for (int kb = g; kb < end; ++kb) {
              ok = __all_sync(0xffffffffu, wait_for(&accf[buf], aphase, ctl, kWhereEpilogue + 1));
              if (!ok) break;
              tc_fence_after();
              const float* sc = reinterpret_cast<const float*>(smem + C::ring + (slot * 4 + kb - g) * C::kRowBytes);
              const float sp = sc[q * 32 + lane];
#pragma unroll 1
              for (int c = 0; c < COLS; c += 8) {
                uint32_t r[8];
                tmem_ld<8>(t_acc + buf * BN + c, r);
                tmem_ld_wait();
                if (c + 8 == COLS) {
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&acce[buf]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  sum[c + i] = add_scaled(__uint_as_float(r[i]), sp, sc[BM + half * COLS + c + i], sum[c + i]);
              }
              if (++buf == NA) { buf = 0; aphase ^= 1; }
            }
#pragma unroll
            for (int c = 0; c < COLS; ++c) acc[c] = sum[c];
          } else {
            for (int kb = g; kb < end; ++kb) {
              ok = __all_sync(0xffffffffu, wait_for(&accf[buf], aphase, ctl, kWhereEpilogue + 1));
              if (!ok) break;
              tc_fence_after();
              const float* sc = reinterpret_cast<const float*>(smem + C::ring + (slot * 4 + kb - g) * C::kRowBytes);
              const float sp = sc[q * 32 + lane];
#pragma unroll
              for (int c = 0; c < COLS; c += CH) {
                uint32_t r[CH];
                tmem_ld<CH>(t_acc + buf * BN + c, r);
                tmem_ld_wait();
                if (c + CH == COLS) {      // everything is read: the buffer may be overwritten
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&acce[buf]);
                }
#pragma unroll
                for (int j = 0; j < CH; j += 4) {
                  const float4 s4 = *reinterpret_cast<const float4*>(sc + BM + half * COLS + c + j);
                  acc[c + j] += __uint_as_float(r[j]) * (sp * s4.x);
                  acc[c + j + 1] += __uint_as_float(r[j + 1]) * (sp * s4.y);
                  acc[c + j + 2] += __uint_as_float(r[j + 2]) * (sp * s4.z);
                  acc[c + j + 3] += __uint_as_float(r[j + 3]) * (sp * s4.w);
                }
              }
              if (++buf == NA) { buf = 0; aphase ^= 1; }
            }
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[slot]);
          if (++slot == kSfSlots) { slot = 0; rphase ^= 1; }
        }
        if (!ok) break;
      }
      const int row = tp * BM + q * 32;          // P row of lane 0
      const int col = tq * BN + half * COLS;     // Q row of accumulator column 0
      if (S > 1) {
        // partial tile in the order of the output: [column][row] swapped, [row][column] otherwise; the pitch
        // puts neighbouring lanes on other banks
        float* part = reinterpret_cast<float*>(smem);
        if (p.swap) {
#pragma unroll
          for (int c = 0; c < COLS; ++c) part[(half * COLS + c) * (BM + 4) + q * 32 + lane] = acc[c];
        } else {
#pragma unroll
          for (int c = 0; c < COLS; c += 4)
            *reinterpret_cast<float4*>(part + (q * 32 + lane) * (BN + 4) + half * COLS + c) =
                make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
        }
      } else if (p.swap) {
        if (row + lane < p.p_rows) {
#pragma unroll
          for (int c = 0; c < COLS; ++c)
            if (col + c < p.q_rows) put_out(p, col + c, row + lane, acc[c]);
        }
      } else if constexpr (COLS >= 32) {
        const int rows = p.p_rows - row;
#pragma unroll
        for (int c = 0; c < COLS; c += 32)
          if (col + c < p.q_rows) store_rows(p, obuf, acc + c, row, col + c, rows, p.q_rows - col - c, lane);
      }
    }
  }
  __syncwarp();
  if (S > 1) {
    cluster_sync();                    // every rank's partial tile is in its shared memory
    if (warp >= 2 && warp < 10) {
      int tp, tq;
      tile_coord(p, blockIdx.x / S, tp, tq);
      uint32_t base[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) base[r] = mapa_shared(smem, r < S ? r : 0);
      // this rank's share of the tile's outer side (output rows); four consecutive outputs a thread
      const int inner = p.swap ? BM : BN, outer = (p.swap ? BN : BM) / S;
      const long m0 = p.swap ? (long)tq * BN : (long)tp * BM, n0 = p.swap ? (long)tp * BM : (long)tq * BN;
      const int m_end = p.swap ? p.q_rows : p.p_rows, n_end = p.swap ? p.p_rows : p.q_rows;
      const int quads = inner / 4;
#pragma unroll 2
      for (int i = threadIdx.x - 64; i < outer * quads; i += 256) {
        const int o = rank * outer + i / quads, c = (i % quads) * 4;
        const uint32_t at = (uint32_t)(o * (inner + 4) + c) * 4;
        float4 w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < S) w[k] = ld_cluster_f4(base[k] + at);
        float4 v = w[0];
#pragma unroll
        for (int k = 1; k < 8; ++k)
          if (k < S) {
            v.x += w[k].x;
            v.y += w[k].y;
            v.z += w[k].z;
            v.w += w[k].w;
          }
        if (m0 + o < m_end) put_out4(p, m0 + o, n0 + c, v, n_end);
      }
    }
    __syncwarp();
    cluster_sync();                    // no rank leaves while another reads its part
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// ------------------------------------------------------------------ host
bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

using Kernel = void (*)(CUtensorMap, CUtensorMap, Fp8Args);
struct Launch {
  Kernel fn;
  uint32_t smem;
  int threads, slot;
};

template <bool MX>
Launch small_of(int bn) {
  switch (bn) {
    case 16: return {gemm_fp8_small_kernel<16, MX>, Cfg<16, MX>::bytes, kSmallThreads, MX};
    case 32: return {gemm_fp8_small_kernel<32, MX>, Cfg<32, MX>::bytes, kSmallThreads, 2 + MX};
    case 64: return {gemm_fp8_small_kernel<64, MX>, Cfg<64, MX>::bytes, kSmallThreads, 4 + MX};
    default: return {gemm_fp8_small_kernel<128, MX>, Cfg<128, MX>::bytes, kSmallThreads, 6 + MX};
  }
}
Launch pair_of(bool mx, bool qrow, int bn) {
  if (mx) return {gemm_fp8_pair_kernel<true, false, 128>, PairCfg<true>::bytes, kPairThreads, 8};
  if (bn == 256)
    return qrow ? Launch{gemm_fp8_pair_kernel<false, true, 128>, PairCfg<false>::bytes, kPairThreads, 9}
                : Launch{gemm_fp8_pair_kernel<false, false, 128>, PairCfg<false>::bytes, kPairThreads, 10};
  if (bn == 224) return {gemm_fp8_pair_kernel<false, true, 112>, PairCfg<false>::bytes, kPairThreads, 13};
  return qrow ? Launch{gemm_fp8_pair_kernel<false, true, 64>, PairCfg<false>::bytes, kPairThreads, 11}
              : Launch{gemm_fp8_pair_kernel<false, false, 64>, PairCfg<false>::bytes, kPairThreads, 12};
}

// The device's SM count, 0 if it is no sm_100, -1 on an error; shared-memory limits raised once.
constexpr int kMaxDevices = 64;
std::mutex g_mutex;
int g_sms[kMaxDevices] = {};
bool g_ready[kMaxDevices][14] = {};

int device_sms(int* device) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return -1;
  *device = dev;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (dev < kMaxDevices && g_sms[dev] > 0) return g_sms[dev];
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  if (major != 10 || minor != 0) return 0;
  if (dev < kMaxDevices) g_sms[dev] = sms;
  return sms;
}

cudaError_t launch(const Launch& l, int device, const CUtensorMap& tp, const CUtensorMap& tq, const Fp8Args& a, int grid,
                   cudaStream_t s) {
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (device >= kMaxDevices || !g_ready[device][l.slot]) {
      const cudaError_t e = cudaFuncSetAttribute(l.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)l.smem);
      if (e != cudaSuccess) return e;
      if (device < kMaxDevices) g_ready[device][l.slot] = true;
    }
  }
  return launch_dependent(l.fn, dim3(grid), l.threads, l.smem, a.splits, s, tp, tq, a);   // the pair kernel has its own pairs
}

// How a product is cut into tiles.
struct Cut {
  bool pair, swap;
  int bn, splits;
};

int up(long a, long b) { return (int)((a + b - 1) / b); }

// The cut with the least estimated time.  The estimates (microseconds) are a straight line through what the
// kernels measured on B200 for a K block (128 deep) of one tile, at K of 2048 to 8192:
//   pair    UE8M0 256 columns 0.45, 128 columns 0.29; fp32 0.57 and 0.35, column scales 0.82 and 0.53; 2 to start
//   small   UE8M0 0.25 to 0.30, fp32 0.26 to 0.50; adding up a split tile 1.5 and its size
// and not less than reading both operands once at 6.2 TB/s.  M = 256, N = 7168, K = 2048, UE8M0: small 8.7, pair
// 11.2 us; M = 8192, N = 4096, K = 7168: pair 170, single CTAs of 256 columns 226 us; M = 1, N = 7168, K = 2048:
// split in two 7.2, not split 8.3 us.
Cut choose(int M, int N, int KB, int sms, bool qrow, bool mx) {
  Cut best{false, M <= 128, 128, 1};
  double least = 1e30;
  const double memory = ((double)M + N) * KB * 128 / 6.2e6;
  auto offer = [&](const Cut& c, double blocks, double block_us, double more) {
    const double busy = blocks * block_us, t = (busy > memory ? busy : memory) + more;
    if (t < least) {
      least = t;
      best = c;
    }
  };
  // small: few tokens as columns (swapped), or 128 x 128 tiles
  static const double kMx[4] = {0.245, 0.245, 0.262, 0.300}, kF32[4] = {0.256, 0.260, 0.349, 0.500};
  const bool swap = M <= 128;
  for (int i = swap ? 0 : 3, bn = swap ? 16 : 128; bn <= 128; bn *= 2, ++i) {
    const long tiles = (long)up(swap ? N : M, 128) * up(swap ? M : N, bn);
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && (tiles * s > sms || KB < s * 4)) break;         // every part a group of four blocks at least
      offer(Cut{false, swap, bn, s}, (double)((tiles * s + sms - 1) / sms) * up(KB, s), mx ? kMx[i] : kF32[i],
            s > 1 ? 1.5 + 0.012 * bn : 0.0);
    }
  }
  if (!swap)
    for (int bn = 256; bn >= 64; bn -= 32) {
      // the widths compiled for fp32 scales.  224, column scales: 4096 x 7168 x 8191 is 512 tiles, 6.9 waves, 338 us; with
      // 256 columns 448 tiles in 6.05 waves, 361 us.  Scales per 128 columns need tiles that start with them
      if (!mx && bn != 256 && bn != 128 && !(qrow && bn == 224)) continue;
      const double waves = (double)up((long)up(M, 256) * up(N, bn), sms / 2);
      const double block = mx ? 0.130 + 0.00124 * bn : qrow ? 0.231 + 0.0023 * bn : 0.131 + 0.00172 * bn;
      offer(Cut{true, false, bn, 1}, waves * KB, block, 2.0 + 0.3 * waves);
    }
  return best;
}

}  // namespace

extern "C" {

size_t moe_gemm_fp8_workspace_bytes(void) { return 256; }

int moe_gemm_fp8(int M, int N, int K, const void* A, long long lda, int a_format, const void* A_scales,
                 long long as_row_stride, long long as_block_stride, int a_scale_rows, const void* B, long long ldb,
                 int b_format, const void* B_scales, long long bs_row_stride, long long bs_block_stride,
                 int b_scale_rows, int scale_type, void* out, long long ldo, int out_type, int accumulate,
                 void* workspace, size_t workspace_bytes, void* stream) {
  // row and column numbers of the last tile stay in 32 bits; a K loop ends well inside the wait limit
  if (M < 0 || N < 0 || K < 0 || M > (1 << 30) || N > (1 << 30) || K > (1 << 28)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((a_format != MOE_FP8_E4M3 && a_format != MOE_FP8_E5M2) || (b_format != MOE_FP8_E4M3 && b_format != MOE_FP8_E5M2) ||
      (scale_type != MOE_SCALE_FP32 && scale_type != MOE_SCALE_UE8M0) ||
      (out_type != MOE_TYPE_BF16 && out_type != MOE_TYPE_FP32) || (accumulate && out_type != MOE_TYPE_FP32) ||
      (a_scale_rows != 1 && a_scale_rows != 128) || (b_scale_rows != 1 && b_scale_rows != 128))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || workspace_bytes < moe_gemm_fp8_workspace_bytes()) return MOE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = out_type == MOE_TYPE_FP32;
  const size_t osize = f32 ? 4 : 2;
  if (M > 0 && N > 0 && (!aligned(out, osize) || (M > 1 && ldo < N))) return MOE_ERR_INVALID_ARG;
  if (M == 0 || N == 0 || K == 0) {
    if (cudaMemsetAsync(workspace, 0, 16, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (M == 0 || N == 0 || accumulate) return MOE_OK;
    return cudaMemset2DAsync(out, (M > 1 ? ldo : N) * osize, 0, N * osize, M, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  const uintptr_t ssize = scale_type == MOE_SCALE_FP32 ? 4 : 1;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(A_scales, ssize) || !aligned(B_scales, ssize) ||
      (M > 1 && (lda < K || lda % 16)) || (N > 1 && (ldb < K || ldb % 16)) || as_row_stride < 0 ||
      as_block_stride < 0 || bs_row_stride < 0 || bs_block_stride < 0)
    return MOE_ERR_INVALID_ARG;
  if ((long long)((M + 127) / 128) * ((N + 15) / 16) > (1ll << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  int device = 0;
  const int sms = device_sms(&device);
  if (sms < 0) return MOE_ERR_CUDA;
  if (sms == 0) return MOE_ERR_UNSUPPORTED_SHAPE;   // built for sm_100a only
  const bool mx = scale_type == MOE_SCALE_UE8M0;

  Fp8Args a{};
  a.KB = up(K, 128);
  const Cut c = choose(M, N, a.KB, sms, b_scale_rows == 1, mx);
  a.swap = c.swap;
  a.splits = c.splits;
  a.bn = c.bn;
  a.p_rows = a.swap ? N : M;
  a.q_rows = a.swap ? M : N;
  a.tiles_p = up(a.p_rows, c.pair ? 256 : 128);
  a.tiles_q = up(a.q_rows, c.bn);
  a.sp = a.swap ? B_scales : A_scales;
  a.sp_row = a.swap ? bs_row_stride : as_row_stride;
  a.sp_blk = a.swap ? bs_block_stride : as_block_stride;
  a.sp_shift = (a.swap ? b_scale_rows : a_scale_rows) == 128 ? 7 : 0;
  a.sq = a.swap ? A_scales : B_scales;
  a.sq_row = a.swap ? as_row_stride : bs_row_stride;
  a.sq_blk = a.swap ? as_block_stride : bs_block_stride;
  a.sq_shift = (a.swap ? a_scale_rows : b_scale_rows) == 128 ? 7 : 0;
  const uintptr_t quad = 4 * ssize;
  a.sp_quad = a.sp_blk == 1 && a.sp_row % 4 == 0 && aligned(a.sp, quad);
  a.sq_quad = a.sq_blk == 1 && a.sq_row % 4 == 0 && aligned(a.sq, quad);
  a.out = out;
  a.ldo = M > 1 ? ldo : N;
  a.out_fp32 = f32;
  a.accumulate = accumulate != 0;
  a.vec = aligned(out, 16) && (M == 1 || ldo * (long long)osize % 16 == 0);
  const uint32_t fp = a.swap ? b_format : a_format, fq = a.swap ? a_format : b_format;
  const int mma_m = c.pair ? 256 : 128;
  a.idesc = mx ? idesc_mxf8f6f4(mma_m, c.bn, 0, 0, fp, fq) : idesc_f8f6f4(mma_m, c.bn, fp, fq);
  a.status = static_cast<uint32_t*>(workspace);
  a.timeout_ns = 2000000000ull;

  const uint64_t one = ((uint64_t)K + 15) / 16 * 16, pitch_a = M > 1 ? lda : one, pitch_b = N > 1 ? ldb : one;
  CUtensorMap tp, tq;
  if (encode_2d(&tp, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.swap ? B : A, K, a.p_rows, a.swap ? pitch_b : pitch_a, BK, BM) != MOE_OK ||
      encode_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.swap ? A : B, K, a.q_rows, a.swap ? pitch_a : pitch_b, BK,
                c.pair ? c.bn / 2 : c.bn) != MOE_OK)
    return MOE_ERR_CUDA;
  const int tiles = a.tiles_p * a.tiles_q;
  const int grid = c.pair ? 2 * (tiles < sms / 2 ? tiles : sms / 2) : c.splits > 1 ? tiles * c.splits : tiles < sms ? tiles : sms;
  const Launch l = c.pair ? pair_of(mx, a.sq_shift == 0, c.bn) : mx ? small_of<true>(c.bn) : small_of<false>(c.bn);
  return launch(l, device, tp, tq, a, grid, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
