// Block-scaled FP8 x FP8 matrix product (moe_gemm_fp8) on tcgen05.
//
//   out[m][n] (+)= sum_b sA(m, b) sB(n, b) sum_{k in block b of 128} A[m][k] B[n][k]
//
// One operand ("P") is the MMA's 128-row side, the other ("Q") its column side of BN columns.  With many
// tokens P = A; with few (M <= 128) the roles swap, P = B: the weight rows fill the 128 lanes and BN
// shrinks to the tokens, so that each weight byte is read once and little is multiplied by padding.
//
//   warp 0      TMA producer: per 128-deep K block the P tile (128 x 128 B) and the Q tile (BN x 128 B),
//               128-byte swizzle; codes past the matrix arrive as zeros
//   warp 1      MMA issuer (one thread)
//   warps 2..9  epilogue: TMEM lane quarter warp % 4, half of the columns each
//   warp 10     scales
// UE8M0 scales (MX): warp 10 writes each stage's scale atoms, tcgen05.mma.kind::mxf8f6f4 applies them and
// the accumulator stays in TMEM over the whole K loop.  fp32 scales: each K block is one kind::f8f6f4
// product into a TMEM buffer of its own, and the epilogue warps add it, scaled, to accumulators in
// registers while the next block's MMAs run; warp 10 brings the scales in through a ring with cp.async.
// A tile whose K loop is split over a cluster's CTAs is added up in rank order through distributed
// shared memory: no workspace, no atomics.
// Every wait is bounded (WaitCtl); on a timeout the CTA records MOE_ERR_DEVICE_TIMEOUT, drains its own
// copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/moe_b200.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int BM = 128, BK = 128;
constexpr int kThreads = 352;                 // TMA, MMA, 8 x epilogue, scales
constexpr int kRing = 8;                      // K blocks of fp32 scales in flight
constexpr uint32_t kPBytes = BM * BK;
enum : uint32_t { kWhereProducer = 0xB00, kWhereMma = 0xB10, kWhereEpilogue = 0xB20, kWhereScales = 0xB30,
                  kWhereDrain = 0xB40 };

struct Fp8Args {
  int p_rows, q_rows, KB;
  int tiles_p, tiles_q, splits;
  const void *sp, *sq;               // scales of P and Q
  long sp_row, sp_blk, sq_row, sq_blk;
  int sp_shift, sq_shift;            // 0: per row, 7: per 128 rows
  void* out;
  long ldo;
  int out_fp32, accumulate, swap, vec;
  uint32_t idesc;                    // formats and shape of the MMA
  uint32_t* status;
  uint64_t timeout_ns;
};

template <int BN, bool MX>
struct Cfg {
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : BN == 64 ? 8 : BN == 32 ? 9 : 10;
  static constexpr int kCols = BN / 2;                           // columns per epilogue thread
  static constexpr int kAcc = MX ? (BN == 256 ? 1 : 2) : (BN == 256 ? 2 : 4);   // TMEM accumulators
  static constexpr uint32_t kSfCol = kAcc * BN;                  // MX: scale columns (P 4, Q 4 or 8)
  static constexpr uint32_t kTmem = (kAcc * BN + (MX ? 12 : 0)) <= 64 ? 64
                                    : (kAcc * BN + (MX ? 12 : 0)) <= 128 ? 128
                                    : (kAcc * BN + (MX ? 12 : 0)) <= 256 ? 256 : 512;
  static constexpr uint32_t kQBytes = BN * BK;
  static constexpr uint32_t kSfq = BN > 128 ? 1024 : 512;        // Q scale atoms of a stage
  static constexpr uint32_t p = 0;
  static constexpr uint32_t q = p + kStages * kPBytes;
  static constexpr uint32_t sfp = q + kStages * kQBytes;
  static constexpr uint32_t sfq = sfp + (MX ? kStages * 512 : 0);
  static constexpr uint32_t ring = sfq + (MX ? kStages * kSfq : 0);
  static constexpr uint32_t kRingBytes = (BM + BN) * 4;
  static constexpr uint32_t staging = ring + (MX ? 0 : kRing * kRingBytes);
  static constexpr uint32_t bars = staging + 8 * 2048;
  static constexpr int kBars = 2 * kStages + 2 * kAcc + 2 * kRing + 1;
  static constexpr uint32_t misc = bars + kBars * 8;
  static constexpr uint32_t total = misc + 16;
  static constexpr uint32_t bytes = total + 1024;                // 1024-byte alignment of the stages
  static_assert(bytes <= 232448, "shared memory");
  static_assert(BM * (BN + 0) * 4 + BN * 4 <= sfp, "a partial tile fits over the stages");
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

// 4 bytes global -> shared, zeros when !ok (nothing is read then)
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 4 : 0)
               : "memory");
}
// one arrival on `bar` when this thread's copies so far are complete
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
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

__device__ __forceinline__ void put_out(const Fp8Args& p, long m, long n, float v) {
  if (p.out_fp32) {
    float* o = static_cast<float*>(p.out) + m * p.ldo + n;
    *o = p.accumulate ? *o + v : v;
  } else {
    static_cast<__nv_bfloat16*>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
  }
}

// 64 bytes of each of the warp's 32 rows (lane = row) through the warp's 2 KB buffer, so that stores cover
// whole sectors: 16-byte pieces, 4 lanes to a row, where the row pitch and the columns allow it, else
// element by element.  row0, col0: first row and column; cols: columns of the matrix from col0 on.
__device__ __forceinline__ void store_64b(const Fp8Args& p, uint8_t* buf, const uint4 (&v)[4], long row0, long col0,
                                          int rows, int cols, int lane) {
#pragma unroll
  for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) * 16)) = v[c];
  __syncwarp();
  const int esize = p.out_fp32 ? 4 : 2, n = 64 / esize;
  if (p.vec && cols >= n) {
    uint8_t* dst = static_cast<uint8_t*>(p.out) + (row0 * p.ldo + col0) * esize;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int r = it * 8 + (lane >> 2), c = lane & 3;
      const uint4 w = *reinterpret_cast<const uint4*>(buf + r * 64 + ((c ^ ((r >> 1) & 3)) * 16));
      if (r < rows) {
        uint8_t* d = dst + (long)r * p.ldo * esize + c * 16;
        if (p.accumulate)            // one addition per element and call: the order of them is fixed
          asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(d), "f"(__uint_as_float(w.x)),
                       "f"(__uint_as_float(w.y)), "f"(__uint_as_float(w.z)), "f"(__uint_as_float(w.w))
                       : "memory");
        else
          *reinterpret_cast<uint4*>(d) = w;
      }
    }
  } else {
    for (int i = lane; i < 32 * n; i += 32) {
      const int r = i / n, c = i - r * n, byte = c * esize;
      const uint8_t* at = buf + r * 64 + (((byte >> 4) ^ ((r >> 1) & 3)) * 16) + (byte & 15);
      if (r < rows && c < cols) {
        const long o = (row0 + r) * p.ldo + col0 + c;
        if (p.out_fp32) {
          float* d = static_cast<float*>(p.out) + o;
          const float x = *reinterpret_cast<const float*>(at);
          *d = p.accumulate ? *d + x : x;
        } else {
          static_cast<uint16_t*>(p.out)[o] = *reinterpret_cast<const uint16_t*>(at);
        }
      }
    }
  }
  __syncwarp();
}

// QROW: Q's scales differ by column; otherwise they are one per 128 columns (fp32 scales only).
template <int BN, bool MX, bool QROW>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
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
  uint64_t* rfull = acce + NA;
  uint64_t* rempty = rfull + kRing;
  uint64_t* drain = rempty + kRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl ctl{abort_flag, p.status, p.timeout_ns};

  if (blockIdx.x == 0 && threadIdx.x < 4) p.status[threadIdx.x] = 0;   // long before any wait can expire
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], MX ? 2 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NA; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 8);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&rfull[i], 32);
      mbar_init(&rempty[i], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmem);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int S = p.splits, rank = blockIdx.x % S;
  const int tiles = p.tiles_p * p.tiles_q, step = gridDim.x / S;
  const int kb0 = (int)((long)p.KB * rank / S), kb1 = (int)((long)p.KB * (rank + 1) / S);   // this CTA's K blocks

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, fills = 0;
      bool ok = true;
      for (int tile = blockIdx.x / S; tile < tiles && ok; tile += step) {
        int tp, tq;
        tile_coord(p, tile, tp, tq);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, ctl, kWhereProducer)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[stage], kPBytes + C::kQBytes);
          tma_load_2d(smem + C::p + stage * kPBytes, &tmP, kb * BK, tp * BM, &full[stage]);
          tma_load_2d(smem + C::q + stage * C::kQBytes, &tmQ, kb * BK, tq * BN, &full[stage]);
          ++fills;
          if (++stage == ST) { stage = 0; phase ^= 1; }
        }
      }
      for (int s = 0; s < ST; ++s) {   // our own copies, before the CTA may exit (they are complete unless aborted)
        const uint32_t n = (fills + ST - 1 - s) / ST;
        if (n > 0 && !mbar_wait_drain(&full[s], (n - 1) & 1, p.timeout_ns))
          report_status(p.status, kStatusTimeout, kWhereDrain, s);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, aphase = 0;
      bool ok = true;
      for (int tile = blockIdx.x / S; tile < tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if ((!MX || kb == kb0) && !mbar_wait(&acce[buf], aphase ^ 1, ctl, kWhereMma)) { ok = false; break; }
          if (!mbar_wait(&full[stage], phase, ctl, kWhereMma + 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t acc = tmem + buf * BN;
          const uint32_t pa = smem_u32(smem + C::p + stage * kPBytes), qa = smem_u32(smem + C::q + stage * C::kQBytes);
          if constexpr (MX) {
            const uint32_t sp = smem_u32(smem + C::sfp + stage * 512), sq = smem_u32(smem + C::sfq + stage * C::kSfq);
            const uint32_t tsp = tmem + C::kSfCol, tsq = tsp + 4;
            tc_cp_32x128b_warpx4(tsp, sf_desc(sp));
            tc_cp_32x128b_warpx4(tsq, sf_desc(sq));
            if constexpr (BN > 128) tc_cp_32x128b_warpx4(tsq + 4, sf_desc(sq + 512));
#pragma unroll
            for (int i = 0; i < 4; ++i)   // the four 32-K blocks of a scale share its byte
              tc_mma_mxf8f6f4(acc, sw128(pa + i * 32), sw128(qa + i * 32), p.idesc, tsp, tsq, (kb > kb0) | i);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tc_mma_f8f6f4(acc, sw128(pa + i * 32), sw128(qa + i * 32), p.idesc, i);
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
    if constexpr (MX) {
      // scale atoms: lane l writes the words of rows l, l + 32, l + 64, l + 96 (one byte per 32-K block, all
      // four alike) at l * 16; the bytes of four K blocks are in flight at a time
      constexpr int NR = BN > 128 ? 12 : 8;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint8_t* sp = static_cast<const uint8_t*>(p.sp);
      const uint8_t* sq = static_cast<const uint8_t*>(p.sq);
      for (int tile = blockIdx.x / S; tile < tiles && ok; tile += step) {
        int tp, tq;
        tile_coord(p, tile, tp, tq);
        long at[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int in = lane + 32 * (i < 4 ? i : i - 4);
          const int row = (i < 4 ? tp * BM : tq * BN) + in;
          const bool live = i < 4 ? row < p.p_rows : in < BN && row < p.q_rows;
          at[i] = !live ? -1 : i < 4 ? (long)(row >> p.sp_shift) * p.sp_row : (long)(row >> p.sq_shift) * p.sq_row;
        }
        uint32_t v[4][NR];
        auto load = [&](int kb, uint32_t (&d)[NR]) {
#pragma unroll
          for (int i = 0; i < NR; ++i)   // rows past the matrix: scale 1
            d[i] = at[i] < 0 || kb >= kb1 ? 127u : i < 4 ? __ldg(sp + at[i] + kb * p.sp_blk) : __ldg(sq + at[i] + kb * p.sq_blk);
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) load(kb0 + j, v[j]);
        for (int kb = kb0; kb < kb1 && ok; kb += 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (kb + j < kb1 && ok) {
              ok = mbar_wait(&empty[stage], phase ^ 1, ctl, kWhereScales);
              ok = __all_sync(0xffffffffu, ok);
              if (ok) {
                constexpr uint32_t kRep = 0x01010101u;
                *reinterpret_cast<uint4*>(smem + C::sfp + stage * 512 + lane * 16) =
                    make_uint4(v[j][0] * kRep, v[j][1] * kRep, v[j][2] * kRep, v[j][3] * kRep);
                *reinterpret_cast<uint4*>(smem + C::sfq + stage * C::kSfq + lane * 16) =
                    make_uint4(v[j][4] * kRep, v[j][5] * kRep, v[j][6] * kRep, v[j][7] * kRep);
                if constexpr (BN > 128)
                  *reinterpret_cast<uint4*>(smem + C::sfq + stage * C::kSfq + 512 + lane * 16) =
                      make_uint4(v[j][8] * kRep, v[j][9] * kRep, v[j][10] * kRep, v[j][11] * kRep);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[stage]);
                load(kb + j + 4, v[j]);
                if (++stage == ST) { stage = 0; phase ^= 1; }
              }
            }
          }
        }
      }
    } else {
      constexpr int NQ = QROW ? (BN + 31) / 32 : 1;
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      const float* sp = static_cast<const float*>(p.sp);
      const float* sq = static_cast<const float*>(p.sq);
      for (int tile = blockIdx.x / S; tile < tiles && ok; tile += step) {
        int tp, tq;
        tile_coord(p, tile, tp, tq);
        long ap[4], aq[NQ];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = tp * BM + lane + 32 * i;
          ap[i] = row < p.p_rows ? (long)(row >> p.sp_shift) * p.sp_row : -1;
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const int in = QROW ? lane + 32 * i : lane * 128;
          const int row = tq * BN + in;
          aq[i] = in < BN && row < p.q_rows ? (long)(row >> p.sq_shift) * p.sq_row : -1;
        }
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&rempty[slot], phase ^ 1, ctl, kWhereScales);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          float* d = reinterpret_cast<float*>(smem + C::ring + slot * C::kRingBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            cp_async4(d + lane + 32 * i, ap[i] < 0 ? sp : sp + ap[i] + kb * p.sp_blk, ap[i] >= 0);
#pragma unroll
          for (int i = 0; i < NQ; ++i)
            if (QROW ? lane + 32 * i < BN : lane < BN / 128)
              cp_async4(d + BM + (QROW ? lane + 32 * i : lane), aq[i] < 0 ? sq : sq + aq[i] + kb * p.sq_blk, aq[i] >= 0);
          cp_async_arrive(&rfull[slot]);
          if (++slot == kRing) { slot = 0; phase ^= 1; }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
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
        ok = __all_sync(0xffffffffu, mbar_wait(&accf[buf], aphase, ctl, kWhereEpilogue));
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
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&rfull[slot], rphase, ctl, kWhereEpilogue) && mbar_wait(&accf[buf], aphase, ctl, kWhereEpilogue + 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const float* sc = reinterpret_cast<const float*>(smem + C::ring + slot * C::kRingBytes);
          const float sp = sc[q * 32 + lane];
          const float spq = QROW ? 0.f : sp * sc[BM + (half * COLS) / 128];
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
            if constexpr (QROW) {
#pragma unroll
              for (int j = 0; j < CH; j += 4) {
                const float4 s4 = *reinterpret_cast<const float4*>(sc + BM + half * COLS + c + j);
                acc[c + j] += __uint_as_float(r[j]) * (sp * s4.x);
                acc[c + j + 1] += __uint_as_float(r[j + 1]) * (sp * s4.y);
                acc[c + j + 2] += __uint_as_float(r[j + 2]) * (sp * s4.z);
                acc[c + j + 3] += __uint_as_float(r[j + 3]) * (sp * s4.w);
              }
            } else {
#pragma unroll
              for (int j = 0; j < CH; ++j) acc[c + j] = fmaf(__uint_as_float(r[j]), spq, acc[c + j]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&rempty[slot]);
          if (++buf == NA) { buf = 0; aphase ^= 1; }
          if (++slot == kRing) { slot = 0; rphase ^= 1; }
        }
        if (!ok) break;
      }
      const int row = tp * BM + q * 32;          // P row of lane 0
      const int col = tq * BN + half * COLS;     // Q row of accumulator column 0
      if (S > 1) {
        // partial tile [column][129]: rows of a column next to each other, columns on other banks
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int c = 0; c < COLS; ++c) part[(half * COLS + c) * (BM + 1) + q * 32 + lane] = acc[c];
      } else if (p.swap) {
        if (row + lane < p.p_rows) {
#pragma unroll
          for (int c = 0; c < COLS; ++c)
            if (col + c < p.q_rows) put_out(p, col + c, row + lane, acc[c]);
        }
      } else if constexpr (COLS >= 32) {
        const int rows = p.p_rows - row;
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          if (col + c < p.q_rows) {
            uint4 v[4];
            if (p.out_fp32) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  v[i] = make_uint4(__float_as_uint(acc[c + h + 4 * i]), __float_as_uint(acc[c + h + 4 * i + 1]),
                                    __float_as_uint(acc[c + h + 4 * i + 2]), __float_as_uint(acc[c + h + 4 * i + 3]));
                store_64b(p, obuf, v, row, col + c + h, rows, p.q_rows - col - c - h, lane);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                __nv_bfloat162 b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = __floats2bfloat162_rn(acc[c + 8 * i + 2 * j], acc[c + 8 * i + 2 * j + 1]);
                v[i] = *reinterpret_cast<const uint4*>(b);
              }
              store_64b(p, obuf, v, row, col + c, rows, p.q_rows - col - c, lane);
            }
          }
        }
      }
    }
  }
  __syncwarp();
  if (S > 1) {
    cluster_sync();                    // every rank's partial tile is in its shared memory
    if (warp >= 2 && warp < 10) {
      int tp, tq;
      tile_coord(p, blockIdx.x / S, tp, tq);
      const uint32_t mine = smem_u32(smem);
      uint32_t base[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base[r]) : "r"(mine), "r"(r < S ? r : 0));
      const int t = threadIdx.x - 64;
      // swapped: this rank's columns, lanes along the rows; otherwise its rows, lanes along the columns
      const int n_col = p.swap ? BN / S : BN, n_row = p.swap ? BM : BM / S;
      const int c_base = p.swap ? rank * n_col : 0, r_base = p.swap ? 0 : rank * n_row;
      for (int i = t; i < n_col * n_row; i += 256) {
        const int c = c_base + (p.swap ? i / BM : i % BN), r = r_base + (p.swap ? i % BM : i / BN);
        const int pr = tp * BM + r, qr = tq * BN + c;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < S) v += ld_cluster_f32(base[k] + (uint32_t)(c * (BM + 1) + r) * 4);
        if (pr < p.p_rows && qr < p.q_rows) put_out(p, p.swap ? qr : pr, p.swap ? pr : qr, v);
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

template <int BN, bool MX, bool QROW>
cudaError_t launch(const CUtensorMap& tp, const CUtensorMap& tq, const Fp8Args& a, int grid, cudaStream_t s) {
  using C = Cfg<BN, MX>;
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(gemm_fp8_kernel<BN, MX, QROW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::bytes);
      if (e != cudaSuccess) return e;
      if (dev < 64) done[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, gemm_fp8_kernel<BN, MX, QROW>, tp, tq, a);
}

template <bool MX>
cudaError_t launch_bn(int bn, bool qrow, const CUtensorMap& tp, const CUtensorMap& tq, const Fp8Args& a, int grid,
                      cudaStream_t s) {
  if constexpr (!MX) {
    if (!qrow) return bn == 128 ? launch<128, MX, false>(tp, tq, a, grid, s) : launch<256, MX, false>(tp, tq, a, grid, s);
  }
  switch (bn) {
    case 16: return launch<16, MX, true>(tp, tq, a, grid, s);
    case 32: return launch<32, MX, true>(tp, tq, a, grid, s);
    case 64: return launch<64, MX, true>(tp, tq, a, grid, s);
    case 128: return launch<128, MX, true>(tp, tq, a, grid, s);
    default: return launch<256, MX, true>(tp, tq, a, grid, s);
  }
}

}  // namespace

extern "C" {

size_t moe_gemm_fp8_workspace_bytes(void) { return 256; }

int moe_gemm_fp8(int M, int N, int K, const void* A, long long lda, int a_format, const void* A_scales,
                 long long as_row_stride, long long as_block_stride, int a_scale_rows, const void* B, long long ldb,
                 int b_format, const void* B_scales, long long bs_row_stride, long long bs_block_stride,
                 int b_scale_rows, int scale_type, void* out, long long ldo, int out_type, int accumulate,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0) return MOE_ERR_UNSUPPORTED_SHAPE;
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
  int dev = -1, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return MOE_ERR_CUDA;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major != 10 || minor != 0) return MOE_ERR_UNSUPPORTED_SHAPE;   // built for sm_100a only
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MOE_ERR_CUDA;
  const bool mx = scale_type == MOE_SCALE_UE8M0;

  Fp8Args a{};
  a.swap = M <= 128;
  int bn = !a.swap ? 256 : M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  a.KB = (K + 127) / 128;
  a.p_rows = a.swap ? N : M;
  a.q_rows = a.swap ? M : N;
  a.tiles_p = (a.p_rows + 127) / 128;
  if (!a.swap && (long)a.tiles_p * ((N + 255) / 256) * 4 <= sms) bn = 128;
  a.tiles_q = (a.q_rows + bn - 1) / bn;
  if ((long)a.tiles_p * a.tiles_q > (1l << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const int tiles = a.tiles_p * a.tiles_q;
  a.splits = 1;
  while (a.splits < 8 && tiles * a.splits * 2 <= sms && a.KB >= a.splits * 4) a.splits *= 2;
  const bool qrow = bn < 128 || (a.swap ? a_scale_rows : b_scale_rows) == 1;
  a.sp = a.swap ? B_scales : A_scales;
  a.sp_row = a.swap ? bs_row_stride : as_row_stride;
  a.sp_blk = a.swap ? bs_block_stride : as_block_stride;
  a.sp_shift = (a.swap ? b_scale_rows : a_scale_rows) == 128 ? 7 : 0;
  a.sq = a.swap ? A_scales : B_scales;
  a.sq_row = a.swap ? as_row_stride : bs_row_stride;
  a.sq_blk = a.swap ? as_block_stride : bs_block_stride;
  a.sq_shift = (a.swap ? a_scale_rows : b_scale_rows) == 128 ? 7 : 0;
  a.out = out;
  a.ldo = M > 1 ? ldo : N;
  a.out_fp32 = f32;
  a.accumulate = accumulate != 0;
  a.vec = aligned(out, 16) && (M == 1 || ldo * (long long)osize % 16 == 0);
  const uint32_t fp = a.swap ? b_format : a_format, fq = a.swap ? a_format : b_format;
  a.idesc = mx ? idesc_mxf8f6f4(BM, bn, 0, 0, fp, fq) : idesc_f8f6f4(BM, bn, fp, fq);
  a.status = static_cast<uint32_t*>(workspace);
  a.timeout_ns = 2000000000ull;

  const uint64_t pitch_a = M > 1 ? lda : ((uint64_t)K + 15) / 16 * 16, pitch_b = N > 1 ? ldb : ((uint64_t)K + 15) / 16 * 16;
  CUtensorMap tp, tq;
  if (encode_2d(&tp, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.swap ? B : A, K, a.p_rows, a.swap ? pitch_b : pitch_a, BK, BM) != MOE_OK ||
      encode_2d(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.swap ? A : B, K, a.q_rows, a.swap ? pitch_a : pitch_b, BK, bn) != MOE_OK)
    return MOE_ERR_CUDA;
  const int grid = a.splits > 1 ? tiles * a.splits : tiles < sms ? tiles : sms;
  const cudaError_t e = mx ? launch_bn<true>(bn, qrow, tp, tq, a, grid, s) : launch_bn<false>(bn, qrow, tp, tq, a, grid, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
