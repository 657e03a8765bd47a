// dflash_gemm_fp4: out[m][n] = sum_k X[m][k] W[n][k] of two microscaled 4-bit
// matrices, on tcgen05's block-scaled path: codes and scales go to the matrix
// unit as they are, which multiplies them exactly and sums in fp32.
//
// A tile is 128 rows of W (the MMA's M: out's columns) x BN rows of X (its N).
// 256 k are a stage of a shared-memory ring: 128-byte rows of codes, swizzled,
// and the scale tiles, which tcgen05.cp puts into TMEM beside the accumulators
// in front of the stage's four MMAs.  BN, the number of CTAs that share a
// tile's k (a cluster; its partial sums meet in shared memory, added in the
// order of the ranks) and the stages are chosen on the host (fp4_plan.h).
//
// Large products take pairs of CTAs (PAIR): two 128-row tiles of W beside each
// other under one MMA of 256 rows, each CTA with half of X's rows in its shared memory.  One CTA alone is bound by
// shared memory's 128 bytes a cycle: a stage of 256 rows of X is 512 cycles of products, but 50 KB
// to write and 48 KB to read (753 measured); in a pair it is 35 and 32.
//
// 2176 rows of X, 24,576 of W, 4096 k (MX): 81 us, 5.4 PFLOP/s, the matrix unit at
// 0.65 of its cycles (without loads it would be 0.8 at this tile, without
// stores 0.75); 16 rows of X: 14.4 us, 3.8 TB/s, of which 4 to start and end.
//
//   warps 8, 11: codes and scales into the ring (one warp for both is through with a stage in about the time
//     of its products);
//   warp 9: MMAs; owns the TMEM allocation;
//   warp 10: scales to TMEM;
//   warps 0-7: read an accumulator out (lane = column of out), 32 rows of out
//     at a time, and store it while the next tile's products fill the other one:
//     through shared memory and a copy per 32 x 32 block where rows of out are
//     whole 16 bytes, else entry by entry.
#include <algorithm>
#include <mutex>

#include "fp4_common.cuh"
#include "fp4_plan.h"
#include "tma_map.h"

namespace dflash {

namespace {

constexpr int kCopyWarp = kOutWarps, kMmaWarp = 9, kScaleWarp = 10, kScaleCopyWarp = 11, kFp4Threads = 384;

struct Fp4Params {
  const uint8_t *w_scales, *x_scales;
  const float *w_scale, *x_scale;
  void* out;
  long long tiles;                      // of all CTAs: n_tiles x m_tiles
  int M, N, kt, m_tiles, bn, stages;
  int last_mmas;                        // MMAs (64 k) of a row's last stage
  int second;                           // column of the second accumulator
  int shared_last, shared_first;        // blocks of 32 columns that they share: of the first one, of the second one
  int sc_first, tmem_cols;              // column of the scales; columns allocated
  int bulk;                             // out goes through shared memory: blocks of it that a warp has there (0: not)
  int* status;
};

// Shared memory: barriers, then (1024-aligned) the ring, then a block of out a warp.
template <typename T>
constexpr int kOutBlock = kOutRows * 32 * static_cast<int>(sizeof(T));
struct Fp4Barriers {
  uint64_t full[kMaxStages], scaled[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  uint32_t tmem;
};
static_assert(sizeof(Fp4Barriers) <= kFp4Head, "the plan keeps room for them");

// mbar_wait where no status word need be given.
__device__ __forceinline__ bool fp4_wait(uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_hint(bar, parity, 20000u)) return true;
    if ((it & 15u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
      if (status != nullptr) atomicOr(status, ST_WAIT_TIMEOUT);
      return false;
    }
  }
}

// Shared-memory descriptors: the address in 16 bytes (the low half), and what does not change beside it: for codes
// those of sw128_kmajor_desc, for scales 32 rows x 16 bytes, rows adjacent (no swizzle, 8-row groups 128 bytes apart).
constexpr uint32_t kCodeDescHi = (1024 >> 4) | 1u << 14 | 2u << 29, kScaleDescHi = (128 >> 4) | 1u << 14;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }
__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
// 32 rows x 16 bytes into 4 columns, the same in all four quarters of the lanes (PAIR: in both CTAs, each its own).
template <bool PAIR>
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Arrive on `bar` when all that was issued before is done; BOTH: on that barrier of both CTAs of the pair.
template <bool PAIR, bool BOTH>
__device__ __forceinline__ void fp4_commit(uint64_t* bar) {
  if constexpr (!PAIR)
    tc_commit(bar);
  else if constexpr (BOTH)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// A box into this CTA's shared memory, counted by the barrier (a cluster address) of the pair's first CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void fp4_tmem_alloc(uint32_t* dst, uint32_t cols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void fp4_tmem_free(uint32_t addr, uint32_t cols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  else
    tmem_dealloc(addr, cols);
}
// fp4_wait for arrivals of the other CTA too.
__device__ __forceinline__ bool fp4_wait_pair(uint64_t* bar, uint32_t parity, int* status) {
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t it = 0;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    if ((it & 15u) == 15u && globaltimer_ns() - t0 > kWaitLimitNs) {
      if (status != nullptr) atomicOr(status, ST_WAIT_TIMEOUT);
      return false;
    }
  }
}

// Instruction descriptor of the block-scaled MMA: E2M1 operands (bits 7-9 and
// 10-11 = 1), both K-major, N / 8 at bits 17-22, the scales' type at bit 23
// (1: powers of two, 0: E4M3), M / 128 at bits 27-28; which of a column's
// bytes hold the scales at bits 4-5 (W's partner X) and 29-30 (W).
__host__ __device__ constexpr uint32_t fp4_idesc(int n, bool nv, int byte, bool pair) {
  return (static_cast<uint32_t>(byte) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (nv ? 0u : 1u << 23) | ((pair ? 2u : 1u) << 27) | (static_cast<uint32_t>(byte) << 29);
}

// (FIRST: the sum starts anew)
template <bool NV, bool FIRST, bool PAIR>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb) {
  if constexpr (NV && PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "n"(FIRST ? 0 : 1)
        : "memory");
  else if constexpr (NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "n"(FIRST ? 0 : 1)
        : "memory");
  else if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "n"(FIRST ? 0 : 1)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "n"(FIRST ? 0 : 1)
        : "memory");
}

template <typename T>
__device__ __forceinline__ T fp4_out(float v);
template <>
__device__ __forceinline__ float fp4_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 fp4_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half fp4_out<__half>(float v) { return __float2half_rn(v); }

// What sums are multiplied by: the product of the two tensors' scales, or, where that leaves fp32's normal range, both one
// after the other, the larger one first (a sum is 0 or 2^-20 to 2^47: where it leaves the range in between, so does
// the result).
struct Fp4Alpha {
  float a, b;
  __device__ __forceinline__ float times(float v) const { return v * a * b; }
};
__device__ __forceinline__ Fp4Alpha fp4_alpha(const float* w, const float* x) {
  const float f = w != nullptr ? *w : 1.f, g = x != nullptr ? *x : 1.f, h = f * g;
  if (fabsf(h) >= 0x1p-126f && fabsf(h) < __int_as_float(0x7f800000)) return {h, 1.f};
  return fabsf(f) >= fabsf(g) ? Fp4Alpha{f, g} : Fp4Alpha{g, f};
}

__device__ __forceinline__ void st_shared(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void st_shared(uint32_t a, __nv_bfloat16 v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(__bfloat16_as_ushort(v)) : "memory");
}
__device__ __forceinline__ void st_shared(uint32_t a, __half v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(__half_as_ushort(v)) : "memory");
}
__device__ __forceinline__ float4 ld_dsmem_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}

// XT: 128-row scale tiles that a tile's rows of X lie in.
template <bool NV, typename T, int XT, bool PAIR>
__global__ void __launch_bounds__(kFp4Threads, 1)
    k_gemm_fp4(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
               const __grid_constant__ CUtensorMap to, const __grid_constant__ CUtensorMap tws,
               const __grid_constant__ CUtensorMap txs, const Fp4Params p) {
  constexpr int CHUNKS = NV ? 4 : 2;          // scale tiles (4 scales of 128 rows) a stage
  constexpr int WS = CHUNKS * 512;
  extern __shared__ uint8_t raw[];
  Fp4Barriers& s = *reinterpret_cast<Fp4Barriers*>(raw);
  const uint32_t ring = (smem_u32(raw) + static_cast<uint32_t>(sizeof(Fp4Barriers)) + 1023u) & ~1023u;
  // a stage: codes of W, codes of X, scales of W, scales of up to two 128-row tiles of X
  const int own_rows = PAIR ? p.bn / 2 : p.bn;  // rows of X whose codes this CTA has
  const uint32_t x_at = kRows * kCodeRow, ws_at = x_at + own_rows * kCodeRow, xs_at = ws_at + WS;
  const uint32_t stage_bytes = (xs_at + XT * WS + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a cluster is a pair, or the CTAs that share a tile's k
  const uint32_t rank = cluster_ctarank(), split = PAIR ? 1 : cluster_nctarank(), k_rank = PAIR ? 0 : rank;
  const uint32_t team = PAIR ? 2 : split;
  const long long first = blockIdx.x / team, step = gridDim.x / team;
  const int k0 = static_cast<int>(static_cast<long long>(p.kt) * k_rank / split);
  const int k1 = static_cast<int>(static_cast<long long>(p.kt) * (k_rank + 1) / split);
  // 128-row tile of W of tile t
  const auto w_tile = [&](long long t) {
    const int n = static_cast<int>(t / p.m_tiles);
    return PAIR ? 2 * n + static_cast<int>(rank) : n;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s.full[i], 2);
      mbar_init(&s.scaled[i], 2);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], PAIR ? 2 * kOutWarps : kOutWarps);
    }
    fence_mbar_init();
  }
  // (before TMEM is taken: a kernel before this one may still have to take its own)
  pdl_wait();
  if (warp == kMmaWarp) {
    fp4_tmem_alloc<PAIR>(&s.tmem, p.tmem_cols);
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  // a set of scale columns for each stage, behind the accumulators: W's, then X's (128-row tile after 128-row tile of a chunk)
  constexpr uint32_t kSet = CHUNKS * 4 * (1 + XT);
  const uint32_t sc_col = tmem + p.sc_first;

  // The two issuing warps run converged (a batch's product 121 us with one thread of each in a branch, most of
  // it that thread's).
  if (warp == kCopyWarp || warp == kScaleCopyWarp) {
    const bool codes = warp == kCopyWarp;
    if (codes && elect_one()) {
      tma_prefetch_desc(&tw);
      tma_prefetch_desc(&tx);
    }
    uint32_t st = 0, round = 0;
    bool ok = true;
    for (long long t = first; t < p.tiles && ok; t += step) {
      const int nt = w_tile(t), m0 = static_cast<int>(t % p.m_tiles) * p.bn;
      const int xt0 = m0 >> 7, xts = XT == 1 ? 1 : ((min(m0 + p.bn, p.M) - 1) >> 7) - xt0 + 1;
      const uint8_t* ws = p.w_scales + (static_cast<long long>(nt) * p.kt + k0) * WS;
      const uint8_t* xs = p.x_scales + (static_cast<long long>(xt0) * p.kt + k0) * WS;
      // (a pair's copies are whole boxes, filled up behind the matrices' ends)
      const uint32_t code_bytes = (PAIR ? 2 : 1) * (kRows + own_rows) * kCodeRow;
      const uint32_t scale_bytes = PAIR ? 2 * WS * (1 + XT) : WS * (1 + xts);
      for (int k = k0; k < k1; ++k, ws += WS, xs += WS) {
        if (round > 0 && !(ok = fp4_wait(&s.empty[st], (round - 1) & 1, p.status))) break;
        const uint32_t base = ring + st * stage_bytes;
        __syncwarp();
        if constexpr (PAIR) {
          const uint32_t bar = dsmem_map(smem_u32(&s.full[st]), 0);
          constexpr int kLines = WS / 256;  // (scales as lines of 256 bytes)
          if (elect_one()) {
            if (codes) {
              if (rank == 0) mbar_arrive_expect_tx(&s.full[st], code_bytes);
              tma_load_pair(base, &tw, bar, k * kCodeRow, nt * kRows);
              tma_load_pair(base + x_at, &tx, bar, k * kCodeRow, m0 + static_cast<int>(rank) * own_rows);
            } else {
              if (rank == 0) mbar_arrive_expect_tx(&s.full[st], scale_bytes);
              tma_load_pair(base + ws_at, &tws, bar, 0, (nt * p.kt + k) * kLines);
#pragma unroll
              for (int x = 0; x < XT; ++x) tma_load_pair(base + xs_at + x * WS, &txs, bar, 0, ((xt0 + x) * p.kt + k) * kLines);
            }
          }
        } else if (elect_one()) {
          if (codes) {
            mbar_arrive_expect_tx(&s.full[st], code_bytes);
            tma_load_2d_to(base, &tw, &s.full[st], k * kCodeRow, nt * kRows);
            tma_load_2d_to(base + x_at, &tx, &s.full[st], k * kCodeRow, m0);
          } else {
            mbar_arrive_expect_tx(&s.full[st], scale_bytes);
            bulk_load_global(base + ws_at, ws, WS, &s.full[st]);
            bulk_load_global(base + xs_at, xs, WS, &s.full[st]);
            if (xts > 1) bulk_load_global(base + xs_at + WS, xs + static_cast<long long>(p.kt) * WS, WS, &s.full[st]);
          }
        }
        __syncwarp();
        if (++st == static_cast<uint32_t>(p.stages)) st = 0, ++round;
      }
    }
    // the copies in flight have landed before the block ends
    for (uint32_t i = 0; i < static_cast<uint32_t>(p.stages); ++i) {
      const uint32_t filled = round + (i < st);
      if (filled > 0 && (!PAIR || rank == 0)) fp4_wait(&s.full[i], (filled - 1) & 1, p.status);
    }
  } else if (PAIR && rank != 0 && (warp == kScaleWarp || warp == kMmaWarp)) {
    // the pair's first CTA issues for both
  } else if (warp == kScaleWarp) {
    // An MMA waits for scales that the same thread copied before it, but a copy does not wait for MMAs, and one
    // warp that issues both has no time for it (four MMAs of 96 cycles a stage).  So copies come from a warp of their own,
    // which says when they are done; there are as many sets of columns as stages, and a set is free when its stage is.
    const uint32_t w_lo = desc_lo(ring + ws_at), x_lo = desc_lo(ring + xs_at), hi = kScaleDescHi;
    const uint32_t total = first < p.tiles ? static_cast<uint32_t>((p.tiles - first + step - 1) / step) * (k1 - k0) : 0;
    uint32_t st = 0, parity = 0, at = 0, sc = sc_col;
    bool ok = true;
    for (uint32_t it = 0; it < total; ++it) {
      ok = ok && fp4_wait(&s.full[st], parity, p.status);
      __syncwarp();
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
          tc_cp_scales<PAIR>(sc + 4 * c, desc64(w_lo + at + c * 32, hi));
#pragma unroll
          for (int x = 0; x < XT; ++x)
            tc_cp_scales<PAIR>(sc + 4 * (CHUNKS + c * XT + x), desc64(x_lo + at + (x * WS + c * 512) / 16, hi));
        }
        fp4_commit<PAIR, false>(&s.scaled[st]);
        mbarrier_arrive_one(&s.scaled[st]);  // (hands on what the wait above saw: the MMAs' codes are there)
      }
      __syncwarp();
      at += stage_bytes >> 4;
      sc += kSet;
      if (++st == static_cast<uint32_t>(p.stages)) st = 0, parity ^= 1, at = 0, sc = sc_col;
    }
    // (the last copies are over before the columns are given back: the MMAs that follow them are)
  } else if (warp == kMmaWarp) {
    const uint32_t a_lo = desc_lo(ring) | 1u << 16, b_lo = desc_lo(ring + x_at) | 1u << 16, hi = kCodeDescHi;
    const uint32_t idesc = fp4_idesc(p.bn, NV, 0, PAIR);
    // (once a wait has given up there are no more waits; the loops run on, so that they do not hang on what a
    // barrier said)
    bool ok = true;
    uint32_t st = 0, parity = 0, nth = 0, at = 0, sc = sc_col;
    for (long long t = first; t < p.tiles; t += step, ++nth) {
      const int m0 = static_cast<int>(t % p.m_tiles) * p.bn;
      const uint32_t a = nth & 1, d = tmem + (a ? p.second : 0), x_off = CHUNKS * 4 + ((m0 & 127) >> 5);
      // an accumulator of its own is free once the tile before last is read out, one that shares columns with the
      // other once the last tile's part of these is (which comes after all of the tile before)
      const uint32_t behind = p.shared_first > 0 ? 1 : 2;
      if (nth >= behind) {
        uint64_t* const bar = &s.acc_empty[(nth - behind) & 1];
        const uint32_t parity_of = ((nth - behind) >> 1) & 1;
        ok = ok && (PAIR ? fp4_wait_pair(bar, parity_of, p.status) : fp4_wait(bar, parity_of, p.status));
      }
      for (int k = k0; k < k1; ++k) {
        const int n = k == p.kt - 1 ? p.last_mmas : 4;
        ok = ok && fp4_wait(&s.scaled[st], parity, p.status);
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
          const auto mma = [&](int j, auto first_one) {
            constexpr uint32_t kByte2 = (2u << 4) | (2u << 29);
            const int c = NV ? j : j / 2;
            tc_mma_fp4<NV, decltype(first_one)::value, PAIR>(d, desc64(a_lo + at + 2 * j, hi), desc64(b_lo + at + 2 * j, hi),
                                                       idesc | (!NV && (j & 1) ? kByte2 : 0u), sc + 4 * c,
                                                       sc + x_off + 4 * c * XT);
          };
          if (k > k0) mma(0, std::false_type{});
          else mma(0, std::true_type{});
          if (n == 4) {
            mma(1, std::false_type{});
            mma(2, std::false_type{});
            mma(3, std::false_type{});
          } else {
            if (n > 1) mma(1, std::false_type{});
            if (n > 2) mma(2, std::false_type{});
          }
          fp4_commit<PAIR, true>(&s.empty[st]);
          if (k == k1 - 1) fp4_commit<PAIR, true>(&s.acc_full[a]);
        }
        at += stage_bytes >> 4;
        sc += kSet;
        if (++st == static_cast<uint32_t>(p.stages)) st = 0, parity ^= 1, at = 0, sc = sc_col;
      }
    }
    __syncwarp();
  } else {
    Fp4Alpha alpha{1.f, 1.f};
    if constexpr (NV) alpha = fp4_alpha(p.w_scale, p.x_scale);
    uint32_t n_tile = 0;
    bool ok = true;
    // two warps a quarter of the lanes, which take turns at the blocks of 32 columns
    const int quad = warp & 3, turn = warp >> 2;
    const uint32_t stage0 = ring + p.stages * stage_bytes + warp * p.bulk * kOutBlock<T>;
    uint32_t turn_out = 0;
    if (p.bulk && lane == 0) tma_prefetch_desc(&to);
    for (long long t = first; t < p.tiles && ok; t += step, ++n_tile) {
      const int nw = w_tile(t) * kRows + quad * 32, m0 = static_cast<int>(t % p.m_tiles) * p.bn;
      const uint32_t a = n_tile & 1;
      ok = fp4_wait(&s.acc_full[a], (n_tile >> 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = tmem + (a ? p.second : 0) + (static_cast<uint32_t>(quad * 32) << 16);
      const int rows = min(p.bn, p.M - m0);
      const int blocks = (p.bn + kOutRows - 1) / kOutRows;
      const auto load = [&](int c, uint32_t (&v)[2][16]) {
        tc_ld_32x32b_x16_nw(at + c, v[0]);
        if (c + 16 < p.bn) tc_ld_32x32b_x16_nw(at + c + 16, v[1]);  // (the last block may be a half)
      };
      const auto store = [&](int c, const uint32_t (&v)[2][16]) {
        const uint32_t stage = stage0 + (turn_out & 1) * (p.bulk == 2 ? kOutBlock<T> : 0);
        if (p.bulk) {
          // what was stored from here last has been read
          if (lane == 0) {
            if (p.bulk == 2) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            else bulk_wait_read_all();
          }
          __syncwarp();
          ++turn_out;
        }
        const auto half = [&](int c, int to_row, const uint32_t (&x)[16]) {
          if (split > 1) {
            // this rank's partial sums, [row of X][row of W], over the ring (whose stages are all used up)
            const uint32_t part = ring + (c * kRows + quad * 32 + lane) * 4;
#pragma unroll
            for (int i = 0; i < 16; ++i) st_shared(part + i * kRows * 4, __uint_as_float(x[i]));
          } else if (p.bulk) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              st_shared(stage + ((to_row + i) * 32 + lane) * static_cast<int>(sizeof(T)),
                        fp4_out<T>(alpha.times(__uint_as_float(x[i]))));
          } else if (nw + lane < p.N) {
            T* o = static_cast<T*>(p.out) + static_cast<long long>(m0 + c) * p.N + nw + lane;
            const int n = rows - c;
#pragma unroll
            for (int i = 0; i < 16; ++i, o += p.N)
              if (i < n) *o = fp4_out<T>(alpha.times(__uint_as_float(x[i])));
          }
        };
        half(c, 0, v[0]);
        if (c + 16 < p.bn) half(c + 16, 16, v[1]);
        if (p.bulk) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            // (rows and columns of the block behind the matrix are left out by the copy)
            if (nw < p.N && c < rows) tma_store_2d(&to, stage, nw, m0 + c);
            bulk_commit();
          }
        }
      };
      // Two of the warp's blocks at a time.  Columns that both accumulators have come first (the first one's last, the
      // second one's first), and the accumulator is given back as soon as these are in registers: behind their
      // stores the next tile's products waited 1.9 us a tile.
      const bool down = a == 0 && p.shared_first > 0;
      const int last = p.shared_first == 0 ? blocks : down ? p.shared_last : p.shared_first;
      bool gave = false;
      const auto give = [&]() {
        gave = true;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR && rank != 0) mbar_remote_arrive(&s.acc_empty[a], 0);
          else mbarrier_arrive_one(&s.acc_empty[a]);
        }
      };
      for (int i = turn; i < blocks; i += 4) {
        const int c0 = (down ? blocks - 1 - i : i) * kOutRows, c1 = (down ? blocks - 3 - i : i + 2) * kOutRows;
        const bool two = i + 2 < blocks;
        uint32_t v[2][2][16];
        load(c0, v[0]);
        if (two) load(c1, v[1]);
        tc_wait_ld();
        if (!gave && i + 4 >= last) give();
        store(c0, v[0]);
        if (two) store(c1, v[1]);
      }
      if (!gave) give();
    }
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
  }
  if (split > 1) {
    // one tile a cluster: rank r adds rows r, r + split, ... of all ranks' sums
    __syncwarp();
    cluster_sync_all();
    if (first < p.tiles) {
      Fp4Alpha alpha{1.f, 1.f};
      if constexpr (NV) alpha = fp4_alpha(p.w_scale, p.x_scale);
      // (a warp a row, four of its columns a lane: with a column a thread and one row after the other 64 rows of two ranks took 4 us)
      const int n = static_cast<int>(first / p.m_tiles) * kRows + lane * 4, m0 = static_cast<int>(first % p.m_tiles) * p.bn;
      const int rows = min(p.bn, p.M - m0);
      const bool whole = n + 4 <= p.N && p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % (4 * sizeof(T)) == 0;
      for (int r = rank + split * warp; r < rows; r += split * (kFp4Threads / 32)) {
        float4 v[kMaxSplit];
#pragma unroll
        for (uint32_t i = 0; i < kMaxSplit; ++i)
          if (i < split) v[i] = ld_dsmem_f32x4(dsmem_map(ring + (r * kRows + lane * 4) * 4, i));
        float4 sum = v[0];
#pragma unroll
        for (uint32_t i = 1; i < kMaxSplit; ++i)
          if (i < split) sum.x += v[i].x, sum.y += v[i].y, sum.z += v[i].z, sum.w += v[i].w;
        T* const o = static_cast<T*>(p.out) + static_cast<long long>(m0 + r) * p.N + n;
        struct alignas(4 * sizeof(T)) Four {
          T t[4];
        } four{{fp4_out<T>(alpha.times(sum.x)), fp4_out<T>(alpha.times(sum.y)), fp4_out<T>(alpha.times(sum.z)),
                   fp4_out<T>(alpha.times(sum.w))}};
        if (whole) {
          *reinterpret_cast<Four*>(o) = four;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < p.N) o[j] = four.t[j];
        }
      }
    }
    cluster_sync_all();
  }
  tc_fence_before();
  __syncwarp();
  // (a pair's CTAs read and arrive in each other's memory until both are through)
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    fp4_tmem_free<PAIR>(tmem, p.tmem_cols);
  }
}

// Codes [rows][K / 2] as boxes of box_rows x 128 bytes, swizzled.
bool code_map(CUtensorMap* map, const void* base, long long rows, int K, int box_rows) {
  const auto encode = tensor_map_encoder();
  const cuuint64_t gdim[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t pitch[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t box[2] = {kCodeRow, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return encode != nullptr &&
         encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, pitch, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as lines of 256 bytes, a stage's of one 128-row tile a box.
bool scale_map(CUtensorMap* map, const void* base, long long lines, int box_lines) {
  const auto encode = tensor_map_encoder();
  const cuuint64_t gdim[2] = {256, static_cast<cuuint64_t>(lines)};
  const cuuint64_t pitch[1] = {256};
  const cuuint32_t box[2] = {256, static_cast<cuuint32_t>(box_lines)}, es[2] = {1, 1};
  return encode != nullptr &&
         encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, pitch, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// out [M][N] as boxes of 32 x 32.
bool out_map(CUtensorMap* map, void* out, int elem, int M, int N, int size) {
  const auto encode = tensor_map_encoder();
  const cuuint64_t gdim[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
  const cuuint64_t pitch[1] = {static_cast<cuuint64_t>(N) * size};
  const cuuint32_t box[2] = {32, kOutRows}, es[2] = {1, 1};
  const CUtensorMapDataType type = elem == DFLASH_ELEM_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : elem == DFLASH_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode != nullptr &&
         encode(map, type, 2, out, gdim, pitch, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of n CTAs with an SM each that run at once: a GPC's SMs beyond whole clusters stay free.  Asked once a device.
int clusters_at_once(int n, int sms) {
  static std::mutex mu;
  static int known[64][kMaxSplit + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return std::max(1, sms / n);
  std::lock_guard<std::mutex> lock(mu);
  int& c = known[dev][n];
  if (c > 0) return c;
  const auto k = k_gemm_fp4<false, float, 1, false>;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = n;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(n);
  lc.blockDim = dim3(kFp4Threads);
  lc.dynamicSmemBytes = kFp4Smem;
  lc.attrs = &at;
  lc.numAttrs = 1;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kFp4Smem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&c, k, &lc) != cudaSuccess || c < 1) {
    cudaGetLastError();
    c = std::max(1, sms / n);
  }
  return c;
}

struct Fp4Maps {
  CUtensorMap w, x, out, w_scales, x_scales;
};

template <bool NV, typename T, int XT, bool PAIR>
cudaError_t launch_fp4_x(const Fp4Plan& c, const Fp4Maps& m, const Fp4Params& p, cudaStream_t s) {
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(kFp4Smem, [](int v) {
    return cudaFuncSetAttribute(k_gemm_fp4<NV, T, XT, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  return launch_k(k_gemm_fp4<NV, T, XT, PAIR>, dim3(c.grid), dim3(kFp4Threads), c.smem, s, dim3(PAIR ? 2 : c.split), true,
                  m.w, m.x, m.out, m.w_scales, m.x_scales, p);
}

template <bool NV, typename T>
cudaError_t launch_fp4(const Fp4Plan& c, const Fp4Maps& m, const Fp4Params& p, cudaStream_t s) {
  if (c.pair) return launch_fp4_x<NV, T, 2, true>(c, m, p, s);
  return c.x_tiles == 1 ? launch_fp4_x<NV, T, 1, false>(c, m, p, s) : launch_fp4_x<NV, T, 2, false>(c, m, p, s);
}

}  // namespace

}  // namespace dflash

using namespace dflash;

extern "C" dflash_status dflash_gemm_fp4(const void* W, const void* w_scales, const float* w_scale, int N, const void* X,
                                         const void* x_scales, const float* x_scale, int M, int K, int format, void* out,
                                         int out_elem, int* status, dflash_stream stream) {
  if (W == nullptr || w_scales == nullptr || X == nullptr || x_scales == nullptr || out == nullptr || N < 1 || M < 1 ||
      K < 1)
    return DFLASH_ERR_INVALID_ARG;
  if ((format != DFLASH_FP4_MX && format != DFLASH_FP4_NV) ||
      (format == DFLASH_FP4_MX && (w_scale != nullptr || x_scale != nullptr)))
    return DFLASH_ERR_INVALID_ARG;
  if (out_elem != DFLASH_ELEM_F32 && out_elem != DFLASH_ELEM_BF16 && out_elem != DFLASH_ELEM_F16)
    return DFLASH_ERR_INVALID_ARG;
  const auto addr = [](const void* a) { return reinterpret_cast<uintptr_t>(a); };
  const int size = out_elem == DFLASH_ELEM_F32 ? 4 : 2;
  if (addr(W) % 16 || addr(X) % 16 || addr(w_scales) % 16 || addr(x_scales) % 16 || addr(w_scale) % 4 ||
      addr(x_scale) % 4 || addr(out) % size || addr(status) % 4)
    return DFLASH_ERR_INVALID_ARG;
  if (!fp4_shape_ok(N, K) || !fp4_shape_ok(M, K)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return DFLASH_ERR_CUDA;
  Fp4Params p{};
  p.kt = (K + 255) / 256;
  const Fp4Plan c = fp4_plan(format == DFLASH_FP4_NV, M, N, p.kt, sms, size, [&](int n) { return clusters_at_once(n, sms); });
  Fp4Maps maps{};
  const long long n_tiles = (N + kRows - 1) / kRows;
  if (!code_map(&maps.w, W, N, K, kRows) || !code_map(&maps.x, X, M, K, c.pair ? c.bn / 2 : c.bn)) return DFLASH_ERR_CUDA;
  if (c.pair) {
    const int lines = format == DFLASH_FP4_NV ? 8 : 4;  // of 256 bytes, a stage of a 128-row tile
    if (!scale_map(&maps.w_scales, w_scales, n_tiles * p.kt * lines, lines) ||
        !scale_map(&maps.x_scales, x_scales, static_cast<long long>((M + kRows - 1) / kRows) * p.kt * lines, lines))
      return DFLASH_ERR_CUDA;
  }
  p.bulk = c.split == 1 && addr(out) % 16 == 0 && static_cast<long long>(N) * size % 16 == 0 ? c.blocks : 0;
  if (p.bulk && !out_map(&maps.out, out, out_elem, M, N, size)) return DFLASH_ERR_CUDA;
  p.w_scales = static_cast<const uint8_t*>(w_scales);
  p.x_scales = static_cast<const uint8_t*>(x_scales);
  p.w_scale = w_scale;
  p.x_scale = x_scale;
  p.out = out;
  p.tiles = (c.pair ? (n_tiles + 1) / 2 : n_tiles) * c.m_tiles;
  p.M = M;
  p.N = N;
  p.m_tiles = c.m_tiles;
  p.bn = c.bn;
  p.stages = c.stages;
  p.last_mmas = (K - (p.kt - 1) * 256 + 63) / 64;
  p.second = c.second;
  p.shared_last = c.shared_last;
  p.shared_first = c.shared_first;
  p.sc_first = c.sc_first;
  p.tmem_cols = c.cols;
  p.status = status;
  const auto run = [&](auto t) {
    using T = decltype(t);
    return format == DFLASH_FP4_NV ? launch_fp4<true, T>(c, maps, p, stream) : launch_fp4<false, T>(c, maps, p, stream);
  };
  e = out_elem == DFLASH_ELEM_F32    ? run(float{})
      : out_elem == DFLASH_ELEM_BF16 ? run(__nv_bfloat16{})
                                     : run(__half{});
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
