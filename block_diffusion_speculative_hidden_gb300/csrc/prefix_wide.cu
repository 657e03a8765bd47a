// Prefix attention, items of many query rows: the fifth-generation tensor
// cores (tcgen05) with two tiles of 128 query rows a CTA.
//
// One warpgroup per row tile runs the softmax, a query row a thread (its
// TMEM lane), so a row's maximum and sum never leave the thread.  Per tile of
// 128 keys: S = Q K^T into TMEM (one MMA chain, Q and K from shared memory),
// P = 2^(S scale - m) rounded to 16 bits over S's own columns, and O += P V
// with P as the A operand from TMEM.  The two row tiles share the K / V
// stream and alternate on the tensor pipe: while one tile's softmax runs, the
// other tile's products do.  m moves only when a row's maximum passes it by
// more than 2^8, and O is rescaled in TMEM only then, so P stays at most 2^8.
#include "prefix_common.cuh"

namespace dflash {

namespace {

constexpr int kWideTile = 128;       // query rows of a tile: one TMEM lane each
constexpr int kWideKeys = 128;       // keys of a tile
constexpr int kWidePages = kWideKeys / kPage;
constexpr int kWideThreads = 384;    // two softmax warpgroups; the TMA warp, the MMA warp and two that only share registers
// registers a thread: 3 * 168 at launch, given to the softmax (224 + 224 + 56 = 3 * 168)
constexpr int kWideSoftRegs = 224, kWideFeedRegs = 56;
constexpr float kWideLazy = 8.f;     // how far (in powers of two) a maximum may pass m

template <int DH>
struct WideLayout {
  static constexpr int NCH = DH / 64;                       // 128-byte column chunks of a head
  static constexpr int Q_CH = kWideTile * 128;
  static constexpr int Q_TILE = NCH * Q_CH;
  static constexpr int KV_CH = kWideKeys * 128;
  static constexpr int SLOT = NCH * KV_CH;                  // a K or a V tile
  static constexpr int NS = DH == 128 ? 5 : 8;              // ring slots: K(0), V(0), K(1), ..
  static constexpr int OFF_KV = 2 * Q_TILE;
  static constexpr int OFF_BAR = OFF_KV + NS * SLOT;
  static constexpr int BYTES = OFF_BAR + 256;
  static constexpr int SMEM = 1024 + BYTES;
  static constexpr uint32_t S_COL = 0, O_COL = 2 * kWideKeys;  // TMEM: two S (and P), two O
  static constexpr uint32_t COLS = 512;
  static_assert(O_COL + 2 * DH <= COLS, "the accumulators fit TMEM");
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  static_assert((2 * NS + 9) * 8 + 8 <= 256, "barriers fit their area");
  // one CTA an SM: its TMEM allocation never waits for another's
  static_assert(2 * SMEM > 233472, "two CTAs of the kernel never share an SM");
};

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float wide_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float wide_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Instruction descriptor of tcgen05.mma kind::f16 with fp32 accumulators: A
// and B fp16 or bf16, B transposed (its N dimension contiguous) for P V.
template <typename T16>
__device__ __forceinline__ constexpr uint32_t wide_idesc(int m, int n, bool b_mn) {
  return mma_idesc_f16_f32(m, n, b_mn) | (std::is_same<T16, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u);
}

template <typename T16, int DH>
__global__ void __launch_bounds__(kWideThreads, 1) k_prefix_wide(const __grid_constant__ CUtensorMap tmK,
                                                                 const __grid_constant__ CUtensorMap tmV,
                                                                 const __grid_constant__ PrefixParams p, int n_prefix) {
  using L = WideLayout<DH>;
  using M16 = Mma16<T16>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* kv_empty = kv_full + L::NS;
  uint64_t* q_full = kv_empty + L::NS;  // [2]: per row tile, like the next three
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_trigger();  // (the kernels behind wait for this one's results on their own)
  Item it;
  if (!find_item(p, blockIdx.x, n_prefix, kWideRows, it)) return;
  const int np = max(0, it.pg1 - it.pg0);
  const int n = (np + kWidePages - 1) / kWidePages;                 // key tiles
  const int nt = it.rows - it.row0 > kWideTile ? 2 : 1;             // row tiles

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], kWideTile);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], kWideTile);
      mbar_init(&o_full[t], 1);
    }
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, L::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    regs_down<kWideFeedRegs>();
    if (warp == 8) {
      // ---------------- K and V tiles: lane l fetches chunk l % NCH of page l / NCH
      const int32_t* table = p.page_table + static_cast<long long>(it.table_row) * p.max_pages + it.pg0;
      const int pg = lane / L::NCH, c = lane % L::NCH;
      auto page_id = [&](int j) {
        const int i = j * kWidePages + pg;
        int id = 0;
        if (pg < kWidePages && i < np) {
          id = table[i];
          if (id < 0 || id >= p.n_pages) {
            if (c == 0) flag_status(p.status, ST_BAD_PAGE);
            id = p.n_pages;  // outside the tensor map: reads as zeros
          }
        }
        return id;
      };
      int next = n > 0 ? page_id(0) : 0, issued = 0;
      bool ok = true;
      for (int j = 0; ok && j < n; ++j) {
        const int id = next, npb = min(kWidePages, np - j * kWidePages);
        if (j + 1 < n) next = page_id(j + 1);
        for (int kv = 0; kv < 2 && ok; ++kv) {
          const int i = 2 * j + kv, s = i % L::NS;
          if (lane == 0) {
            if (i >= L::NS) ok = mbar_wait(&kv_empty[s], (i / L::NS - 1) & 1, p.status);
            if (ok) mbar_arrive_expect_tx(&kv_full[s], npb * L::NCH * 2048);
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (ok) {
            if (pg < npb)
              tma_page(smem_u32(smem + L::OFF_KV + s * L::SLOT + c * L::KV_CH + pg * 2048), kv ? &tmV : &tmK,
                       &kv_full[s], c * 64, it.kvh, id);
            issued = i + 1;
          }
        }
      }
      // every copy has landed before the CTA may leave
      for (int i = max(0, issued - L::NS); i < issued; ++i) mbar_wait(&kv_full[i % L::NS], (i / L::NS) & 1, p.status);
    } else if (warp == 9) {
      // ---------------- MMAs.  S(j + 1) of a row tile overwrites its P(j), so
      // it waits for P(j) V; the other row tile's products fill that time.
      if (lane == 0 && n > 0) {
        const uint32_t q0 = smem_u32(smem), kv0 = smem_u32(smem + L::OFF_KV);
        auto kv_wait = [&](int i) { return mbar_wait(&kv_full[i % L::NS], (i / L::NS) & 1, p.status); };
        auto issue_s = [&](int t, int j) {
          const uint32_t a = q0 + t * L::Q_TILE, k = kv0 + ((2 * j) % L::NS) * L::SLOT;
          const uint32_t id = wide_idesc<T16>(kWideTile, 16 * min(kWidePages, np - j * kWidePages), false);
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks)
            tc_mma_bf16(tmem + L::S_COL + t * kWideKeys, sw128_desc(a + (ks >> 2) * L::Q_CH + (ks & 3) * 32, 16, 1024),
                        sw128_desc(k + (ks >> 2) * L::KV_CH + (ks & 3) * 32, 16, 1024), id, ks > 0 ? 1u : 0u);
          tc_commit(&s_full[t]);
          if (t == nt - 1) tc_commit(&kv_empty[(2 * j) % L::NS]);
        };
        bool ok = kv_wait(0);
        for (int t = 0; ok && t < nt; ++t) {
          ok = mbar_wait(&q_full[t], 0, p.status);
          tc_fence_after();
          if (ok) issue_s(t, 0);
        }
        for (int j = 0; ok && j < n; ++j) {
          const int npb = min(kWidePages, np - j * kWidePages);
          const uint32_t v = kv0 + ((2 * j + 1) % L::NS) * L::SLOT;
          ok = kv_wait(2 * j + 1);
          for (int t = 0; ok && t < nt; ++t) {
            ok = mbar_wait(&p_full[t], j & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t id = wide_idesc<T16>(kWideTile, DH, true);
            for (int ks = 0; ks < npb; ++ks)
              tc_mma_bf16_ts(tmem + L::O_COL + t * DH, tmem + L::S_COL + t * kWideKeys + 8 * ks,
                             sw128_desc(v + ks * 2048, L::KV_CH, 1024), id, (j | ks) > 0 ? 1u : 0u);
            tc_commit(&o_full[t]);
            if (t == nt - 1) tc_commit(&kv_empty[(2 * j + 1) % L::NS]);
            if (j + 1 < n) {
              ok = (t > 0 || kv_wait(2 * j + 2)) && mbar_wait(&o_full[t], j & 1, p.status);
              tc_fence_after();
              if (ok) issue_s(t, j + 1);
            }
          }
        }
      }
      __syncwarp();
    }
  } else if (warp < 4 * nt) {
    regs_up<kWideSoftRegs>();
    // ---------------- softmax: thread r of warpgroup t owns row r of tile t
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const Row row = find_row(p, it, it.row0 + t * kWideTile + r);
    {
      const uint4* src =
          reinterpret_cast<const uint4*>(static_cast<const T16*>(p.q) + row.token * p.ld_q + (row.at - row.token * p.Hq) * DH);
      uint8_t* dst = smem + t * L::Q_TILE + r * 128;
#pragma unroll
      for (int u = 0; u < DH / 8; ++u)
        *reinterpret_cast<uint4*>(dst + (u >> 3) * L::Q_CH + (((u & 7) ^ (r & 7)) << 4)) =
            row.live ? src[u] : make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      mbarrier_arrive_one(&q_full[t]);
    }
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + L::S_COL + t * kWideKeys, o_at = tmem + lanes + L::O_COL + t * DH;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int npb = min(kWidePages, np - j * kWidePages);
      const int key0 = (it.pg0 + j * kWidePages) * kPage;
      ok = ok && mbar_wait(&s_full[t], j & 1, p.status);
      __syncwarp();
      tc_fence_after();
      uint32_t sv[kWidePages][16];
#pragma unroll
      for (int g = 0; g < kWidePages; ++g)
        if (g < npb) tc_ld_32x32b_x16_nw(s_at + 16 * g, sv[g]);
      tc_wait_ld();
      // keys of the tile that this row sees (the chunk may end inside the tile)
      const int lim = min(row.seen, it.pg1 * kPage) - key0;
      if (__any_sync(0xffffffffu, lim < kWideKeys)) {
#pragma unroll
        for (int g = 0; g < kWidePages; ++g)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (g * 16 + k >= lim) sv[g][k] = 0xff800000u;  // -infinity
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int g = 0; g < kWidePages; ++g)
#pragma unroll
        for (int k = 0; k < 16; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = wide_max3(mx[e], __uint_as_float(sv[g][k + 2 * e]), __uint_as_float(sv[g][k + 2 * e + 1]));
      const float cand = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      const bool move = cand > m + kWideLazy;
      if (__any_sync(0xffffffffu, move)) {
        const float al = move ? wide_ex2(m - cand) : 1.f;  // (m = -infinity: 0)
        if (move) m = cand;
        l *= al;
        if (j > 0) {
          // S(j) was issued after P(j - 1) V was done, so O is at rest
#pragma unroll
          for (int d = 0; d < DH; d += 32) {
            uint32_t v0[16], v1[16];
            tc_ld_32x32b_x16_nw(o_at + d, v0);
            tc_ld_32x32b_x16_nw(o_at + d + 16, v1);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              v0[e] = __float_as_uint(__uint_as_float(v0[e]) * al);
              v1[e] = __float_as_uint(__uint_as_float(v1[e]) * al);
            }
            tc_st_32x32b_x16(o_at + d, v0);
            tc_st_32x32b_x16(o_at + d + 16, v1);
          }
        }
      }
      const float mu = m == -INFINITY ? 0.f : m;
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), mneg2 = make_float2(-mu, -mu);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int g = 0; g < kWidePages; ++g) {
        uint32_t pk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 x = __ffma2_rn(
              make_float2(__uint_as_float(sv[g][2 * k]), __uint_as_float(sv[g][2 * k + 1])), sc2, mneg2);
          const float2 e = make_float2(wide_ex2(x.x), wide_ex2(x.y));
          sum = __fadd2_rn(sum, e);
          pk[k] = M16::pack(e.x, e.y);
        }
        tc_st_32x32b_x8(s_at + 8 * g, pk);
      }
      l += sum.x + sum.y;
      if (key0 + npb * kPage > it.tokens) {
        // the last page is partial: what its V rows hold past the last token
        // meets probabilities of zero and must be finite
        const int i = 2 * j + 1, first = it.tokens - (key0 + (npb - 1) * kPage);
        ok = ok && mbar_wait(&kv_full[i % L::NS], (i / L::NS) & 1, p.status);
        uint8_t* v = smem + L::OFF_KV + (i % L::NS) * L::SLOT + (npb - 1) * 2048;
        for (int e = r; e < (kPage - first) * L::NCH * 8; e += kWideTile) {
          const int c = e / ((kPage - first) * 8), f = e % ((kPage - first) * 8);
          *reinterpret_cast<uint4*>(v + c * L::KV_CH + first * 128 + f * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tc_wait_st();
      tc_fence_before();
      mbarrier_arrive_one(&p_full[t]);
    }
    if (n > 0) ok = ok && mbar_wait(&o_full[t], (n - 1) & 1, p.status);
    __syncwarp();
    tc_fence_after();
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const float lse2 = l > 0.f ? m + log2f(l) : -INFINITY;
    const long long R = static_cast<long long>(p.B) * p.T * p.Hq;
    const long long part = (it.shared ? it.chunk : p.p_chunks + it.chunk) * R + row.at;
#pragma unroll
    for (int d = 0; d < DH; d += 16) {
      uint32_t v[16];
      if (n > 0) {
        tc_ld_32x32b_x16_nw(o_at + d, v);
        tc_wait_ld();
      }
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = l > 0.f ? __uint_as_float(v[e]) * inv : 0.f;
      if (row.live && it.whole) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T16*>(p.out) + row.at * DH + d);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          dst[e] = make_uint4(M16::pack(x[8 * e], x[8 * e + 1]), M16::pack(x[8 * e + 2], x[8 * e + 3]),
                              M16::pack(x[8 * e + 4], x[8 * e + 5]), M16::pack(x[8 * e + 6], x[8 * e + 7]));
      } else if (row.live) {
        float4* dst = reinterpret_cast<float4*>(p.part_o + part * DH + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
      }
    }
    if (row.live && it.whole) {
      if (p.lse != nullptr) p.lse[row.at] = lse2 * 0.69314718055994531f;
    } else if (row.live) {
      p.part_lse[part] = lse2;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, L::COLS);
  }
}

template <typename T16, int DH>
cudaError_t launch_wide_t(const PrefixParams& p, long long n_prefix, long long n_own, const CUtensorMap& tk,
                          const CUtensorMap& tv, cudaStream_t s) {
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(WideLayout<DH>::SMEM, [](int v) {
    return cudaFuncSetAttribute(k_prefix_wide<T16, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  return launch_k(k_prefix_wide<T16, DH>, dim3(static_cast<unsigned>(n_prefix + n_own)), dim3(kWideThreads),
                  WideLayout<DH>::SMEM, s, dim3(1), false, tk, tv, p, static_cast<int>(n_prefix));
}

}  // namespace

cudaError_t launch_prefix_wide(const PrefixParams& p, int elem, int head_dim, long long n_prefix, long long n_own,
                               const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  if (elem == DFLASH_ELEM_BF16)
    return head_dim == 64 ? launch_wide_t<__nv_bfloat16, 64>(p, n_prefix, n_own, tk, tv, s)
                          : launch_wide_t<__nv_bfloat16, 128>(p, n_prefix, n_own, tk, tv, s);
  return head_dim == 64 ? launch_wide_t<__half, 64>(p, n_prefix, n_own, tk, tv, s)
                        : launch_wide_t<__half, 128>(p, n_prefix, n_own, tk, tv, s);
}

}  // namespace dflash
