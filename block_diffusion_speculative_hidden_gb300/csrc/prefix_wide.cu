// Prefix attention, items of many query rows: the fifth-generation tensor
// cores (tcgen05) with a tile of 128 query rows a CTA and two CTAs an SM.
//
// Per tile of 128 keys: S = Q K^T into TMEM (one MMA chain, Q and K from shared
// memory), P = 2^(S scale - m) rounded to 16 bits into TMEM, and O += P V with
// P as the A operand from there.  Eight warps run the softmax, two threads a
// query row (its TMEM lane), each with half of the keys and of the head's
// dimensions.  While one CTA's softmax runs, the other's products do; with 64
// dimensions S(j + 1) is made under the softmax of tile j as well.  m is the
// maximum of a row's first tile (less kLift) and moves (O is then rescaled in TMEM) only
// when a later tile's P sums to 2^14 or more, so P stays within 16 bits and
// most tiles need no maximum.
//
// Of 128 query rows and 128 keys with 128 dimensions an SM makes one product
// pair in 0.95 us (two CTAs, 1060 TFLOP/s over the card; 0.66 us would be the
// matrix units'): the latencies between the softmax's steps keep them from more
// (issue slots 0.49 taken, matrix units 0.46, exponentials 0.23).  32 entries
// of 17 rows, 32 query heads on 8 kv heads: a prefix of 8192 75 us, 16384 135;
// own sequences of 700 22 us.  With two S of 64 keys in the place of one of 128
// (S of the next half under the softmax) the same prefixes take 76 and 136 us.
#include "prefix_common.cuh"

namespace dflash {

namespace {

constexpr int kWideKeys = 128;       // keys of a tile
constexpr int kWidePages = kWideKeys / kPage;
constexpr int kWideLazy = 14;        // how far (in powers of two) a tile's P may sum up before m moves

template <int DH>
struct WideLayout {
  static constexpr int SOFT = 8;                            // softmax warps; then the TMA warp, the MMA warp and
  static constexpr int THREADS = (SOFT + 4) * 32;           // two warps that only hand their registers on
  // registers a thread: at launch, and after the warps' exchange
  static constexpr int REGS = 80, SOFT_REGS = 104, FEED_REGS = 32;
  static_assert(SOFT * SOFT_REGS + 4 * FEED_REGS <= (SOFT + 4) * REGS, "the exchange stays within the launch's registers");
  static constexpr int NCH = DH / 64;                       // 128-byte column chunks of a head
  static constexpr int Q_CH = kWideTile * 128;
  static constexpr int Q_BYTES = NCH * Q_CH;
  static constexpr int KV_CH = kWideKeys * 128;
  static constexpr int SLOT = NCH * KV_CH;                  // a K or a V tile
  static constexpr int NS = DH == 128 ? 2 : 5;              // ring slots: K(0), V(0), K(1), ..
  static constexpr int OFF_KV = Q_BYTES;
  static constexpr int OFF_RED = OFF_KV + NS * SLOT;        // [2][warp][lane] row maxima, sums
  static constexpr int OFF_BAR = OFF_RED + 2 * SOFT * 32 * 4;
  // pack_item's result: a tile's tokens, a scan's sums, the group, the item.  (In
  // bytes of their own: the warps read them until the end, and no barrier stands
  // between a warp's last look and another's first row maximum.)
  static constexpr int OFF_PACK = OFF_BAR + 256;
  static constexpr int PACK_BYTES = kWideTile * 4 + 128 + 128 + 64;
  static constexpr int SMEM = 1024 + OFF_PACK + PACK_BYTES;
  // TMEM: S, then O; with 128 dimensions P lies over S (each page's 16 keys in
  // the first 8 of its own 16 columns), with 64 there is room for it beside
  static constexpr bool P_APART = DH == 64;
  static constexpr uint32_t S_COL = 0, P_COL = P_APART ? kWideKeys : 0, O_COL = P_APART ? kWideKeys * 3 / 2 : kWideKeys;
  static constexpr uint32_t P_PAGE = P_APART ? 8 : 16, COLS = 256;
  static_assert(O_COL + DH <= COLS, "the accumulators fit TMEM");
  static_assert(SMEM <= 115712, "shared memory of a CTA");
  static_assert((2 * NS + 5) * 8 + 8 <= 256, "barriers fit their area");
  // the CTAs that an SM can hold by their shared memory find room in its 512
  // TMEM columns: an allocation never waits for another CTA's
  static_assert((512 / COLS + 1) * (SMEM + 1024) > 233472, "no more CTAs an SM than TMEM has room for");
  // at the end Q and the ring stage the output rows (fp32, or 16 bits)
  static constexpr int PITCH = DH * 4 + 16;
  static_assert(kWideTile * PITCH <= OFF_RED, "the staged rows fit");
};

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void wide_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Whether v holds for any of the 64 threads that meet at the barrier.
__device__ __forceinline__ bool wide_any(int id, bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 64, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(v ? 1 : 0), "r"(id)
      : "memory");
  return r != 0;
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
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int token) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(token), "r"(smem_u32(bar))
      : "memory");
}
// Rows between shared memory (32 rows of a pair of warps from `stage` on, pitch
// apart) and global memory: the whole warp takes row after row of its 16, so
// that a row or two cost one instruction (bulk copies of a row a thread are
// issued one thread at a time: 1.4 us for 32).  at: the row of lane l, -1: none.
template <int BYTES, typename Each>
__device__ __forceinline__ void wide_rows_each(uint8_t* stage, int pitch, int half, int at, Each&& each) {
  constexpr int LANES = BYTES / 16, ROWS = 32 / LANES;  // of a row; at once
  const int lane = threadIdx.x & 31, piece = lane % LANES;
#pragma unroll
  for (int i = 0; i < 16; i += ROWS) {
    const int r = half * 16 + i + lane / LANES, a = __shfl_sync(0xffffffffu, at, r);
    if (a >= 0) each(stage + r * pitch + piece * 16, static_cast<long long>(a) * BYTES + piece * 16);
  }
}

// Instruction descriptor of tcgen05.mma kind::f16 with fp32 accumulators: A
// and B fp16 or bf16, B transposed (its N dimension contiguous) for P V.
template <typename T16>
__device__ __forceinline__ constexpr uint32_t wide_idesc(int m, int n, bool b_mn) {
  return mma_idesc_f16_f32(m, n, b_mn) | (std::is_same<T16, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u);
}

// A running sum over the CTA's threads: of v up to and including this thread's,
// and (all) of every thread's.  warps: an int per warp in shared memory.
template <int WARPS>
__device__ __forceinline__ int cta_scan(int v, int* warps, int& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) v += warps[w];
    all += warps[w];
  }
  __syncthreads();
  return v;
}

// Prefix item `index` where entries have different numbers of rows: a group's
// tiles take its live tokens one after the other, so that only a group's last
// tile has rows without a query (a batch whose entries have 1 to 16 rows of 16
// is half the work).  tokens[i]: the tile's i-th token (entry x T + row), or -1.  cum:
// B + 1 ints.  The whole CTA asks.
template <int WARPS>
__device__ __noinline__ bool pack_item(const PrefixParams& p, int tile_tokens, Item* out, int* cum, int* warps, int* found,
                                       int* tokens) {
  int index = blockIdx.x;
  Item it;
  it.shared = true;
  it.last = false;
  it.chunk = index % p.p_chunks;
  index /= p.p_chunks;
  it.kvh = index % p.Hkv;
  const int tile = index / p.Hkv;
  // (a thread's first group is on the way while the entries are counted)
  Group g{0, 0, -1, 0, 0, 0};
  if (threadIdx.x < p.NG) g = load_group(p, threadIdx.x);
  if (!bounds_ok(p)) return false;
  int before = 0, all;
  for (int e0 = 0; e0 < p.B; e0 += WARPS * 32) {
    const int e = e0 + threadIdx.x, n = e < p.B ? entry_rows(p, e) : 0;
    const int sum = cta_scan<WARPS>(n, warps, all);
    if (e < p.B) cum[e + 1] = before + sum;
    before += all;
  }
  if (threadIdx.x == 0) {
    cum[0] = 0;
    found[0] = -1;
  }
  __syncthreads();
  before = 0;
  for (int g0 = 0; g0 < p.NG; g0 += WARPS * 32) {
    const int i = g0 + threadIdx.x;
    if (g0 > 0 && i < p.NG) g = load_group(p, i);
    int n = 0;
    if (i < p.NG) {
      n = (cum[g.hi] - cum[g.lo] + tile_tokens - 1) / tile_tokens;
      if (blockIdx.x == 0) check_prefix(p, g.row);
    }
    const int sum = before + cta_scan<WARPS>(n, warps, all);
    if (sum - n <= tile && tile < sum) {
      found[0] = g.lo;
      found[1] = g.hi;
      found[2] = g.row;
      found[3] = g.tokens;
      found[4] = tile - (sum - n);
    }
    before += all;
  }
  __syncthreads();
  if (found[0] < 0) return false;
  g = Group{found[0], found[1], found[2], found[3], found[4], 0};
  const int first = cum[g.lo] + g.tile * tile_tokens;
  it.b0 = g.lo;
  it.row0 = g.tile * tile_tokens * p.G;
  it.rows = (cum[g.hi] - cum[g.lo]) * p.G;
  it.tokens = g.tokens;
  it.table_row = g.row;
  const int pages = pages_of(it.tokens), per = chunk_pages(pages, p.p_chunks);
  it.pg0 = it.chunk * per;
  it.pg1 = min(pages, it.pg0 + per);
  if (it.pg0 >= it.pg1) return false;
  for (int i = threadIdx.x; i < tile_tokens; i += WARPS * 32) {
    int lo = g.lo, hi = g.hi - 1;  // the last entry of those that begin no later
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= first + i) lo = mid;
      else hi = mid - 1;
    }
    tokens[i] = first + i < cum[g.hi] ? lo * p.T + first + i - cum[lo] : -1;
  }
  if (threadIdx.x == 0) *out = it;
  __syncthreads();
  return true;
}

// PACK: prefix items of entries with different numbers of rows (pack_item).
template <typename T16, int DH, bool PACK>
__global__ void __launch_bounds__(WideLayout<DH>::THREADS, 2)
    k_prefix_wide(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ1,
                  const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PrefixParams p, int n_prefix) {
  using L = WideLayout<DH>;
  using M16 = Mma16<T16>;
  // (64 keys of a half tile at 2^kLift sum to less than 2^kWideLazy)
  constexpr float kLift = M16::kLifted ? 6.f : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(smem + L::OFF_RED);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* kv_empty = kv_full + L::NS;
  uint64_t* q_full = kv_empty + L::NS;
  uint64_t* s_full = q_full + 1;
  uint64_t* s_read = s_full + 1;  // S is in registers (P_APART)
  uint64_t* p_full = s_read + 1;
  uint64_t* o_full = p_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_full + 1);
  // (through a shuffle, so that what follows from it is known to be alike in a warp)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  constexpr int kTmaWarp = L::SOFT, kMmaWarp = L::SOFT + 1;

  pdl_trigger();  // (the kernels behind wait for this one's results on their own)
  const int rows_tile = wide_rows(p.G);
  Item it;
  int* tokens = reinterpret_cast<int*>(smem + L::OFF_PACK);  // (PACK)
  if constexpr (PACK) {
    Item* found = reinterpret_cast<Item*>(tokens + kWideTile + 64);
    static_assert(L::THREADS / 32 <= 32 && sizeof(Item) <= 64 && alignof(Item) <= 16, "their places");
    if (!pack_item<L::THREADS / 32>(p, rows_tile / p.G, found, reinterpret_cast<int*>(smem + L::OFF_KV),
                                    tokens + kWideTile, tokens + kWideTile + 32, tokens))
      return pdl_wait();
    // (known to be alike in a warp, these are kept in the uniform registers: else
    // the softmax loop, short of registers, is 5 to 10 percent slower)
    const auto alike = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    it.shared = true;
    it.last = false;
    it.b0 = alike(found->b0);
    it.row0 = alike(found->row0);
    it.rows = alike(found->rows);
    it.kvh = alike(found->kvh);
    it.chunk = alike(found->chunk);
    it.tokens = alike(found->tokens);
    it.table_row = alike(found->table_row);
    it.pg0 = alike(found->pg0);
    it.pg1 = alike(found->pg1);
  } else if (!find_item(p, blockIdx.x, n_prefix, rows_tile, it)) {
    return pdl_wait();
  }
  const int np = max(0, it.pg1 - it.pg0);
  const int n = (np + kWidePages - 1) / kWidePages;  // key tiles

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(s_full, 1);
    mbar_init(s_read, 256);
    mbar_init(p_full, 256);
    mbar_init(o_full, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (PACK && threadIdx.x < kWideTile) {  // rows without a query: zeros
    const int r = threadIdx.x;
    if (r >= rows_tile || tokens[r / p.G] < 0) {
      for (int z = 0; z < L::NCH * 8; ++z)
        *reinterpret_cast<uint4*>(smem + z / 8 * L::Q_CH + r * 128 + z % 8 * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, L::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp >= L::SOFT) {
    regs_down<L::FEED_REGS>();
    if (warp == kTmaWarp) {
      // ---------------- Q, then K and V tiles: lane l has the ids of page l % 8 of four tiles
      const int key_tiles = __shfl_sync(0xffffffffu, n, 0), pages = __shfl_sync(0xffffffffu, np, 0);
      const int kvh = __shfl_sync(0xffffffffu, it.kvh, 0);
      const int32_t* table = p.page_table + static_cast<long long>(it.table_row) * p.max_pages + it.pg0;
      const bool elected = elect_one();
      auto page_ids = [&](int i0) {
        int id = 0;
        if (i0 + lane < np) {
          id = table[i0 + lane];
          if (id < 0 || id >= p.n_pages) {
            flag_status(p.status, ST_BAD_PAGE);
            id = p.n_pages;  // outside the tensor map: reads as zeros
          }
        }
        return id;
      };
      int ids = page_ids(0), next = page_ids(32), issued = 0;
      bool ok = true;
      if constexpr (PACK) {  // the tile's tokens, a copy each
        const int live = __shfl_sync(0xffffffffu, min(rows_tile, it.rows - it.row0), 0) / p.G;
        if (elected) mbar_arrive_expect_tx(q_full, live * p.G * L::NCH * 128);
        const int begin = __shfl_sync(0xffffffffu, tokens[0], 0);
        const bool run = live * p.G == rows_tile && __shfl_sync(0xffffffffu, tokens[live - 1], 0) == begin + live - 1;
        if (run && elected) {  // (of entries with all their rows)
#pragma unroll
          for (int cc = 0; cc < L::NCH; ++cc)
            tma_rows(smem_u32(smem) + cc * L::Q_CH, &tmQ, q_full, cc * 64, kvh * p.G, begin);
        }
        for (int t = run ? live : 0; t < live; ++t) {
          const int token = __shfl_sync(0xffffffffu, tokens[t], 0);
          if (elected) {
#pragma unroll
            for (int cc = 0; cc < L::NCH; ++cc)
              tma_rows(smem_u32(smem) + cc * L::Q_CH + t * p.G * 128, &tmQ1, q_full, cc * 64, kvh * p.G, token);
          }
        }
      } else if (elected && key_tiles > 0) {
        // whole tokens: a tile's first row is a token's first head of the group
        mbar_arrive_expect_tx(q_full, rows_tile * L::NCH * 128);
        for (int cc = 0; cc < L::NCH; ++cc)
          tma_rows(smem_u32(smem + cc * L::Q_CH), &tmQ, q_full, cc * 64, it.kvh * p.G, it.b0 * p.T + it.row0 / p.G);
      }
      for (int j = 0; ok && j < key_tiles; ++j) {
        const int npb = min(kWidePages, pages - j * kWidePages);
        if (j > 0 && j % 4 == 0) {
          ids = next;
          next = page_ids((j + 4) * kWidePages);
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int i = 2 * j + kv, s = i % L::NS;
          if (ok && i >= L::NS)
            ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[s], (i / L::NS - 1) & 1, p.status)) != 0;
          if (!ok) break;
          if (elected) mbar_arrive_expect_tx(&kv_full[s], npb * L::NCH * 2048);
          const uint32_t dst = smem_u32(smem + L::OFF_KV) + s * L::SLOT;
#pragma unroll
          for (int g = 0; g < kWidePages; ++g) {
            const int id = __shfl_sync(0xffffffffu, ids, j % 4 * kWidePages + g);
            if (g < npb && elected) {
#pragma unroll
              for (int cc = 0; cc < L::NCH; ++cc)
                tma_page(dst + cc * L::KV_CH + g * 2048, kv ? &tmV : &tmK, &kv_full[s], cc, kvh, id);
            }
          }
          issued = i + 1;
        }
      }
      // every copy has landed before the CTA may leave
      if (key_tiles > 0) mbar_wait(q_full, 0, p.status);
      for (int i = max(0, issued - L::NS); i < issued; ++i) mbar_wait(&kv_full[i % L::NS], (i / L::NS) & 1, p.status);
    } else if (warp == kMmaWarp) {
      // ---------------- MMAs.  Where P lies over S, S(j + 1) waits for P(j) V,
      // else only for the softmax to have S(j) in registers.  The whole warp
      // walks along and one thread issues: the operands are then uniform values
      // (computed by that thread alone, each of them crosses over to the uniform
      // registers on its own: 110 cycles an MMA of 64).
      const int key_tiles = __shfl_sync(0xffffffffu, n, 0), pages = __shfl_sync(0xffffffffu, np, 0);
      const bool elected = elect_one();
      const uint64_t qd = sw128_desc(smem_u32(smem), 16, 1024), kd = sw128_desc(smem_u32(smem + L::OFF_KV), 16, 1024);
      const uint64_t vd = sw128_desc(smem_u32(smem + L::OFF_KV), L::KV_CH, 1024);
      auto wait = [&](uint64_t* bar, int phase) {
        // (polling costs the softmax issue slots and wakes sooner: 128 dimensions 2
        // percent faster with it, 64, where the next S is under way, 2 percent slower)
        const bool up = L::P_APART ? mbar_wait(bar, phase & 1, p.status) : mbar_wait_spin(bar, phase & 1, p.status);
        const bool ok = __all_sync(0xffffffffu, up) != 0;
        tc_fence_after();
        return ok;
      };
      auto kv_wait = [&](int i) { return wait(&kv_full[i % L::NS], i / L::NS); };
      // (a descriptor's address field counts 16 bytes)
      auto issue_s = [&](int j) {
        const uint64_t k = kd + (2 * j) % L::NS * (L::SLOT >> 4);
        const uint32_t id = wide_idesc<T16>(kWideTile, 16 * min(kWidePages, pages - j * kWidePages), false);
        if (elected) {
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks)
            tc_mma_bf16(tmem + L::S_COL, qd + (((ks >> 2) * L::Q_CH + (ks & 3) * 32) >> 4),
                        k + (((ks >> 2) * L::KV_CH + (ks & 3) * 32) >> 4), id, ks > 0 ? 1u : 0u);
          tc_commit(s_full);
          tc_commit(&kv_empty[(2 * j) % L::NS]);
        }
        __syncwarp();
      };
      auto issue_o = [&](int j) {
        const uint64_t v = vd + (2 * j + 1) % L::NS * (L::SLOT >> 4);
        const int npb = min(kWidePages, pages - j * kWidePages);
        const uint32_t id = wide_idesc<T16>(kWideTile, DH, true);
        if (elected) {
#pragma unroll
          for (int ks = 0; ks < kWidePages; ++ks)
            if (ks < npb)
              tc_mma_bf16_ts(tmem + L::O_COL, tmem + L::P_COL + L::P_PAGE * ks, v + ks * (2048 >> 4), id,
                             (j | ks) > 0 ? 1u : 0u);
          tc_commit(o_full);
          tc_commit(&kv_empty[(2 * j + 1) % L::NS]);
        }
        __syncwarp();
      };
      bool ok = key_tiles > 0 && wait(q_full, 0) && kv_wait(0);
      if (ok) issue_s(0);
      for (int j = 0; ok && j < key_tiles; ++j) {
        if (L::P_APART && j + 1 < key_tiles) {
          ok = kv_wait(2 * j + 2) && wait(s_read, j);
          if (ok) issue_s(j + 1);
        }
        ok = ok && kv_wait(2 * j + 1) && wait(p_full, j);
        if (ok) issue_o(j);
        if (!L::P_APART && j + 1 < key_tiles) {
          ok = ok && kv_wait(2 * j + 2) && wait(o_full, j);
          if (ok) issue_s(j + 1);
        }
      }
    }
  } else {
    regs_up<L::SOFT_REGS>();
    // ---------------- softmax: threads r of the two halves own row r
    const int quad = warp & 3, half = warp >> 2, r = quad * 32 + lane;
    const int pair = 1 + quad;  // the named barrier of the row's two warps
    int at, seen;  // the row's place in the output (-1: none; below 2^30) and the keys that it sees
    if constexpr (PACK) {
      const int token = r < rows_tile ? tokens[r / p.G] : -1;
      at = token < 0 ? -1 : token * p.Hq + it.kvh * p.G + r % p.G;
      seen = it.tokens;
    } else {
      const Row row = find_row(p, it, it.row0 + r);
      at = row.live && r < rows_tile ? static_cast<int>(row.at) : -1;
      seen = row.seen;
    }
    const int parts = !PACK && it.last && p.merge ? chunks_of(pages_of(group_of(p, it.b0).tokens), p.p_chunks) : 0;  // of the prefix, to be added at the end
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_at = tmem + lanes + L::S_COL + 64 * half, p_at = tmem + lanes + L::P_COL + 4 * L::P_PAGE * half;
    const uint32_t o_at = tmem + lanes + L::O_COL + DH / 2 * half;
    auto partner = [&](int slot, float v) {  // the other half's value
      red[(slot * L::SOFT + warp) * 32 + lane] = v;
      wide_bar(pair, 64);
      return red[(slot * L::SOFT + (warp ^ 4)) * 32 + lane];
    };
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int npb = min(kWidePages, np - j * kWidePages);
      const int key0 = (it.pg0 + j * kWidePages) * kPage;
      ok = ok && mbar_wait(s_full, j & 1, p.status);
      __syncwarp();
      tc_fence_after();
      uint32_t sv[4][16];
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (4 * half + g < npb) tc_ld_32x32b_x16_nw(s_at + 16 * g, sv[g]);
      tc_wait_ld();
      if (L::P_APART) {
        tc_fence_before();
        mbarrier_arrive_one(s_read);
        // (P(j - 1) V is done before its P is written over, and O is then at rest)
        if (j > 0) ok = ok && mbar_wait(o_full, (j - 1) & 1, p.status);
        __syncwarp();
        tc_fence_after();
      }
      // keys of this half that the row sees (the chunk may end inside the tile)
      const int lim = min(seen, it.pg1 * kPage) - key0 - 64 * half;
      if (__any_sync(0xffffffffu, lim < 64)) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (g * 16 + k >= lim) sv[g][k] = 0xff800000u;  // -infinity
      }
      auto row_top = [&]() {
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int k = 0; k < 16; k += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = wide_max3(mx[e], __uint_as_float(sv[g][k + 2 * e]), __uint_as_float(sv[g][k + 2 * e + 1]));
        return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      };
      // P against m; returns its sum
      auto make_p = [&]() {
        const float mu = m == -INFINITY ? 0.f : m;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), mneg2 = make_float2(-mu, -mu);
        float2 sum[2] = {};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t pk[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 x = __ffma2_rn(
                make_float2(__uint_as_float(sv[g][2 * k]), __uint_as_float(sv[g][2 * k + 1])), sc2, mneg2);
            const float2 e = make_float2(wide_ex2(x.x), wide_ex2(x.y));
            sum[k & 1] = __fadd2_rn(sum[k & 1], e);
            pk[k] = M16::pack(e.x, e.y);
          }
          tc_st_32x32b_x8(p_at + L::P_PAGE * g, pk);
        }
        return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      };
      if (j == 0) {
        float top = row_top();
        top = fmaxf(top, partner(0, top));
        // (rows without a query hold the caller's padding, or what was never
        // written: against +infinity their P is 0 or NaN, and they never vote below)
        m = at >= 0 ? top * p.scale_log2 - kLift : INFINITY;
        l = make_p();
      } else {
        // P against the m so far.  Its sum shows whether m still serves: below
        // 2^kWideLazy no term has grown past 16 bits.  Only where a row of the
        // two warps fails that (an infinity included; a NaN stays one either way)
        // the maxima are taken, m moves and P is made again.
        const float sum = make_p();
        if (!wide_any(pair, sum >= static_cast<float>(1 << kWideLazy) || m == -INFINITY)) {
          l += sum;
        } else {
          float top = row_top();
          top = fmaxf(top, partner(j & 1, top));
          const float cand = fmaxf(m, top * p.scale_log2 - kLift);
          const float al = cand > m ? wide_ex2(m - cand) : 1.f;  // (m = -infinity: 0)
          m = cand;
          // (where P lies over S, S(j) was issued after P(j - 1) V was done)
#pragma unroll
          for (int d = 0; d < DH / 2; d += 16) {
            uint32_t v[16];
            tc_ld_32x32b_x16_nw(o_at + d, v);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
            tc_st_32x32b_x16(o_at + d, v);
          }
          tc_wait_st();  // (the first P has landed before it is written again)
          l = l * al + make_p();
        }
      }
      if (key0 + npb * kPage > it.tokens) {
        // the last page is partial: what its V rows hold past the last token
        // meets probabilities of zero and must be finite
        const int i = 2 * j + 1, first = it.tokens - (key0 + (npb - 1) * kPage);
        ok = ok && mbar_wait(&kv_full[i % L::NS], (i / L::NS) & 1, p.status);
        uint8_t* v = smem + L::OFF_KV + (i % L::NS) * L::SLOT + (npb - 1) * 2048;
        for (int e = half * kWideTile + r; e < (kPage - first) * L::NCH * 8; e += 2 * kWideTile) {
          const int c = e / ((kPage - first) * 8), f = e % ((kPage - first) * 8);
          *reinterpret_cast<uint4*>(v + c * L::KV_CH + first * 128 + f * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tc_wait_st();
      tc_fence_before();
      mbarrier_arrive_one(p_full);
    }
    // the last product: then O is whole, and Q and the ring are free
    if (n > 0) ok = ok && mbar_wait(o_full, (n - 1) & 1, p.status);
    __syncwarp();
    tc_fence_after();
    l += partner(n & 1, l);
    float lse2 = l != 0.f ? m + log2f(l) : -INFINITY;  // (l is a NaN where a score is one)
    float x[DH / 2];  // the row's result, this half's dimensions
    {
      const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int d = 0; d < DH / 2; d += 16) {
        uint32_t v[16];
        if (n > 0) {
          tc_ld_32x32b_x16_nw(o_at + d, v);
          tc_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) x[d + e] = l != 0.f ? __uint_as_float(v[e]) * inv : 0.f;
      }
    }
    const long long R = static_cast<long long>(p.B) * p.T * p.Hq;
    uint8_t *rows = smem + quad * 32 * L::PITCH, *stage = rows + lane * L::PITCH;  // the pair's, this one
    if (it.last && parts > 0) {
      // add the prefix's partial results, a copy of the row at a time (in order)
      pdl_wait();
      float weight = 1.f;
      for (int c = 0; c < parts; ++c) {
        const uint8_t* from = reinterpret_cast<const uint8_t*>(p.part_o + c * R * DH);
        wide_rows_each<DH * 4>(rows, L::PITCH, half, at, [&](uint8_t* d, long long o) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(d)), "l"(from + o) : "memory");
        });
        const float other = at >= 0 ? p.part_lse[c * R + at] : -INFINITY;
        const float top = fmaxf(lse2, other), base = top == -INFINITY ? 0.f : top;
        const float f0 = wide_ex2(lse2 - base), f1 = wide_ex2(other - base);
        asm volatile("cp.async.wait_all;" ::: "memory");
        wide_bar(pair, 64);
#pragma unroll
        for (int d = 0; d < DH / 2; d += 4) {
          const float4 y = *reinterpret_cast<const float4*>(stage + (DH / 2 * half + d) * 4);
          x[d] = x[d] * f0 + (f1 != 0.f ? y.x * f1 : 0.f);
          x[d + 1] = x[d + 1] * f0 + (f1 != 0.f ? y.y * f1 : 0.f);
          x[d + 2] = x[d + 2] * f0 + (f1 != 0.f ? y.z * f1 : 0.f);
          x[d + 3] = x[d + 3] * f0 + (f1 != 0.f ? y.w * f1 : 0.f);
        }
        // (x and weight are relative to 2^top; the first term's weight is 1 where it has any)
        weight = (lse2 != -INFINITY ? weight * f0 : 0.f) + f1;
        lse2 = top;
        wide_bar(pair, 64);  // both halves are through with the copy
      }
      const float inv = weight != 0.f ? 1.f / weight : 0.f;
#pragma unroll
      for (int d = 0; d < DH / 2; ++d) x[d] *= inv;
      lse2 = weight != 0.f ? lse2 + log2f(weight) : -INFINITY;
    }
    if (it.last) {
#pragma unroll
      for (int d = 0; d < DH / 2; d += 8)
        *reinterpret_cast<uint4*>(stage + (DH / 2 * half + d) * 2) =
            make_uint4(M16::pack(x[d], x[d + 1]), M16::pack(x[d + 2], x[d + 3]), M16::pack(x[d + 4], x[d + 5]),
                       M16::pack(x[d + 6], x[d + 7]));
    } else {
#pragma unroll
      for (int d = 0; d < DH / 2; d += 4)
        *reinterpret_cast<float4*>(stage + (DH / 2 * half + d) * 4) = make_float4(x[d], x[d + 1], x[d + 2], x[d + 3]);
    }
    wide_bar(pair, 64);
    const long long part = (it.shared ? it.chunk : p.p_chunks + it.chunk) * R;
    if (it.last) {
      wide_rows_each<DH * 2>(rows, L::PITCH, half, at, [&](uint8_t* d, long long o) {
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + o) = *reinterpret_cast<const uint4*>(d);
      });
      if (at >= 0 && half == 0 && p.lse != nullptr) p.lse[at] = lse2 * 0.69314718055994531f;
    } else {
      uint8_t* to = reinterpret_cast<uint8_t*>(p.part_o + part * DH);
      wide_rows_each<DH * 4>(rows, L::PITCH, half, at, [&](uint8_t* d, long long o) {
        *reinterpret_cast<uint4*>(to + o) = *reinterpret_cast<const uint4*>(d);
      });
      if (at >= 0 && half == 0) p.part_lse[part + at] = lse2;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, L::COLS);
  }
  pdl_wait();  // (the joining kernel behind starts once all of this one has left)
}

template <typename T16, int DH, bool PACK>
cudaError_t launch_wide_t(const PrefixParams& p, long long n_prefix, long long n_own, bool behind,
                          const CUtensorMap& tq, const CUtensorMap& tq1, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  using L = WideLayout<DH>;
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(L::SMEM, [](int v) {
    return cudaFuncSetAttribute(k_prefix_wide<T16, DH, PACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  return launch_k(k_prefix_wide<T16, DH, PACK>, dim3(static_cast<unsigned>(n_prefix + n_own)), dim3(L::THREADS), L::SMEM, s,
                  dim3(1), behind, tq, tq1, tk, tv, p, static_cast<int>(n_prefix));
}

}  // namespace

cudaError_t launch_prefix_wide(const PrefixParams& p, int elem, int head_dim, long long n_prefix, long long n_own,
                               bool behind, const CUtensorMap& tq, const CUtensorMap& tq1, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
  const auto run = [&](auto t, auto pack) {
    using T16 = decltype(t);
    constexpr bool PACK = decltype(pack)::value;
    return head_dim == 64 ? launch_wide_t<T16, 64, PACK>(p, n_prefix, n_own, behind, tq, tq1, tk, tv, s)
                          : launch_wide_t<T16, 128, PACK>(p, n_prefix, n_own, behind, tq, tq1, tk, tv, s);
  };
  const bool pack = n_own == 0 && p.pack;
  if (elem == DFLASH_ELEM_BF16)
    return pack ? run(__nv_bfloat16{}, std::true_type{}) : run(__nv_bfloat16{}, std::false_type{});
  return pack ? run(__half{}, std::true_type{}) : run(__half{}, std::false_type{});
}

}  // namespace dflash
