// dflash_prefix_attention: attention of a batch over prefixes that groups of
// sequences share and over each sequence's own tokens, on a paged cache.
//
// A query row r sees the keys of its group's prefix and keys of its own
// sequence.  Softmax attention over a union of key sets splits exactly: with
// z = scale q.k, each set S gives l_S = log sum_S exp z and o_S = sum_S
// exp(z - l_S) v, and
//     out = sum_S exp(l_S - l) o_S,  l = log sum_S exp l_S.
// So a prefix is read once for all query rows of its group (as one tall
// matrix of rows) and each sequence's own keys for its own rows.  Parts of
// more than 8 rows are the wide kernel's (prefix_wide.cu: tcgen05, chunks of
// pages), those of fewer the thin one's (here: mma.sync, warps that stream
// pages).  Partial results are joined in a fixed order: by the wide kernel's
// own parts where they are whole and the prefix has at most four chunks, else
// by a kernel of its own.
#include <algorithm>

#include "prefix_common.cuh"
#include "tma_map.h"

namespace dflash {

namespace {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

constexpr int kThinRows = 8;    // query rows of a tile (a multiple of the 8 columns of an MMA)
constexpr int kThinPages = 1;   // pages that a warp takes at least (one sequence of 577 tokens: 1 7.4 us, 2 9.9, 4 10.9)
constexpr int kMaxEntries = 4096;  // batch entries, and groups, of a call

template <int DH>
struct ThinLayout {
  // Warps and pages in flight a warp.  Heads of 128 (64): 64 sequences of up to
  // 1500 tokens beside a shared prefix, 4 warps x 3 pages 68 us, 6 x 2 58; 64
  // sequences of 1024 (64 query heads of 64), 33 and 37.
  static constexpr int WARPS = DH == 64 ? 4 : 6, THREADS = WARPS * 32, STAGES = DH == 64 ? 3 : 2;
  static constexpr int CTAS = DH == 64 ? 4 : 2;           // that an SM holds
  static constexpr int HALF_PAGE = kPage * DH * 2;        // bytes of a page of K (or V) of one head
  static constexpr int STAGE = 2 * HALF_PAGE;
  static constexpr int WARP = STAGES * STAGE;
  static constexpr int OFF_SCAN = WARPS * WARP;
  static constexpr int OFF_BAR = OFF_SCAN + 64;
  static constexpr int BYTES = OFF_BAR + WARPS * STAGES * 8;
  static constexpr int SMEM = 1024 + BYTES;               // + the line: first pages of its elements, their rows and pages
  static_assert(BYTES % 16 == 0, "the line is aligned");
};

// The thin kernel's work is a line of pages: for every group (where it takes
// the prefixes) and then every entry, its row tiles x kv heads x pages.  Warp
// w of the grid takes pages [w * per, (w + 1) * per) of the line, whatever
// parts they belong to, so that all warps stream alike however uneven the
// lengths are.  A part (one tile and head) that one warp takes whole goes to
// whole_*; of one that several share, each leaves its share in its own slot:
// 2w if the share starts at the warp's first page, 2w + 1 otherwise.
// Rows and pages of element e (groups, then entries) of the line.
struct ThinPart {
  bool shared;
  int b0, rows, tokens, table_row;
};
constexpr int kThinHeld = 512;  // elements whose rows and pages the CTA holds in shared memory
__device__ __forceinline__ ThinPart thin_read(const PrefixParams& p, int groups, int e) {
  ThinPart t;
  t.shared = e < groups;
  if (t.shared) {
    t.b0 = p.group_off[e];
    t.rows = (p.group_off[e + 1] - t.b0) * p.T * p.G;
    t.table_row = p.prefix_seq[e];
  } else {
    t.b0 = e - groups;
    t.rows = entry_rows(p, t.b0) * p.G;
    t.table_row = p.seq != nullptr ? p.seq[t.b0] : t.b0;
  }
  t.tokens = seq_tokens(p, t.table_row);
  return t;
}
__device__ __forceinline__ int thin_tiles(int rows, int tile) { return (rows + tile - 1) / tile; }

// Where an element's rows and pages are held, behind the line's first pages.
__device__ __forceinline__ int4* thin_held(long long* first, int n) {
  return reinterpret_cast<int4*>(first + (n + 2) / 2 * 2);
}

// The same, from the copy that thin_line() left there.
__device__ __forceinline__ ThinPart thin_part(const PrefixParams& p, int groups, long long* first, int e) {
  const int n = groups + p.B;
  if (n > kThinHeld) return thin_read(p, groups, e);
  const int4 v = thin_held(first, n)[e];
  return ThinPart{e < groups, v.x, v.y, v.z, v.w};
}

// Sets the line up: first[e] for every element and the length after the last
// (the whole CTA of WARPS warps; ok: the group bounds are sound; check: look at
// the elements' sequences and flag bad ones).
template <int WARPS>
__device__ __forceinline__ void thin_line(const PrefixParams& p, int groups, bool ok, bool check, long long* first,
                                          int4* held, long long* scan) {
  const int n = groups + p.B, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long before = 0;
  for (int e0 = 0; e0 < n; e0 += WARPS * 32) {
    const int e = e0 + threadIdx.x;
    long long size = 0;
    if (e < n && (e >= groups || ok)) {
      const ThinPart t = thin_read(p, groups, e);
      if (held != nullptr) held[e] = make_int4(t.b0, t.rows, t.tokens, t.table_row);
      size = static_cast<long long>(thin_tiles(t.rows, kThinRows)) * p.Hkv * pages_of(t.tokens);
      if (check) {
        if (t.shared) check_prefix(p, t.table_row);
        else check_entry(p, t.b0, t.table_row);
      }
    }
    long long sum = size;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) scan[warp] = sum;
    __syncthreads();
    long long all = 0;
    for (int q = 0; q < WARPS; ++q) {
      if (q < warp) sum += scan[q];
      all += scan[q];
    }
    if (e < n) first[e] = before + sum - size;
    before += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) first[n] = before;
  __syncthreads();
}

// The element that page f of the line belongs to: the last e with first[e] <= f.
__device__ __forceinline__ int thin_find(const long long* first, int n, long long f) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= f) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// a / b of non-negative numbers (64-bit divisions are long; few need one).
__device__ __forceinline__ long long thin_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

__device__ __forceinline__ long long thin_per(long long length, int warps) {
  const long long per = thin_div(length + warps - 1, warps);
  return per < kThinPages ? kThinPages : per;
}

__device__ __forceinline__ float thin_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The transpose of an 8 x 8 matrix of 16-bit values (row g, columns 2t and 2t + 1 in lane 4g + t).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// Independent warps, each with a ring of pages that runs on over the parts it
// takes, and its own running maxima, sums and outputs.  The products are taken
// transposed, S^T = K Q^T and O^T = V^T P^T, so that keys and dimensions fill
// the 16 rows of an MMA and the query rows its 8 columns.
//
// Bound by memory while it streams (64 sequences, 8 kv heads of 128: from 1024
// to 1500 tokens 125 MB in 18.4 us, 6.8 TB/s); what is left is what a call takes
// to start and to join: 64 sequences of 1024 tokens take 51 us, 5.2 TB/s, one
// of 77 tokens 7.1.  Until a warp's first page is there: 1.3 us for the line,
// 1.4 for the first page ids, 1.2 for the copy.
template <typename T16, int DH>
__global__ void __launch_bounds__(ThinLayout<DH>::THREADS) k_prefix_thin(const __grid_constant__ CUtensorMap tmK,
                                                              const __grid_constant__ CUtensorMap tmV,
                                                              const __grid_constant__ PrefixParams p) {
  using L = ThinLayout<DH>;
  using M = Mma16<T16>;
  constexpr int KS = DH / 16, NR = kThinRows / 8;
  constexpr float kLift = M::kLifted ? 15.f : 0.f;  // (m moves with every page: no weight is above 2^kLift)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  long long* first = reinterpret_cast<long long*>(smem + L::BYTES);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int gr = lane >> 2, t4 = lane & 3;

  pdl_trigger();  // (the joining kernel waits for this one's results on its own)
  const int groups = p.p_thin ? p.NG : 0, n_line = groups + p.B;
  const bool sound = p.NG == 0 || bounds_ok(p);
  if (blockIdx.x == 0 && threadIdx.x == 0 && !sound) flag_status(p.status, ST_BAD_BLOCK);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR) + warp * L::STAGES;
  if (lane == 0) {
    for (int s = 0; s < L::STAGES; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  thin_line<L::WARPS>(p, groups, sound, blockIdx.x == 0, first, n_line <= kThinHeld ? thin_held(first, n_line) : nullptr,
                        reinterpret_cast<long long*>(smem + L::OFF_SCAN));
  const long long length = first[n_line], per = thin_per(length, p.warps);
  if (blockIdx.x == 0 && n_line > kThinHeld) {  // (a shorter line the joining kernel sets up itself)
    for (int e = threadIdx.x; e <= n_line; e += L::THREADS) p.work[e] = first[e];
  }
  const int self = blockIdx.x * L::WARPS + warp;
  const long long f0 = self * per, f1 = min(length, f0 + per);
  const int mine = f1 > f0 ? static_cast<int>(f1 - f0) : 0;
  uint8_t* ring = smem + warp * L::WARP;

  // page id and kv head of this warp's next 32 pages, one per lane
  int ids = 0, heads = 0;
  auto fetch_ids = [&](int i0) {
    const int i = i0 + lane;
    if (i < mine) {
      const int e = thin_find(first, n_line, f0 + i);
      const ThinPart t = thin_part(p, groups, first, e);
      const int pages = pages_of(t.tokens);
      const long long x = f0 + i - first[e];
      const int unit = static_cast<int>(thin_div(x, pages)), pg = static_cast<int>(x - static_cast<long long>(unit) * pages);
      heads = unit % p.Hkv;
      ids = p.page_table[static_cast<long long>(t.table_row) * p.max_pages + pg];
      if (ids < 0 || ids >= p.n_pages) {
        flag_status(p.status, ST_BAD_PAGE);
        ids = p.n_pages;  // outside the tensor map: reads as zeros
      }
    }
  };
  const bool elected = elect_one();
  auto issue = [&](int i) {
    if (i > 0 && (i & 31) == 0) fetch_ids(i);
    const int id = __shfl_sync(0xffffffffu, ids, i & 31), head = __shfl_sync(0xffffffffu, heads, i & 31);
    const int s = i % L::STAGES;
    const uint32_t kd = smem_u32(smem) + warp * L::WARP + s * L::STAGE;
    if (elected) {
      mbar_arrive_expect_tx(&bars[s], L::STAGE);
      tma_page(kd, &tmK, &bars[s], 0, head, id);
      tma_page(kd + L::HALF_PAGE, &tmV, &bars[s], 0, head, id);
    }
    __syncwarp();
  };
  // ldmatrix lane addresses within a [16 keys][128 bytes] swizzled box
  const int lr = lane & 7, lm = lane >> 3;
  const int k_key = (lm & 1) * 8 + lr, k_unit = lm >> 1;  // K: (keys, d), (keys + 8, d), (keys, d + 8), ..
  const int v_key = (lm >> 1) * 8 + lr, v_unit = lm & 1;  // V, transposed: (keys, d), (keys, d + 8), (keys + 8, d), ..
  const long long R = static_cast<long long>(p.B) * p.T * p.Hq;

  fetch_ids(0);
  bool ok = true;
  int i = 0;
  while (i < mine && ok) {
    // the part that page i belongs to, and this warp's share of it
    const int e = thin_find(first, n_line, f0 + i);
    const ThinPart part = thin_part(p, groups, first, e);
    const int pages = pages_of(part.tokens);
    const long long x = f0 + i - first[e];
    const int unit = static_cast<int>(thin_div(x, pages)), pg0 = static_cast<int>(x - static_cast<long long>(unit) * pages);
    const int share = min(pages - pg0, mine - i);
    Item it;
    it.shared = part.shared;
    it.b0 = part.b0;
    it.rows = part.rows;
    it.tokens = part.tokens;
    it.kvh = unit % p.Hkv;
    it.row0 = unit / p.Hkv * kThinRows;

    // query row 8j + gr as a B fragment
    uint32_t qf[NR][KS][2];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const Row row = find_row(p, it, it.row0 + 8 * j + gr);
      const T16* src = static_cast<const T16*>(p.q) + row.token * p.ld_q + (row.at - row.token * p.Hq) * DH + 2 * t4;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[j][ks][0] = row.live ? *reinterpret_cast<const uint32_t*>(src + ks * 16) : 0u;
        qf[j][ks][1] = row.live ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8) : 0u;
      }
    }
    if (i == 0) {  // (the pages' first copies, behind the loads of the first queries)
      for (int c = 0; c < min(mine, L::STAGES); ++c) issue(c);
    }
    // rows 8j + 2 t4 and the next one are this thread's in S^T and O^T
    int seen[NR][2];
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) seen[j][c] = find_row(p, it, it.row0 + 8 * j + 2 * t4 + c).seen;
    float o[NR][KS][4] = {};
    float m[NR][2], l[NR][2] = {};
#pragma unroll
    for (int j = 0; j < NR; ++j) m[j][0] = m[j][1] = -INFINITY;

    for (int c = 0; c < share; ++c, ++i) {
      const int s = i % L::STAGES;
      ok = ok && mbar_wait(&bars[s], (i / L::STAGES) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok) != 0;
      if (!ok) break;
      const int key0 = (pg0 + c) * kPage;
      const uint32_t kd = smem_u32(ring + s * L::STAGE), vd = kd + L::HALF_PAGE;
      // values past the last token would meet probabilities of zero: they must be finite
      if (key0 + kPage > it.tokens) {
        const int held = it.tokens - key0;
        for (int z = lane; z < (kPage - held) * (DH / 64) * 8; z += 32) {
          const int ch = z / ((kPage - held) * 8), f = z % ((kPage - held) * 8);
          *reinterpret_cast<uint4*>(ring + s * L::STAGE + L::HALF_PAGE + ch * 2048 + held * 128 + f * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // (a later page's copy comes to the same place)
        __syncwarp();
      }
      float sc[NR][2][4] = {};  // (two chains: the products of even and odd steps)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t ka[4];
        const int u = (ks & 3) * 2 + k_unit;
        ldsm_x4(kd + (ks >> 2) * 2048 + k_key * 128 + ((u ^ (k_key & 7)) << 4), ka);
#pragma unroll
        for (int j = 0; j < NR; ++j) M::mma(sc[j][ks & 1], ka, qf[j][ks][0], qf[j][ks][1]);
      }
      uint32_t pb[NR][2];
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        // z[q]: key gr + 8 (q / 2), row 8j + 2 t4 + q % 2
        float z[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          z[q] = key0 + gr + (q >> 1) * 8 < seen[j][q & 1] ? (sc[j][0][q] + sc[j][1][q]) * p.scale_log2 : -INFINITY;
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = fmaxf(z[h], z[2 + h]);
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float mn = fmaxf(m[j][h], mx - kLift), ms = mn == -INFINITY ? 0.f : mn;
          al[h] = thin_ex2(m[j][h] - ms);
          m[j][h] = mn;
          z[h] = thin_ex2(z[h] - ms);
          z[2 + h] = thin_ex2(z[2 + h] - ms);
          l[j][h] = l[j][h] * al[h] + (z[h] + z[2 + h]);
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int d = 0; d < KS; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q) o[j][d][q] *= al[q & 1];
        }
        pb[j][0] = transpose8(M::pack(z[0], z[1]));
        pb[j][1] = transpose8(M::pack(z[2], z[3]));
      }
#pragma unroll
      for (int d = 0; d < KS; ++d) {
        uint32_t va[4];
        const int u = (d & 3) * 2 + v_unit;
        ldsm_x4_t(vd + (d >> 2) * 2048 + v_key * 128 + ((u ^ (v_key & 7)) << 4), va);
#pragma unroll
        for (int j = 0; j < NR; ++j) M::mma(o[j][d], va, pb[j][0], pb[j][1]);
      }
      __syncwarp();
      if (i + L::STAGES < mine) issue(i + L::STAGES);
    }

    // the share's result, normalised by its own sum
    const bool all = pg0 == 0 && share == pages;
    const int slot = 2 * self + (x + first[e] == f0 ? 0 : 1);
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[j][h] += __shfl_xor_sync(0xffffffffu, l[j][h], w);
        const int r = 8 * j + 2 * t4 + h;
        const Row row = find_row(p, it, it.row0 + r);
        if (!row.live) continue;
        const long long at = all ? (it.shared ? 0 : R) + row.at : static_cast<long long>(slot) * kThinRows + r;
        const float inv = l[j][h] != 0.f ? 1.f / l[j][h] : 0.f;
        float* dst = (all ? p.whole_o : p.slot_o) + at * DH + gr;
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          dst[16 * d] = o[j][d][h] * inv;
          dst[16 * d + 8] = o[j][d][2 + h] * inv;
        }
        if (gr == 0) (all ? p.whole_lse : p.slot_lse)[at] = l[j][h] != 0.f ? m[j][h] + log2f(l[j][h]) : -INFINITY;
      }
  }
  if (!ok) {  // a wait gave up: what is still in flight gets its own bounded waits before the CTA leaves
    for (int c = i; c < min(mine, i + L::STAGES); ++c) mbar_wait(&bars[c % L::STAGES], (c / L::STAGES) & 1, p.status);
  }
  pdl_wait();  // (the joining kernel starts its work once all of this one has left, and what ran before it)
}

constexpr int kJoinWarps = 8;

// out of the partial results: `share` warps (1 or 8) a query row, each adding
// every share-th part, and `rows` rows one after the other (an entry's rows have
// its lookups in common).  Parts: of the prefix, then of the entry's own sequence;
// the wide kernel leaves them by chunk, the thin one as said above.
template <typename T16, int DH, int PARTS>
__global__ void __launch_bounds__(kJoinWarps * 32) k_prefix_join(const __grid_constant__ PrefixParams p, int share, int rows) {
  using M = Mma16<T16>;
  constexpr int E = DH / 32;  // elements a lane
  __shared__ float s_a[kJoinWarps][DH], s_sum[kJoinWarps], s_top[kJoinWarps];
  __shared__ long long s_first[kThinHeld + 1], s_scan[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % share;
  const int R = p.B * p.T * p.Hq;  // (below 2^30)
  const int row0 = (blockIdx.x * (kJoinWarps / share) + warp / share) * rows;
  int at_b = -1, rows_b = 0, own = 0;
  Group g{0, 0, -1, 0, 0, 0};
  auto entry = [&](int row) {  // what the row's entry has, once for all its rows
    const int b = row / (p.Hq * p.T);
    if (row >= R || b == at_b) return;
    at_b = b;
    rows_b = entry_rows(p, b);
    g = group_of(p, b);
    own = pages_of(seq_tokens(p, p.seq != nullptr ? p.seq[b] : b));
  };
  entry(row0);
  // the thin kernel's line (a long one is read where that kernel left it)
  const int groups = p.p_thin ? p.NG : 0;
  const bool held = groups + p.B <= kThinHeld;
  const long long* first = held ? s_first : p.work;
  if (p.warps > 0 && held)
    thin_line<kJoinWarps>(p, groups, p.NG == 0 || bounds_ok(p), false, s_first, nullptr, s_scan);
  if (!held) pdl_wait();
  for (int i = 0; i < rows; ++i) {
    const int row = row0 + i;
    entry(row);
    const int tok = row / p.Hq, b = tok / p.T, t = tok - b * p.T, h = row - tok * p.Hq, kvh = h / p.G;
    const bool live = row < R && t < rows_b;
    // [0] the prefix's parts, [1] the own ones: how many, and where they are
    int n[2] = {0, 0}, lane_row[2] = {0, 0};
    long long f0[2] = {0, 0}, w0[2] = {0, 0};  // (thin) first page on the line, and the warp that takes it
    long long per = 1;
    if (live) {
      const int pre = pages_of(g.tokens);
      if (p.p_chunks > 0) n[0] = chunks_of(pre, p.p_chunks);
      if (p.s_chunks > 0) n[1] = chunks_of(own, p.s_chunks);
      if (p.warps > 0) per = thin_per(first[groups + p.B], p.warps);
      auto on_line = [&](int which, int e, int pages, int r) {
        f0[which] = first[e] + static_cast<long long>(r / kThinRows * p.Hkv + kvh) * pages;
        w0[which] = thin_div(f0[which], per);
        lane_row[which] = r % kThinRows;
        n[which] = pages > 0 ? static_cast<int>(thin_div(f0[which] + pages - 1, per) - w0[which]) + 1 : 0;
      };
      const int gi = h - kvh * p.G;
      if (p.p_thin && pre > 0) on_line(0, g.index, pre, ((b - g.lo) * p.T + t) * p.G + gi);
      if (p.s_chunks == 0) on_line(1, groups + b, own, t * p.G + gi);
    }
    const int n_all = n[0] + n[1];
    // where part c is: its log-sum-exp, and its output
    auto place = [&](int c, const float*& lse, const float*& o) {
      const int which = c < n[0] ? 0 : 1, k = which ? c - n[0] : c;
      long long at;
      if (which ? p.s_chunks > 0 : p.p_chunks > 0) {
        at = (which ? p.p_chunks + k : k) * static_cast<long long>(R) + row;
        lse = p.part_lse;
        o = p.part_o;
      } else if (n[which] == 1) {
        at = which * static_cast<long long>(R) + row;
        lse = p.whole_lse;
        o = p.whole_o;
      } else {
        const long long w = w0[which] + k;
        at = (2 * w + (k > 0 || f0[which] == w * per ? 0 : 1)) * kThinRows + lane_row[which];
        lse = p.slot_lse;
        o = p.slot_o;
      }
      lse += at;
      o += at * DH;
    };
    // PARTS parts (of 4, 16) at a time: a lane finds one and its weight, then all add
    // them up.  What they need from before is found first, so that one wait for
    // memory is left once the partial results are there.
    float mx = -INFINITY, sum = 0.f, a[E] = {};
    for (int c0 = 0; c0 * share + sub < n_all || c0 == 0; c0 += PARTS) {
      const int c = (c0 + (lane & (PARTS - 1))) * share + sub;
      const int count = min(PARTS, (n_all - sub + share - 1) / share - c0);
      const float *lse = nullptr, *mine = nullptr;
      if (c < n_all) place(c, lse, mine);
      const unsigned long long addr = reinterpret_cast<unsigned long long>(mine);
      if (c0 == 0 && i == 0 && held) pdl_wait();
      const float z = c < n_all && lane < PARTS ? *lse : -INFINITY;
      float v[PARTS][E];
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, addr, k)) + lane * E;
        if (k >= count) {
#pragma unroll
          for (int e = 0; e < E; ++e) v[k][e] = 0.f;
        } else if constexpr (E == 4) {
          *reinterpret_cast<float4*>(v[k]) = *reinterpret_cast<const float4*>(src);
        } else {
          *reinterpret_cast<float2*>(v[k]) = *reinterpret_cast<const float2*>(src);
        }
      }
      const float top = fmaxf(mx, warp_max(z)), at = top == -INFINITY ? 0.f : top;
      const float keep = exp2f(mx - at), f = exp2f(z - at);
      mx = top;
      sum = sum * keep + warp_sum(f);
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] *= keep;
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const float w = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] += w * v[k][e];
      }
    }
    if (share > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) s_a[warp][lane * E + e] = a[e];
      if (lane == 0) {
        s_sum[warp] = sum;
        s_top[warp] = mx;
      }
      __syncthreads();
      if (warp != 0) return;
      for (int w = 0; w < kJoinWarps; ++w) mx = fmaxf(mx, s_top[w]);
      const float at = mx == -INFINITY ? 0.f : mx;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        const float f = exp2f(s_top[w] - at);
        sum += f * s_sum[w];
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] += f * s_a[w][lane * E + e];
      }
    }
    const float ms = mx == -INFINITY ? 0.f : mx;
    if (!live) continue;
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    T16* dst = static_cast<T16*>(p.out) + static_cast<long long>(row) * DH + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = M::pack(a[e] * inv, a[e + 1] * inv);
    if (lane == 0 && p.lse != nullptr) p.lse[row] = sum != 0.f ? (ms + log2f(sum)) * 0.69314718055994531f : -INFINITY;
  }
}

// ------------------------------------------------------------------ host side

// From this many query rows (of an entry; of a group on average) on, the wide
// kernel takes them: where a second thin tile would read the keys again.
// Thin / wide, heads of 128 with 4 (8) query heads a kv head, 64 sequences of
// 1024 tokens: 4 rows 51 / 53 us, 8 rows 56 / 54, 16 rows 71 / 55; two
// sequences of 300: 4 rows 7.5 / 10.1, 8 rows 7.7 / 10.2, 16 rows 11.3 / 10.5;
// a prefix of 131000: 8 rows 91 / 89, 16 rows 148 / 90.
constexpr int kWideFrom = 9;

struct PrefixPlan {
  bool p_wide, s_wide;         // whether the wide kernel takes the prefix, the own parts (else the thin one)
  bool pack;                   // prefix row tiles hold live rows only (where n_rows is given)
  bool merge, join;            // own parts add the prefix's partial results; a kernel joins them all
  long long p_tiles, s_tiles;  // row tiles of the wide kernel: of all groups (a bound), of an entry
  long long rows;
  int sms;
  int p_chunks, s_chunks;      // of the wide kernel's parts (0: the thin kernel's)
  int warps;                   // of the thin kernel (0: not used)
  size_t off_work, off_lse, off_o, off_whole_lse, off_whole_o, off_slot_lse, off_slot_o, bytes;
};

int plan_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 152;
  }
  return n;
}

// Chunks of a wide item: the count that takes the least time on `slots` CTAs
// at once, a CTA costing its key tiles and about three more to start and to
// write its rows.  Items of one length run in waves; of several (the mean taken
// as 0.6 of the longest) they fill the slots and leave the longest as a tail.
int plan_chunks(long long items, int tokens, long long slots, bool even, double join) {
  const int tiles = std::max(1, (tokens + 127) / 128);
  int best = 1;
  double cost = 1e300;
  for (int c = 1; c <= std::min(tiles, 64); ++c) {
    const double per = (tiles + c - 1) / c + 3, n = static_cast<double>(items) * c / slots;
    double t = per;
    if (n > 1 && even) t = static_cast<double>((items * c + slots - 1) / slots) * per;
    else if (n > 1) t = n * (0.6 * tiles / c + 3) + per;
    if (c > 1) t += join;
    if (t < cost) {
      cost = t;
      best = c;
    }
  }
  return best;
}

bool make_plan(const dflash_paged_kv& kv, int Hq, int B, int T, int NG, int max_prefix, int max_len, PrefixPlan* out) {
  const int G = Hq / kv.n_kv_heads, Hkv = kv.n_kv_heads;
  const long long tg = static_cast<long long>(T) * G;
  const int cap = kv.max_pages * kPage;
  const int mp = max_prefix > 0 ? std::min(max_prefix, cap) : cap, ml = max_len > 0 ? std::min(max_len, cap) : cap;
  PrefixPlan r{};
  r.rows = static_cast<long long>(B) * T * Hq;
  const bool fits = G <= kWideTile;  // (a token's heads stay in one row tile)
  r.s_wide = fits && tg >= kWideFrom;
  r.p_wide = fits && NG > 0 && (r.s_wide || B * tg >= static_cast<long long>(kWideFrom) * NG);
  const int sms = plan_sms(), rows = wide_rows(std::min(G, kWideTile));
  r.sms = sms;
  if (r.p_wide) {
    r.p_tiles = (B * tg + static_cast<long long>(NG) * (rows - 1)) / rows;
    // Packing the live rows takes a tile longer (3 us, and 4 percent of the loop)
    // and pays where it saves CTAs a turn: 48 entries of 16 rows x 64 heads, a
    // prefix of 8192, 160 us unpacked; packed 165 with all rows live, 96 with
    // half of them.  In one turn (32 entries of 17 rows x 32 heads, 16384) the
    // longest CTA stays as long: 134 us unpacked, packed 143 and 133.
    r.pack = r.p_tiles * Hkv > 2ll * sms;
    // Beside a thin kernel that reads as much (it waits for memory) one CTA an
    // SM, else two: 4 sequences of 300 tokens behind 131000, 118 and 93 us.
    const bool beside = !r.s_wide && static_cast<long long>(B) * ml >= static_cast<long long>(NG) * mp;
    r.p_chunks = plan_chunks(r.p_tiles * Hkv, mp, beside ? sms : 2 * sms, NG == 1, 0);
  }
  if (r.s_wide) {
    r.s_tiles = (tg + rows - 1) / rows;
    r.s_chunks = plan_chunks(B * r.s_tiles * Hkv, ml, 2 * sms, B == 1, 4);
    // (a wide own part adds a row's copies one after the other)
    r.merge = NG > 0 && r.s_chunks == 1 && r.p_chunks <= 4;
    r.join = r.s_chunks > 1 || (NG > 0 && !r.merge);
  } else {
    // as many warps as the SMs hold, or as there can be shares of kThinPages pages
    const auto tiles = [](long long n) { return (n + kThinRows - 1) / kThinRows; };
    const long long line = B * tiles(tg) * Hkv * ((ml + kPage - 1) / kPage) +
                           (NG > 0 && !r.p_wide ? (tiles(B * tg) + NG) * Hkv * ((mp + kPage - 1) / kPage) : 0);
    // (beside the wide kernel's CTAs half of them: all of a line's warps start at once)
    const bool d64 = kv.head_dim == 64;
    const int per_cta = d64 ? ThinLayout<64>::WARPS : ThinLayout<128>::WARPS;
    const int ctas = d64 ? ThinLayout<64>::CTAS : ThinLayout<128>::CTAS;
    const long long most = static_cast<long long>(sms) * ctas / (r.p_wide ? 2 : 1) * per_cta;
    const long long want = (line + kThinPages - 1) / kThinPages;
    r.warps = static_cast<int>(std::min(most, (want + per_cta - 1) / per_cta * per_cta));
    r.join = true;
  }
  if (r.p_tiles * Hkv * r.p_chunks > INT32_MAX || B * r.s_tiles * Hkv * r.s_chunks > INT32_MAX) return false;
  const size_t parts = r.join || r.merge ? r.p_chunks + (r.join ? r.s_chunks : 0) : 0;
  const size_t dh = kv.head_dim, whole = r.warps > 0 ? 2 * r.rows : 0, slots = 2ull * r.warps * kThinRows;
  size_t off = 256;  // (the first 256 bytes: a status word for callers without one)
  const auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  r.off_work = take(r.warps > 0 ? 8 * (static_cast<size_t>(NG) + B + 1) : 0);
  r.off_lse = take(4 * r.rows * parts);
  r.off_whole_lse = take(4 * whole);
  r.off_slot_lse = take(4 * slots);
  r.off_o = take(4 * r.rows * parts * dh);
  r.off_whole_o = take(4 * whole * dh);
  r.off_slot_o = take(4 * slots * dh);
  r.bytes = off;
  *out = r;
  return true;
}

dflash_status check_prefix(const dflash_paged_kv* kv, int Hq, int B, int T, int NG, int max_prefix, int max_len) {
  if (!paged_kv_ok(kv) || B < 1 || T < 1 || NG < 0 || max_prefix < 0 || max_len < 0 || Hq < 1)
    return DFLASH_ERR_INVALID_ARG;
  if (Hq % kv->n_kv_heads) return DFLASH_ERR_INVALID_ARG;
  if (kv->elem == DFLASH_ELEM_F32 || (kv->head_dim != 64 && kv->head_dim != 128)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  // row counts stay well inside 32 bits
  if (static_cast<long long>(B) * T * Hq > INT32_MAX / 2 || B > kMaxEntries || NG > kMaxEntries)
    return DFLASH_ERR_UNSUPPORTED_SHAPE;
  return DFLASH_OK;
}

// Pages of one layer as a 5-D map (64 elements, token, chunk of 64, head, page)
// with boxes of 16 tokens x `chunks` chunks (128-byte swizzled rows).
bool page_map(const dflash_paged_kv& kv, void* base, int chunks, CUtensorMap* out) {
  const auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dh = kv.head_dim;
  const cuuint64_t gdim[5] = {64, kPage, dh / 64, static_cast<cuuint64_t>(kv.n_kv_heads),
                              static_cast<cuuint64_t>(kv.n_pages)};
  const cuuint64_t gstride[4] = {dh * 2, 128, dh * 2 * kPage, dh * 2 * kPage * kv.n_kv_heads};
  const cuuint32_t box[5] = {64, kPage, static_cast<cuuint32_t>(chunks), 1, 1}, es[5] = {1, 1, 1, 1, 1};
  return fn(out, kv.elem == DFLASH_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
            base, gdim, gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as a 3-D map (elements, heads, tokens) with boxes of 64 elements x
// the group's heads x box_tokens.
bool query_map(const dflash_paged_kv& kv, const void* q, int Hq, long long tokens, long long ld, int box_tokens,
               CUtensorMap* out) {
  const auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const int G = Hq / kv.n_kv_heads;
  const cuuint64_t gdim[3] = {static_cast<cuuint64_t>(kv.head_dim), static_cast<cuuint64_t>(Hq),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t gstride[2] = {static_cast<cuuint64_t>(kv.head_dim) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(box_tokens)}, es[3] = {1, 1, 1};
  return fn(out, kv.elem == DFLASH_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(q), gdim, gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct PrefixMaps {
  CUtensorMap q, q_one, wide_k, wide_v, thin_k, thin_v;
};

template <typename T16, int DH>
cudaError_t launch_thin(const PrefixParams& p, bool behind, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t s) {
  const int line = (p.p_thin ? p.NG : 0) + p.B;
  const int smem = ThinLayout<DH>::SMEM + (line + 2) / 2 * 16 + (line <= kThinHeld ? line * 16 : 0);
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(smem, [](int v) {
    return cudaFuncSetAttribute(k_prefix_thin<T16, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  return launch_k(k_prefix_thin<T16, DH>, dim3(p.warps / ThinLayout<DH>::WARPS), dim3(ThinLayout<DH>::THREADS), smem, s, dim3(1), behind,
                  tk, tv, p);
}

template <typename T16, int DH>
cudaError_t launch_prefix(const PrefixParams& p, const PrefixPlan& plan, int elem, const PrefixMaps& m, cudaStream_t s) {
  const long long n_prefix = plan.p_tiles * plan.p_chunks * p.Hkv, n_own = p.B * plan.s_tiles * plan.s_chunks * p.Hkv;
  cudaError_t e = cudaSuccess;
  if (plan.p_wide) e = launch_prefix_wide(p, elem, DH, n_prefix, 0, false, m.q, m.q_one, m.wide_k, m.wide_v, s);
  if (e == cudaSuccess)
    e = plan.s_wide ? launch_prefix_wide(p, elem, DH, 0, n_own, plan.p_wide, m.q, m.q_one, m.wide_k, m.wide_v, s)
                    : launch_thin<T16, DH>(p, plan.p_wide, m.thin_k, m.thin_v, s);
  if (e != cudaSuccess || !plan.join) return e;
  // few rows: a row's parts over all the warps of a CTA
  // (many rows: as many warps as the SMs hold at once take several)
  const int share = plan.rows < 8ll * plan.sms ? kJoinWarps : 1;
  const int rows = static_cast<int>((plan.rows + 32ll * plan.sms - 1) / (32ll * plan.sms));
  const long long per = static_cast<long long>(kJoinWarps / share) * rows;
  const auto join = [&](auto kernel) {
    return launch_k(kernel, dim3(static_cast<unsigned>((plan.rows + per - 1) / per)), dim3(kJoinWarps * 32), 0, s, dim3(1),
                    true, p, share, rows);
  };
  // (few parts leave room for more warps an SM)
  return plan.warps == 0 && plan.p_chunks + plan.s_chunks <= 4 ? join(k_prefix_join<T16, DH, 4>)
                                                               : join(k_prefix_join<T16, DH, 16>);
}

}  // namespace

bool paged_kv_ok(const dflash_paged_kv* kv) {
  if (kv == nullptr || kv->k == nullptr || kv->v == nullptr || kv->page_table == nullptr || kv->seq_len == nullptr)
    return false;
  if (kv->n_pages < 1 || kv->n_seqs < 1 || kv->max_pages < 1 || kv->max_pages > INT32_MAX / (2 * kPage) ||
      kv->n_kv_heads < 1 || kv->head_dim < 1)
    return false;
  if (kv->elem != DFLASH_ELEM_F32 && kv->elem != DFLASH_ELEM_BF16 && kv->elem != DFLASH_ELEM_F16) return false;
  return reinterpret_cast<uintptr_t>(kv->k) % 16 == 0 && reinterpret_cast<uintptr_t>(kv->v) % 16 == 0;
}

}  // namespace dflash

using namespace dflash;

extern "C" {

size_t dflash_prefix_attention_workspace(const dflash_paged_kv* kv, int n_q_heads, int B, int T, int NG,
                                         int max_prefix, int max_len) {
  PrefixPlan plan;
  if (check_prefix(kv, n_q_heads, B, T, NG, max_prefix, max_len) != DFLASH_OK ||
      !make_plan(*kv, n_q_heads, B, T, NG, max_prefix, max_len, &plan))
    return 0;
  return plan.bytes;
}

dflash_status dflash_prefix_attention(const dflash_paged_kv* kv, const void* q, long long ld_q, int n_q_heads,
                                      const int32_t* n_rows, const int32_t* seq, int B, int T,
                                      const int32_t* group_off, const int32_t* prefix_seq, int NG, int causal,
                                      float scale, int max_prefix, int max_len, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, int* status, dflash_stream stream) {
  const dflash_status st = check_prefix(kv, n_q_heads, B, T, NG, max_prefix, max_len);
  if (st != DFLASH_OK) return st;
  // (times log2(e) it is an fp32 number still)
  if (q == nullptr || out == nullptr || workspace == nullptr || !(scale >= 0.f) || scale > 2.35e38f)
    return DFLASH_ERR_INVALID_ARG;
  if (NG > 0 ? group_off == nullptr || prefix_seq == nullptr : group_off != nullptr || prefix_seq != nullptr)
    return DFLASH_ERR_INVALID_ARG;
  if (seq == nullptr && B > kv->n_seqs) return DFLASH_ERR_INVALID_ARG;
  const auto addr = [](const void* a) { return reinterpret_cast<uintptr_t>(a); };
  const long long qd = static_cast<long long>(n_q_heads) * kv->head_dim;
  const bool one = static_cast<long long>(B) * T == 1;
  if (addr(q) % 16 || addr(out) % 16 || addr(workspace) % 256 || (!one && (ld_q % 8 || ld_q < qd)) ||
      (q == out && !one && ld_q != qd))
    return DFLASH_ERR_INVALID_ARG;
  PrefixPlan plan;
  if (!make_plan(*kv, n_q_heads, B, T, NG, max_prefix, max_len, &plan)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < plan.bytes) return DFLASH_ERR_WORKSPACE;
  const long long ldq = one ? qd : ld_q;
  PrefixMaps maps{};
  const int chunks = kv->head_dim / 64, G = n_q_heads / kv->n_kv_heads;
  if ((plan.warps > 0 && (!page_map(*kv, kv->k, chunks, &maps.thin_k) || !page_map(*kv, kv->v, chunks, &maps.thin_v))) ||
      ((plan.p_wide || plan.s_wide) &&
       (!page_map(*kv, kv->k, 1, &maps.wide_k) || !page_map(*kv, kv->v, 1, &maps.wide_v) ||
        !query_map(*kv, q, n_q_heads, static_cast<long long>(B) * T, ldq, kWideTile / G, &maps.q) ||
        !query_map(*kv, q, n_q_heads, static_cast<long long>(B) * T, ldq, 1, &maps.q_one))))
    return DFLASH_ERR_CUDA;
  PrefixParams p{};
  p.q = q;
  p.ld_q = ldq;
  p.n_rows = n_rows;
  p.seq = seq;
  p.group_off = group_off;
  p.prefix_seq = prefix_seq;
  p.page_table = kv->page_table;
  p.seq_len = kv->seq_len;
  p.B = B;
  p.T = T;
  p.Hq = n_q_heads;
  p.Hkv = kv->n_kv_heads;
  p.G = n_q_heads / kv->n_kv_heads;
  p.NG = NG;
  p.n_pages = kv->n_pages;
  p.n_seqs = kv->n_seqs;
  p.max_pages = kv->max_pages;
  p.causal = causal;
  p.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(kv->head_dim))) * 1.4426950408889634f;
  p.out = out;
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.pack = plan.pack && n_rows != nullptr;
  p.merge = plan.merge;
  p.p_thin = NG > 0 && !plan.p_wide;
  p.work = reinterpret_cast<long long*>(ws + plan.off_work);
  p.part_lse = reinterpret_cast<float*>(ws + plan.off_lse);
  p.part_o = reinterpret_cast<float*>(ws + plan.off_o);
  p.whole_lse = reinterpret_cast<float*>(ws + plan.off_whole_lse);
  p.whole_o = reinterpret_cast<float*>(ws + plan.off_whole_o);
  p.slot_lse = reinterpret_cast<float*>(ws + plan.off_slot_lse);
  p.slot_o = reinterpret_cast<float*>(ws + plan.off_slot_o);
  p.warps = plan.warps;
  p.status = status != nullptr ? status : reinterpret_cast<int*>(ws);
  p.p_tiles = static_cast<int>(plan.p_tiles);
  p.p_chunks = plan.p_chunks;
  p.s_tiles = static_cast<int>(plan.s_tiles);
  p.s_chunks = plan.s_chunks;
  cudaError_t e;
  if (kv->elem == DFLASH_ELEM_BF16)
    e = kv->head_dim == 64 ? launch_prefix<__nv_bfloat16, 64>(p, plan, kv->elem, maps, stream)
                           : launch_prefix<__nv_bfloat16, 128>(p, plan, kv->elem, maps, stream);
  else
    e = kv->head_dim == 64 ? launch_prefix<__half, 64>(p, plan, kv->elem, maps, stream)
                           : launch_prefix<__half, 128>(p, plan, kv->elem, maps, stream);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
