// dflash_prefix_attention: attention of a batch over prefixes that groups of
// sequences share and over each sequence's own tokens, on a paged cache.
//
// A query row r sees the keys of its group's prefix and keys of its own
// sequence.  Softmax attention over a union of key sets splits exactly: with
// z = scale q.k, each set S gives l_S = log sum_S exp z and o_S = sum_S
// exp(z - l_S) v, and
//     out = sum_S exp(l_S - l) o_S,  l = log sum_S exp l_S.
// So a prefix is read once for all query rows of its group (as one tall
// matrix of rows), each sequence's own keys for its own rows, either of them
// in several chunks of pages, and a last kernel joins the partial results in
// a fixed order.
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

constexpr int kThinWarps = 4;
constexpr int kThinThreads = kThinWarps * 32;
constexpr int kThinRows = 16;   // query rows of a tile (one MMA's rows)
constexpr int kThinStages = 3;  // pages in flight per warp
constexpr int kMaxParts = 128;  // chunks of a prefix

template <int DH>
struct ThinLayout {
  static constexpr int HALF_PAGE = kPage * DH * 2;        // bytes of a page of K (or V) of one head
  static constexpr int STAGE = 2 * HALF_PAGE;
  static constexpr int WARP = kThinStages * STAGE;
  static constexpr int LDO = DH + 8;                      // floats per row of a warp's partial output
  static constexpr int OFF_ML = kThinWarps * WARP;        // [warps][16][2] maxima and sums
  static constexpr int OFF_TOP = OFF_ML + kThinWarps * kThinRows * 8;  // [16] what the weights are relative to
  static constexpr int OFF_W = kThinRows * LDO * 4;       // weights of four rows' parts, in each warp's ring
  static_assert(OFF_W + 4 * kMaxParts * 4 <= WARP, "the weights fit beside a warp's partial output");
  static constexpr int OFF_BAR = OFF_TOP + kThinRows * 4;
  static constexpr int BYTES = OFF_BAR + kThinWarps * kThinStages * 8;
  static constexpr int SMEM = 1024 + BYTES;
  static_assert(kThinRows * LDO * 4 <= WARP, "a warp's partial output fits its ring");
};

// One CTA: a tile of 16 query rows of one kv head over a chunk of pages.
// Every warp takes every fourth page with a ring of its own, keeps its own
// running maximum, sum and output, and the CTA joins its warps at the end.
template <typename T16, int DH>
__global__ void __launch_bounds__(kThinThreads) k_prefix_thin(const __grid_constant__ CUtensorMap tmK,
                                                              const __grid_constant__ CUtensorMap tmV,
                                                              const __grid_constant__ PrefixParams p, int n_prefix) {
  using L = ThinLayout<DH>;
  using M = Mma16<T16>;
  constexpr int KS = DH / 16, NT = DH / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, t4 = lane & 3;

  Item it;
  // (the kernel before it, where there is one, is waited for on every way
  // out: the joining kernel behind starts once all of this one has left)
  if (!find_item(p, blockIdx.x, n_prefix, kThinRows, it)) return pdl_wait();
  const int pg0 = it.pg0, pg1 = it.pg1, tokens = it.tokens, kvh = it.kvh;
  const Row row[2] = {find_row(p, it, it.row0 + gr), find_row(p, it, it.row0 + gr + 8)};

  const int parts = it.last && p.merge ? prefix_parts(p, it.b0) : 0;  // of the prefix, to be added at the end

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR) + warp * kThinStages;
  uint8_t* ring = smem + warp * L::WARP;
  const int mine = pg1 > pg0 + warp ? (pg1 - pg0 - warp + kThinWarps - 1) / kThinWarps : 0;
  if (lane == 0) {
    for (int s = 0; s < kThinStages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  // page ids of this warp's next 32 pages, one per lane
  int ids = 0;
  auto fetch_ids = [&](int i0) {
    const int i = i0 + lane;
    int id = 0;
    if (i < mine) {
      id = p.page_table[static_cast<long long>(it.table_row) * p.max_pages + pg0 + warp + i * kThinWarps];
      if (id < 0 || id >= p.n_pages) {
        flag_status(p.status, ST_BAD_PAGE);
        id = p.n_pages;  // outside the tensor map: reads as zeros
      }
    }
    ids = id;
  };
  auto issue = [&](int i) {
    if ((i & 31) == 0) fetch_ids(i);
    const int id = __shfl_sync(0xffffffffu, ids, i & 31);
    if (lane == 0) {
      const int s = i % kThinStages;
      const uint32_t kd = smem_u32(ring + s * L::STAGE);
      mbar_arrive_expect_tx(&bars[s], L::STAGE);
#pragma unroll
      for (int c = 0; c < DH / 64; ++c) {
        tma_page(kd + c * 2048, &tmK, &bars[s], c * 64, kvh, id);
        tma_page(kd + L::HALF_PAGE + c * 2048, &tmV, &bars[s], c * 64, kvh, id);
      }
    }
  };
  for (int i = 0; i < min(mine, kThinStages); ++i) issue(i);

  // the query rows as A fragments
  uint32_t qf[KS][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const T16* src = static_cast<const T16*>(p.q) + row[i].token * p.ld_q + (row[i].at - row[i].token * p.Hq) * DH + 2 * t4;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qf[ks][i] = row[i].live ? *reinterpret_cast<const uint32_t*>(src + ks * 16) : 0u;
      qf[ks][2 + i] = row[i].live ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8) : 0u;
    }
  }

  float o[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  // ldmatrix lane addresses within a [16 keys][128 bytes] swizzled box
  const int lr = lane & 7, lm = lane >> 3;
  const int k_key = (lm >> 1) * 8 + lr, k_unit = lm & 1;   // K: matrices (keys, d), (keys, d + 8), (keys + 8, ..)
  const int v_key = (lm & 1) * 8 + lr, v_unit = lm >> 1;   // V, transposed: (keys, d), (keys + 8, d), (keys, d + 8), ..

  bool ok = true;
  for (int i = 0; i < mine; ++i) {
    const int s = i % kThinStages;
    ok = ok && mbar_wait(&bars[s], (i / kThinStages) & 1, p.status);
    if (!__all_sync(0xffffffffu, ok)) break;
    const int key0 = (pg0 + warp + i * kThinWarps) * kPage;
    const uint32_t kd = smem_u32(ring + s * L::STAGE), vd = kd + L::HALF_PAGE;
    // values past the last token would meet probabilities of zero: they must be finite
    if (key0 + kPage > tokens) {
      const int first = tokens - key0;
      for (int e = lane; e < (kPage - first) * (DH / 64) * 8; e += 32) {
        const int c = e / ((kPage - first) * 8), f = e % ((kPage - first) * 8);
        *reinterpret_cast<uint4*>(ring + s * L::STAGE + L::HALF_PAGE + c * 2048 + first * 128 + f * 16) =
            make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
    float sc[2][4] = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t kb[4];
      const int unit = (ks & 3) * 2 + k_unit;
      ldsm_x4(kd + (ks >> 2) * 2048 + k_key * 128 + ((unit ^ (k_key & 7)) << 4), kb);
      M::mma(sc[0], qf[ks], kb[0], kb[1]);
      M::mma(sc[1], qf[ks], kb[2], kb[3]);
    }
    uint32_t pa[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = key0 + (e >> 1) * 8 + 2 * t4 + (e & 1);
        x[e] = key < row[h].seen ? sc[e >> 1][2 * h + (e & 1)] * p.scale_log2 : -INFINITY;
      }
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[h], mx), ms = mn == -INFINITY ? 0.f : mn;
      const float al = exp2f(m[h] - ms);
      m[h] = mn;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = exp2f(x[e] - ms);
        sum += x[e];
      }
      l[h] = l[h] * al + sum;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j][2 * h] *= al;
        o[j][2 * h + 1] *= al;
      }
      pa[h] = M::pack(x[0], x[1]);
      pa[2 + h] = M::pack(x[2], x[3]);
    }
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      uint32_t vb[4];
      const int unit = (j & 7) + v_unit;
      ldsm_x4_t(vd + (j >> 3) * 2048 + v_key * 128 + ((unit ^ (v_key & 7)) << 4), vb);
      M::mma(o[j], pa, vb[0], vb[1]);
      M::mma(o[j + 1], pa, vb[2], vb[3]);
    }
    __syncwarp();
    if (i + kThinStages < mine) issue(i + kThinStages);
  }
  if (!ok) {  // a wait gave up: what is still in flight gets its own bounded waits before the CTA leaves
    for (int s = 0; s < min(mine, kThinStages); ++s) mbar_wait(&bars[s], 0, p.status);
  }

  // join the warps: each leaves (m, l) and its unnormalised output in its ring
  float* ml = reinterpret_cast<float*>(smem + L::OFF_ML);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    const int r = gr + 8 * h;
    if (t4 == 0) {
      ml[(warp * kThinRows + r) * 2] = m[h];
      ml[(warp * kThinRows + r) * 2 + 1] = l[h];
    }
    float* dst = reinterpret_cast<float*>(ring) + r * L::LDO + 2 * t4;
#pragma unroll
    for (int j = 0; j < NT; ++j) *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
  }
  __syncthreads();
  const long long R = static_cast<long long>(p.B) * p.T * p.Hq;
  const int out_chunk = it.shared ? it.chunk : p.p_chunks + it.chunk;
  // weights of the prefix's partial results (each is normalised by its own
  // sum), eight threads a row, in the unused part of the rings
  auto weights = [&](int r) { return reinterpret_cast<float*>(smem + r / 4 * L::WARP + L::OFF_W) + r % 4 * kMaxParts; };
  if (parts > 0) {
    pdl_wait();
    const int r = threadIdx.x / 8;
    const Row w = find_row(p, it, it.row0 + r);
    float mx = -INFINITY;
#pragma unroll
    for (int q = 0; q < kThinWarps; ++q) mx = fmaxf(mx, ml[(q * kThinRows + r) * 2]);
    float top = mx;
    if (w.live)
      for (int c = threadIdx.x % 8; c < parts; c += 8) {
        const float v = p.part_lse[c * R + w.at];
        weights(r)[c] = v;
        top = fmaxf(top, v);
      }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    if (w.live)
      for (int c = threadIdx.x % 8; c < parts; c += 8) weights(r)[c] = exp2f(weights(r)[c] - base);
    if (threadIdx.x % 8 == 0) reinterpret_cast<float*>(smem + L::OFF_TOP)[r] = base;
    __syncthreads();
  }
  for (int e = threadIdx.x; e < kThinRows * (DH / 4); e += kThinThreads) {
    const int r = e / (DH / 4), d = (e % (DH / 4)) * 4;
    const Row w = find_row(p, it, it.row0 + r);
    if (!w.live) continue;
    float ms;
    if (parts > 0) {
      ms = reinterpret_cast<const float*>(smem + L::OFF_TOP)[r];
    } else {
      float mx = -INFINITY;
#pragma unroll
      for (int q = 0; q < kThinWarps; ++q) mx = fmaxf(mx, ml[(q * kThinRows + r) * 2]);
      ms = mx == -INFINITY ? 0.f : mx;
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kThinWarps; ++q) {
      const float f = exp2f(ml[(q * kThinRows + r) * 2] - ms);
      const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + q * L::WARP) + r * L::LDO + d);
      sum += f * ml[(q * kThinRows + r) * 2 + 1];
      a.x += f * v.x;
      a.y += f * v.y;
      a.z += f * v.z;
      a.w += f * v.w;
    }
    const float* src = p.part_o + w.at * DH + d;
#pragma unroll 8
    for (int c = 0; c < parts; ++c) {
      const float f = weights(r)[c];
      const float4 v = *reinterpret_cast<const float4*>(src + c * R * DH);
      sum += f;
      a.x += f * v.x;
      a.y += f * v.y;
      a.z += f * v.z;
      a.w += f * v.w;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    a = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    const float lse2 = sum > 0.f ? ms + log2f(sum) : -INFINITY;
    if (it.last) {
      *reinterpret_cast<uint2*>(static_cast<T16*>(p.out) + w.at * DH + d) = make_uint2(M::pack(a.x, a.y), M::pack(a.z, a.w));
      if (d == 0 && p.lse != nullptr) p.lse[w.at] = lse2 * 0.69314718055994531f;
    } else {
      *reinterpret_cast<float4*>(p.part_o + (out_chunk * R + w.at) * DH + d) = a;
      if (d == 0) p.part_lse[out_chunk * R + w.at] = lse2;
    }
  }
  pdl_wait();
}

constexpr int kJoinWarps = 8;

// out of the partial results, chunks in order: `share` warps (1 or 8) a query
// row, each adding every share-th chunk.
template <typename T16, int DH>
__global__ void __launch_bounds__(kJoinWarps * 32) k_prefix_join(const __grid_constant__ PrefixParams p, int share) {
  using M = Mma16<T16>;
  constexpr int E = DH / 32;  // elements a lane
  __shared__ float s_a[kJoinWarps][DH], s_sum[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % share;
  const long long R = static_cast<long long>(p.B) * p.T * p.Hq;
  const long long row = static_cast<long long>(blockIdx.x) * (kJoinWarps / share) + warp / share;
  const long long tok = row / p.Hq;
  const int b = static_cast<int>(tok / p.T), t = static_cast<int>(tok - static_cast<long long>(b) * p.T);
  const bool live = row < R && t < entry_rows(p, b);
  int n_pre = 0, n_all = 0;
  if (live) {
    n_pre = prefix_parts(p, b);
    const int pages = (seq_tokens(p, p.seq != nullptr ? p.seq[b] : b) + kPage - 1) / kPage;
    const int per = chunk_pages(pages, p.s_chunks);
    n_all = n_pre + (pages + per - 1) / per;
  }
  pdl_wait();
  float mx = -INFINITY, sum = 0.f, a[E] = {};
  auto place = [&](int c) { return static_cast<long long>(c < n_pre ? c : p.p_chunks + c - n_pre) * R + row; };
  for (int c = lane; c < n_all; c += 32) mx = fmaxf(mx, p.part_lse[place(c)]);
  mx = warp_max(mx);
  const float ms = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
  for (int c = sub; c < n_all; c += share) {
    const long long at = place(c);
    const float f = exp2f(p.part_lse[at] - ms);
    const float* src = p.part_o + at * DH + lane * E;
    float v[E];
    if constexpr (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] += f * v[e];
    sum += f;
  }
  if (share > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_a[warp][lane * E + e] = a[e];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
    sum = 0.f;
    for (int w = 0; w < kJoinWarps; ++w) {
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] += s_a[w][lane * E + e];
      sum += s_sum[w];
    }
  }
  if (!live) return;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  T16* dst = static_cast<T16*>(p.out) + row * DH + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = M::pack(a[e] * inv, a[e + 1] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[row] = sum > 0.f ? (ms + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

// ------------------------------------------------------------------ host side

// From this many query rows (of an entry; of a group on average) on, the
// wide kernel takes them.
constexpr int kWideFrom = 48;

struct PrefixPlan {
  bool p_wide, s_wide;         // whether the wide kernel takes the part (else the thin one)
  bool merge;                  // own parts add the prefix's partial results
  long long p_tiles, s_tiles;  // row tiles: of all groups (a bound), of an entry
  long long rows;
  int p_chunks, s_chunks;
  size_t off_lse, bytes;
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

// Chunks per item: the count whose waves of CTAs (`slots` at once) take the
// least time, a CTA costing its steps (of `step` pages) and `start` more to
// start and to write its rows, and a part in several chunks `join` more.
int plan_chunks(long long items, int tokens, long long slots, int step, int start, int join, int most) {
  const int steps = std::max(1, (tokens + step * kPage - 1) / (step * kPage));
  int best = 1;
  long long cost = INT64_MAX;
  for (int c = 1; c <= std::min(steps, most); ++c) {
    const long long t = (items * c + slots - 1) / slots * ((steps + c - 1) / c + start) + (c > 1 ? join : 0);
    if (t < cost) {
      cost = t;
      best = c;
    }
  }
  return best;
}

bool make_plan(const dflash_paged_kv& kv, int Hq, int B, int T, int NG, int max_prefix, int max_len, PrefixPlan* out) {
  const int G = Hq / kv.n_kv_heads;
  const long long tg = static_cast<long long>(T) * G;
  const int cap = kv.max_pages * kPage;
  const int mp = max_prefix > 0 ? std::min(max_prefix, cap) : cap, ml = max_len > 0 ? std::min(max_len, cap) : cap;
  PrefixPlan r{};
  r.rows = static_cast<long long>(B) * T * Hq;
  const bool fits = G <= kWideTile;  // (a token's heads stay in one row tile)
  r.p_wide = fits && NG > 0 && B * tg >= static_cast<long long>(kWideFrom) * NG;
  r.s_wide = fits && tg >= kWideFrom;
  const int p_rows = r.p_wide ? wide_rows(G) : kThinRows;
  const int s_rows = r.s_wide ? wide_rows(G) : kThinRows;
  r.p_tiles = NG > 0 ? (B * tg + static_cast<long long>(NG) * (p_rows - 1)) / p_rows : 0;
  r.s_tiles = (tg + s_rows - 1) / s_rows;
  const int sms = plan_sms(), thin_slots = sms * (kv.head_dim == 64 ? 4 : 2);
  const long long p_items = r.p_tiles * kv.n_kv_heads, s_items = B * r.s_tiles * kv.n_kv_heads;
  const auto chunks = [&](bool wide, long long items, int tokens, int join) {
    return wide ? plan_chunks(items, tokens, 2 * sms, kMinChunkPages, 3, join, kMaxParts / 2)
                : plan_chunks(items, tokens, thin_slots, kMinChunkPages, 2, join, kMaxParts);
  };
  r.p_chunks = NG == 0 ? 0 : chunks(r.p_wide, p_items, mp, 0);
  r.s_chunks = chunks(r.s_wide, s_items, ml, 3);
  // (a wide own part adds a row's copies one after the other)
  r.merge = NG > 0 && r.s_chunks == 1 && !(r.s_wide && r.p_chunks > 4);
  if (p_items * r.p_chunks + s_items * r.s_chunks > INT32_MAX) return false;
  const int parts = r.p_chunks + (r.merge || (NG == 0 && r.s_chunks == 1) ? 0 : r.s_chunks);
  r.off_lse = 256;  // (the first 256 bytes: a status word for callers without one)
  r.bytes = r.off_lse + (sizeof(float) * r.rows * parts + 255) / 256 * 256 + sizeof(float) * r.rows * parts * kv.head_dim;
  *out = r;
  return true;
}

dflash_status check_prefix(const dflash_paged_kv* kv, int Hq, int B, int T, int NG, int max_prefix, int max_len) {
  if (!paged_kv_ok(kv) || B < 1 || T < 1 || NG < 0 || max_prefix < 0 || max_len < 0 || Hq < 1)
    return DFLASH_ERR_INVALID_ARG;
  if (Hq % kv->n_kv_heads) return DFLASH_ERR_INVALID_ARG;
  if (kv->elem == DFLASH_ELEM_F32 || (kv->head_dim != 64 && kv->head_dim != 128)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  // row counts stay well inside 32 bits
  if (static_cast<long long>(B) * T * Hq > INT32_MAX / 2 || NG > (1 << 20))
    return DFLASH_ERR_UNSUPPORTED_SHAPE;
  return DFLASH_OK;
}

// Pages of one layer as a 4-D map with boxes of 16 tokens x 64 elements (128-byte swizzled rows).
bool page_map(const dflash_paged_kv& kv, void* base, CUtensorMap* out) {
  const auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dh = kv.head_dim;
  const cuuint64_t gdim[4] = {dh, kPage, static_cast<cuuint64_t>(kv.n_kv_heads), static_cast<cuuint64_t>(kv.n_pages)};
  const cuuint64_t gstride[3] = {dh * 2, dh * 2 * kPage, dh * 2 * kPage * kv.n_kv_heads};
  const cuuint32_t box[4] = {64, kPage, 1, 1}, es[4] = {1, 1, 1, 1};
  return fn(out, kv.elem == DFLASH_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            base, gdim, gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as a 3-D map (elements, heads, tokens) with boxes of a row tile's
// whole tokens x the group's heads x 64 elements.
bool query_map(const dflash_paged_kv& kv, const void* q, int Hq, long long tokens, long long ld, CUtensorMap* out) {
  const auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const int G = Hq / kv.n_kv_heads;
  const cuuint64_t gdim[3] = {static_cast<cuuint64_t>(kv.head_dim), static_cast<cuuint64_t>(Hq),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t gstride[2] = {static_cast<cuuint64_t>(kv.head_dim) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(kWideTile / G)}, es[3] = {1, 1, 1};
  return fn(out, kv.elem == DFLASH_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(q), gdim, gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T16, int DH>
cudaError_t launch_thin(const PrefixParams& p, long long n_prefix, long long n_own, bool behind, const CUtensorMap& tk,
                        const CUtensorMap& tv, cudaStream_t s) {
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(ThinLayout<DH>::SMEM, [](int v) {
    return cudaFuncSetAttribute(k_prefix_thin<T16, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  return launch_k(k_prefix_thin<T16, DH>, dim3(static_cast<unsigned>(n_prefix + n_own)), dim3(kThinThreads),
                  ThinLayout<DH>::SMEM, s, dim3(1), behind, tk, tv, p, static_cast<int>(n_prefix));
}

template <typename T16, int DH>
cudaError_t launch_prefix(const PrefixParams& p, const PrefixPlan& plan, int elem, const CUtensorMap& tq,
                          const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  const long long n_prefix = plan.p_tiles * plan.p_chunks * p.Hkv, n_own = p.B * plan.s_tiles * plan.s_chunks * p.Hkv;
  cudaError_t e = cudaSuccess;
  if (n_prefix > 0)
    e = plan.p_wide ? launch_prefix_wide(p, elem, DH, n_prefix, 0, false, tq, tk, tv, s)
                    : launch_thin<T16, DH>(p, n_prefix, 0, false, tk, tv, s);
  if (e == cudaSuccess)
    e = plan.s_wide ? launch_prefix_wide(p, elem, DH, 0, n_own, n_prefix > 0, tq, tk, tv, s)
                    : launch_thin<T16, DH>(p, 0, n_own, n_prefix > 0, tk, tv, s);
  if (e != cudaSuccess || p.merge || (p.NG == 0 && p.s_chunks == 1)) return e;
  // few rows of many parts: a row's parts over all the warps of a CTA
  const int share = p.p_chunks + p.s_chunks >= 16 ? kJoinWarps : 1, per = kJoinWarps / share;
  return launch_k(k_prefix_join<T16, DH>, dim3(static_cast<unsigned>((plan.rows + per - 1) / per)),
                  dim3(kJoinWarps * 32), 0, s, dim3(1), true, p, share);
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
  if (q == nullptr || out == nullptr || workspace == nullptr || !(scale >= 0.f) || scale > 3e38f)
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
  CUtensorMap tq{}, tk, tv;
  if (!page_map(*kv, kv->k, &tk) || !page_map(*kv, kv->v, &tv) ||
      ((plan.p_wide || plan.s_wide) && !query_map(*kv, q, n_q_heads, static_cast<long long>(B) * T, ldq, &tq)))
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
  p.merge = plan.merge;
  const int parts = plan.p_chunks + (plan.merge ? 0 : plan.s_chunks);
  p.part_lse = reinterpret_cast<float*>(ws + plan.off_lse);
  p.part_o = reinterpret_cast<float*>(ws + plan.off_lse + (sizeof(float) * plan.rows * parts + 255) / 256 * 256);
  p.status = status != nullptr ? status : reinterpret_cast<int*>(ws);
  p.p_tiles = static_cast<int>(plan.p_tiles);
  p.p_chunks = plan.p_chunks;
  p.s_tiles = static_cast<int>(plan.s_tiles);
  p.s_chunks = plan.s_chunks;
  cudaError_t e;
  if (kv->elem == DFLASH_ELEM_BF16)
    e = kv->head_dim == 64 ? launch_prefix<__nv_bfloat16, 64>(p, plan, kv->elem, tq, tk, tv, stream)
                           : launch_prefix<__nv_bfloat16, 128>(p, plan, kv->elem, tq, tk, tv, stream);
  else
    e = kv->head_dim == 64 ? launch_prefix<__half, 64>(p, plan, kv->elem, tq, tk, tv, stream)
                           : launch_prefix<__half, 128>(p, plan, kv->elem, tq, tk, tv, stream);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
