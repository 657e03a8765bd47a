// Shared by the kernels of dflash_prefix_attention (prefix_attn.cu,
// prefix_wide.cu): parameters, the search for a CTA's rows and keys, and
// the 16-bit element types.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "decode_common.cuh"
#include "kernels.cuh"

namespace dflash {

struct PrefixParams {
  const void* q;
  long long ld_q;
  const int32_t *n_rows, *seq, *group_off, *prefix_seq, *page_table, *seq_len;
  int B, T, Hq, Hkv, G, NG, n_pages, n_seqs, max_pages, causal;
  float scale_log2;  // scale * log2(e): scores are taken in powers of two
  void* out;
  float* lse;
  float* part_o;    // [chunk][B*T*Hq][DH], normalised by its own sum
  float* part_lse;  // [chunk][B*T*Hq], in powers of two
  int* status;
  int p_tiles, p_chunks;  // prefix parts: row tiles over all groups (a bound), chunks of pages
  int s_tiles, s_chunks;  // own parts: row tiles of an entry, chunks of pages
  bool merge;             // own parts (of one chunk) add the prefix's partial results and write the result
  bool pack;              // prefix row tiles of the wide kernel hold live rows only
  bool p_thin;            // the thin kernel takes the prefix parts (no p_chunks then)
  // what the thin kernel leaves for the joining one
  long long* work;                // the line's first pages of [NG] + [B] elements, and its length
  float *whole_lse, *whole_o;     // [2][B*T*Hq], [..][DH]: prefix and own parts that one warp took whole
  float *slot_lse, *slot_o;       // [2 * warps][rows of a tile], [..][DH]: a warp's first and last part, where others share them
  int warps;                      // its warps
};

// Chunks are whole multiples of this many pages (a key tile of the wide
// kernel), so that a short context is not spread over chunks of a page each.
constexpr int kMinChunkPages = 8;

__host__ __device__ __forceinline__ int chunk_pages(int pages, int chunks) {
  const int per = (pages + chunks - 1) / chunks;
  return per < kMinChunkPages ? kMinChunkPages : (per + kMinChunkPages - 1) / kMinChunkPages * kMinChunkPages;
}

__device__ __forceinline__ void flag_status(int* status, int bit) { atomicOr(status, bit); }

// Rows of entry b (0 where n_rows is out of range).
__device__ __forceinline__ int entry_rows(const PrefixParams& p, int b) {
  const int n = p.n_rows != nullptr ? p.n_rows[b] : p.T;
  return n < 0 || n > p.T ? 0 : n;
}

// Tokens of the cache's sequence s, at most what its page table can name (0 for a bad index).
__device__ __forceinline__ int seq_tokens(const PrefixParams& p, int s) {
  if (s < 0 || s >= p.n_seqs) return 0;
  return max(0, min(p.seq_len[s], p.max_pages * kPage));
}

struct Group {
  int lo, hi;   // its entries
  int row;      // the prefix's sequence (-1: none)
  int tokens;   // and length
  int tile;     // row tile within the group
  int index;
};

__device__ __forceinline__ Group load_group(const PrefixParams& p, int g) {
  Group r;
  r.lo = p.group_off[g];
  r.hi = p.group_off[g + 1];
  r.row = p.prefix_seq[g];
  r.tokens = seq_tokens(p, r.row);
  r.tile = 0;
  r.index = g;
  return r;
}

// Whether group bounds run from 0 to B without falling (the whole warp asks).
__device__ __forceinline__ bool bounds_ok(const PrefixParams& p) {
  const int lane = threadIdx.x & 31;
  bool ok = p.group_off[0] == 0 && p.group_off[p.NG] == p.B;
  for (int g = lane; g < p.NG; g += 32) ok = ok && p.group_off[g] <= p.group_off[g + 1];
  return __all_sync(0xffffffffu, ok);
}

// The group that row tile `tile` (of `rows` rows) falls in, counting every
// group's tiles in order (the whole warp asks; false past the last one).
__device__ __forceinline__ bool find_tile(const PrefixParams& p, int tile, int rows, Group& out) {
  const int lane = threadIdx.x & 31;
  for (int g0 = 0; g0 < p.NG; g0 += 32) {
    const int g = g0 + lane;
    int n = 0;
    if (g < p.NG) {
      const long long r = static_cast<long long>(p.group_off[g + 1] - p.group_off[g]) * p.T * p.G;
      n = static_cast<int>((r + rows - 1) / rows);
    }
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, tile < sum);
    if (past != 0) {
      const int at = __ffs(past) - 1;
      const int before = __shfl_sync(0xffffffffu, sum - n, at);
      out = load_group(p, g0 + at);
      out.tile = tile - before;
      return true;
    }
    tile -= __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

// The group of entry b (the whole warp asks; the bounds are ok).
__device__ __forceinline__ Group find_entry(const PrefixParams& p, int b) {
  const int lane = threadIdx.x & 31;
  for (int g0 = 0; g0 < p.NG; g0 += 32) {
    const int g = g0 + lane;
    const unsigned in = __ballot_sync(0xffffffffu, g < p.NG && b >= p.group_off[g] && b < p.group_off[g + 1]);
    if (in != 0) return load_group(p, g0 + __ffs(in) - 1);
  }
  return Group{0, 0, -1, 0, 0, 0};
}

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPage - 1) / kPage; }

// The group of entry b where the bounds are sound (the whole warp asks).
__device__ __forceinline__ Group group_of(const PrefixParams& p, int b) {
  return p.NG > 0 && bounds_ok(p) ? find_entry(p, b) : Group{0, 0, -1, 0, 0, 0};
}

// Chunks that hold `pages` pages (chunks > 0).
__device__ __forceinline__ int chunks_of(int pages, int chunks) {
  const int per = chunk_pages(pages, chunks);
  return (pages + per - 1) / per;
}

__device__ __forceinline__ void check_prefix(const PrefixParams& p, int row) {
  if (row == -1) return;
  if (row < -1 || row >= p.n_seqs) flag_status(p.status, ST_BAD_BLOCK);
  else if (p.seq_len[row] > p.max_pages * kPage) flag_status(p.status, ST_SEQ_TOO_LONG);
}

// Every group's prefix, of those without rows too (the whole CTA asks; a call, so
// that what surrounds it keeps its registers).
inline __device__ __noinline__ void check_groups(const PrefixParams& p) {
  for (int g = threadIdx.x; g < p.NG; g += blockDim.x) check_prefix(p, p.prefix_seq[g]);
}

__device__ __forceinline__ void check_entry(const PrefixParams& p, int b, int row) {
  const int n = p.n_rows != nullptr ? p.n_rows[b] : p.T;
  if (n < 0 || n > p.T) flag_status(p.status, ST_BAD_ROWS);
  if (row < 0 || row >= p.n_seqs) flag_status(p.status, ST_BAD_BLOCK);
  else if (p.seq_len[row] > p.max_pages * kPage) flag_status(p.status, ST_SEQ_TOO_LONG);
}

// What one CTA works on: a tile of query rows of one kv head over a chunk of pages.
struct Item {
  bool shared;    // a group's prefix (else an entry's own sequence)
  int b0;         // first entry of the rows
  int row0, rows; // the tile's first row, and the rows there are (entry, token, head of the group; row-major)
  int kvh, chunk;
  int tokens;     // keys of the sequence
  int table_row;
  int pg0, pg1;   // its pages
  bool last;      // an own part that writes the result, even when it holds no key
};

// Item `index` of the prefix parts (n_prefix of them come first) and own
// parts, tiles of `rows` query rows.  False: nothing to do.  The whole warp
// asks.  Device-side errors are reported by one thread of one CTA.
__device__ __forceinline__ bool find_item(const PrefixParams& p, int index, int n_prefix, int tile_rows, Item& it) {
  it.shared = index < n_prefix;
  int item = it.shared ? index : index - n_prefix;
  const int chunks = it.shared ? p.p_chunks : p.s_chunks;
  it.chunk = item % chunks;
  item /= chunks;
  it.kvh = item % p.Hkv;
  const int tile = item / p.Hkv;
  const bool first = it.chunk == 0 && threadIdx.x == 0;  // the thread that reports
  if (it.shared) {
    Group g;
    if (!bounds_ok(p)) return false;
    if (index == 0) check_groups(p);
    if (!find_tile(p, tile, tile_rows, g)) return false;
    it.b0 = g.lo;
    it.row0 = g.tile * tile_rows;
    it.rows = (g.hi - g.lo) * p.T * p.G;
    it.tokens = g.tokens;
    it.table_row = g.row;
  } else {
    const int b = tile / p.s_tiles;
    it.b0 = b;
    it.row0 = (tile - b * p.s_tiles) * tile_rows;
    it.table_row = p.seq != nullptr ? p.seq[b] : b;
    it.tokens = seq_tokens(p, it.table_row);
    it.rows = entry_rows(p, b) * p.G;
    if (p.NG > 0 && b == 0 && it.row0 == 0 && it.kvh == 0 && it.chunk == 0 && threadIdx.x < 32 && !bounds_ok(p) &&
        threadIdx.x == 0)
      flag_status(p.status, ST_BAD_BLOCK);
    if (first && it.row0 == 0) check_entry(p, b, it.table_row);
  }
  if (it.row0 >= it.rows) return false;
  const int pages = pages_of(it.tokens), per = chunk_pages(pages, chunks);
  it.pg0 = it.chunk * per;
  it.pg1 = min(pages, it.pg0 + per);
  it.last = !it.shared && (p.merge || (p.NG == 0 && p.s_chunks == 1));
  return it.pg0 < it.pg1 || it.last;
}

// A query row of an item: whether there is one, its place in q and out
// ((entry, token, head), row-major), and how many of the item's keys it sees.
struct Row {
  bool live;
  long long token, at;
  int seen;
};

__device__ __forceinline__ Row find_row(const PrefixParams& p, const Item& it, int r) {
  Row w;
  w.live = r < it.rows;
  const int tg = p.T * p.G;
  const int b = w.live ? it.b0 + r / tg : it.b0;
  const int t = w.live ? r % tg / p.G : 0, gi = w.live ? r % p.G : 0;
  const int n = entry_rows(p, b);
  w.live = w.live && t < n;
  w.token = static_cast<long long>(b) * p.T + t;
  w.at = w.token * p.Hq + it.kvh * p.G + gi;
  w.seen = it.shared || !p.causal ? it.tokens : min(it.tokens, it.tokens - n + t + 1);
  return w;
}

// Probabilities enter the second product in the cache's type, relative to
// 2^(m - kLift), so that the largest is about 2^kLift.  Rounding them costs half
// a step of the type each, as the one rounding of the output does (errors against
// 64 bits 1.0 to 1.4 times those of fp32 probabilities); two products with a
// high and a low half would cost as much again as the first.  fp16 steps no
// finer than 2^-24: the lift moves that edge from 2^-24 of the largest weight to
// 2^-24 - kLift, where even a million faint keys lose less than the output's half
// step.  bf16 has the exponents to go without.
template <typename T>
struct Mma16;
template <>
struct Mma16<__nv_bfloat16> {
  static constexpr bool kLifted = false;
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Mma16<__half> {
  static constexpr bool kLifted = true;
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// One head's 16 tokens of a page, from 64-element chunk c on (the map says how
// many chunks: [chunk][16 tokens][128 bytes], swizzled).
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c, int h, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c), "r"(h), "r"(page), "r"(smem_u32(bar))
      : "memory");
}
// prefix_wide.cu: items of a tile of wide_rows(G) query rows (whole tokens),
// n_prefix prefix items or n_own own ones.
constexpr int kWideTile = 128;  // rows of an MMA
__host__ __device__ inline int wide_rows(int G) { return kWideTile / G * G; }
cudaError_t launch_prefix_wide(const PrefixParams& p, int elem, int head_dim, long long n_prefix, long long n_own,
                               bool behind, const CUtensorMap& tq, const CUtensorMap& tq1, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s);

}  // namespace dflash
