// dflash_pages_*: the pages of a cache shared by reference counts, for all of
// its layers at once: forked, cut back, given room, copied and compacted.
//
// The counts (refs[page]: how many sequences hold it) are the whole state
// beside the page table and the lengths: a page is free where its count is 0,
// and new ones are the lowest free ids, so that nothing depends on the order in
// which threads come.  A call reads the state as it was before it, and where
// it cannot be done as a whole nothing changes.
//
// Two kernels: one cluster of CTAs plans (checks, counts, tables, the list of
// pages to copy), and a grid copies them, started early and waiting for the
// plan.  Planning is bound by the latency of its few passes over the tables
// and counts and the barriers between them (a fork of one sequence of 2043 tokens 8.7 us
// with its copy, of 96 from 6 of up to 4500 25.7, a cut 3 to 4.4, room 4 to 7; blocks of 1024 threads, whose
// barriers take longer, 9.8 and 27, of 256 11.8 and 31; 16 CTAs 8.8 and 23.6, but a small compaction 11.4 against 10.8), copying by memory
// (2900 of 7001 pages of 5 layers, 1.05 GB read and written, 166 us with the plan: 6.3 TB/s).
#include <algorithm>
#include <initializer_list>

#include "decode_common.cuh"
#include "internal.h"

namespace dflash {

namespace {

constexpr int kMaxLayers = 128;
constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCluster = 8;
constexpr int kCopyThreads = 256, kCopyBytes = 64;  // a thread, at a time
constexpr int kMaxSeqs = 1 << 19;                  // two bitmaps of them in shared memory
constexpr int kMaxPages = 1 << 20;                 // (sums of a block's counts stay far inside 32 bits)

struct PagesParams {
  int32_t *table, *len, *refs;
  int n_pages, n_seqs, max_pages;
  const int32_t *a, *b;     // fork: src, dst; else: seq (or null), and new lengths (or null) or rows
  int B;
  int32_t* ws;              // [0]: pages to copy; then the lists
  int *status;
  // compact
  int32_t *table_out, *refs_out, *page_map, *n_used;
};

// The workspace: a header, three lists of n_pages ids, two numbers a sequence.
constexpr int kWsHead = 64;
__host__ __device__ __forceinline__ long long ws_ints(int n_pages, int n_seqs) {
  return kWsHead + 3ll * n_pages + 2ll * n_seqs;
}

// (of any length from 0 on: a caller may cut to one next to 2^31)
__device__ __forceinline__ int pages_of(int len) { return len / kPage + (len % kPage != 0); }

constexpr int kStaged = 1024;  // entries whose sequences and lengths are kept in shared memory
struct PlanShared {
  unsigned long long warp_sum[kPlanWarps];
  int bad;
  unsigned long long word[4];  // what the cluster's CTAs tell one another, a word a time
  int x[2][kStaged], len[2][kStaged];
};

// Inclusive sum over the block's threads; *all gets the total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, PlanShared& s, T* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s.warp_sum[warp] = static_cast<unsigned long long>(v);
  __syncthreads();
  T w = lane < kPlanWarps ? static_cast<T>(s.warp_sum[lane]) : T(0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *all = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return warp > 0 ? v + before : v;
}

// A barrier of the cluster, behind which what its threads wrote to global memory before is seen.  (One CTA alone is
// a cluster too, but its barrier takes longer than the block's.)
__device__ __forceinline__ void plan_sync(int C) {
  if (C == 1) __syncthreads();
  else cluster_sync_all();
}

// A number of every CTA's thread 0, each `slot` once a kernel: the sum of the ranks' before this one, and of all.
// Behind it a barrier as above.  (A CTA leaves only after one more barrier: its word may still be read.)
__device__ __forceinline__ unsigned long long exchange(PlanShared& s, int slot, unsigned long long v, int C, int rank,
                                                       unsigned long long* all) {
  if (C == 1) {
    __syncthreads();
    *all = v;
    return 0;
  }
  if (threadIdx.x == 0) s.word[slot] = v;
  cluster_sync_all();
  unsigned long long w[kPlanCluster];
#pragma unroll
  for (int r = 0; r < kPlanCluster; ++r) {
    w[r] = 0;
    if (r < C)
      asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(w[r]) : "r"(dsmem_map(smem_u32(&s.word[slot]), r)) : "memory");
  }
  unsigned long long before = 0, total = 0;
#pragma unroll
  for (int r = 0; r < kPlanCluster; ++r) {
    if (r == rank) before = total;
    total += w[r];
  }
  *all = total;
  return before;
}

// The bits of all CTAs' threads (s.bad starts as 0), through slot 0: a count for each bit, so that they add up.
__device__ __forceinline__ int cluster_or(PlanShared& s, int bits, int C, int rank) {
  if (bits != 0) atomicOr(&s.bad, bits);
  __syncthreads();
  const int mine = s.bad;
  if (C == 1) return mine;
  unsigned long long v = 0, all;
  for (int b = 0; b < 8; ++b) v |= static_cast<unsigned long long>(mine >> b & 1) << (8 * b);
  exchange(s, 0, v, C, rank, &all);
  int got = 0;
  for (int b = 0; b < 8; ++b) got |= (all >> (8 * b) & 255u) != 0 ? 1 << b : 0;
  return got;
}

// The lowest `need` pages whose count is 0, in order, to ids; false where there are fewer.  Uses slot 1.
__device__ bool lowest_free(const PagesParams& p, PlanShared& s, int need, int32_t* ids, int C, int rank) {
  if (need == 0) return true;
  const int lo = static_cast<int>(static_cast<long long>(p.n_pages) * rank / C);
  const int hi = static_cast<int>(static_cast<long long>(p.n_pages) * (rank + 1) / C);
  int mine = 0;
  for (int i = lo + threadIdx.x; i < hi; i += kPlanThreads) mine += __ldcg(p.refs + i) == 0;
  int own;
  block_scan(mine, s, &own);
  unsigned long long all;
  int at = static_cast<int>(exchange(s, 1, own, C, rank, &all));
  if (all < static_cast<unsigned long long>(need)) return false;
  for (int i0 = lo; i0 < hi && at < need; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int is = i < hi && __ldcg(p.refs + i) == 0;
    int n;
    const int r = at + block_scan(is, s, &n) - 1;
    if (is && r < need) ids[r] = i;
    at += n;
  }
  return true;
}

// The entries of a call: sequence x(i) and its length, from shared memory for the first ones.
struct Entries {
  const PlanShared& s;
  const int32_t *ids, *len;
  int which;
  __device__ __forceinline__ int x(int i) const { return i < kStaged ? s.x[which][i] : ids != nullptr ? ids[i] : i; }
  __device__ __forceinline__ int tokens(int i) const { return i < kStaged ? s.len[which][i] : len[x(i)]; }
};

// A bitmap of the sequences named by `ids`, the first of which go to shared memory with their lengths; returns
// BAD_BLOCK for one out of range or, where `once`, named twice.
__device__ int mark(uint32_t* bits, const PagesParams& p, PlanShared& s, int which, const int32_t* ids, bool once) {
  int bad = 0;
  for (int i = threadIdx.x; i < p.B; i += kPlanThreads) {
    const int x = ids != nullptr ? ids[i] : i;
    if (i < kStaged) s.x[which][i] = x;
    if (x < 0 || x >= p.n_seqs) {
      bad = ST_BAD_BLOCK;
    } else {
      if (i < kStaged) s.len[which][i] = p.len[x];
      const uint32_t old = atomicOr(&bits[x >> 5], 1u << (x & 31));
      if (once && (old >> (x & 31) & 1u)) bad = ST_BAD_BLOCK;
    }
  }
  return bad;
}

// Entries of table rows in pieces of 128, four a lane with their loads in flight together: f(row, j, entries) for
// the pieces of `B` rows that `count(i)` says hold anything, spread over the cluster's warps.
constexpr int kPiece = 128;
template <typename Count, typename F>
__device__ __forceinline__ void each_piece(const PagesParams& p, int B, int w0, int warps, Count&& count, F&& f) {
  const int per = (p.max_pages + kPiece - 1) / kPiece;
  const long long all = static_cast<long long>(B) * per;
  int i = w0 / per, c = w0 % per;
  for (long long w = w0; w < all; w += warps) {
    const int n = count(i) - c * kPiece;
    if (n > 0) f(i, c * kPiece, min(n, kPiece));
    i += warps / per;
    c += warps % per;
    if (c >= per) c -= per, ++i;
  }
}

// Whether the pages j0 .. j0 + n - 1 (up to 128) of sequence x's row, from `lo` on, are in the pool and held (a warp).
__device__ __forceinline__ int check_piece(const PagesParams& p, int x, int j0, int n, int lo) {
  const int32_t* row = p.table + static_cast<long long>(x) * p.max_pages + j0;
  int id[kPiece / 32], bad = 0;
#pragma unroll
  for (int k = 0; k < kPiece / 32; ++k) {
    const int j = (threadIdx.x & 31) + 32 * k;
    id[k] = j < n && j0 + j >= lo ? row[j] : -2;
  }
#pragma unroll
  for (int k = 0; k < kPiece / 32; ++k)
    if (id[k] != -2 && (id[k] < 0 || id[k] >= p.n_pages || p.refs[id[k]] < 1)) bad = ST_BAD_PAGE;
  // (an entry of -2 is out of the pool like -1)
#pragma unroll
  for (int k = 0; k < kPiece / 32; ++k) {
    const int j = (threadIdx.x & 31) + 32 * k;
    if (id[k] == -2 && j < n && j0 + j >= lo) bad = ST_BAD_PAGE;
  }
  return bad;
}

__device__ __forceinline__ int check_len(const PagesParams& p, int len) {
  return len < 0 || len > p.max_pages * kPage ? ST_SEQ_TOO_LONG : 0;
}

// dst[i] becomes a second src[i]: whole pages are shared, a part-full last one is copied.
__global__ void __launch_bounds__(kPlanThreads, 1) k_plan_fork(const PagesParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ PlanShared s;
  if (threadIdx.x == 0) s.bad = 0;
  pdl_wait();
  pdl_trigger();
  const int C = cluster_nctarank(), rank = cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = C * kPlanWarps, w0 = rank * kPlanWarps + warp;
  const int words = (p.n_seqs + 31) / 32;
  int32_t *ids = p.ws + kWsHead, *from = ids + p.n_pages, *to = from + p.n_pages;
  for (int i = threadIdx.x; i < 2 * words; i += kPlanThreads) bits[i] = 0;
  __syncthreads();
  int bad = mark(bits, p, s, 0, p.a, false) | mark(bits + words, p, s, 1, p.b, true);
  __syncthreads();
  for (int i = threadIdx.x; i < words; i += kPlanThreads)
    if (bits[i] & bits[words + i]) bad = ST_BAD_BLOCK;
  bad = __syncthreads_or(bad) ? ST_BAD_BLOCK : 0;
  const Entries src{s, p.a, p.len, 0}, dst{s, p.b, p.len, 1};
  if (!bad) {
    // (sources first, then targets; a bad length counts no pages)
    const auto seq = [&](int i) { return i < p.B ? src.x(i) : dst.x(i - p.B); };
    const auto len = [&](int i) { return i < p.B ? src.tokens(i) : dst.tokens(i - p.B); };
    for (int i = threadIdx.x; i < 2 * p.B; i += kPlanThreads) bad |= check_len(p, len(i));
    each_piece(p, 2 * p.B, w0, warps, [&](int i) { return check_len(p, len(i)) ? 0 : pages_of(len(i)); },
               [&](int i, int j0, int n) { bad |= check_piece(p, seq(i), j0, n, 0); });
  }
  bad = cluster_or(s, bad, C, rank);
  if (bad) {
    if (rank == 0 && threadIdx.x == 0) {
      p.ws[0] = 0;
      if (p.status != nullptr) atomicOr(p.status, bad);
    }
    return plan_sync(C);
  }
  // what the targets held goes
  const auto release = [&](int by) {
    each_piece(p, p.B, w0, warps, [&](int i) { return pages_of(dst.tokens(i)); }, [&](int i, int j0, int n) {
      const int32_t* row = p.table + static_cast<long long>(dst.x(i)) * p.max_pages + j0;
#pragma unroll
      for (int k = 0; k < kPiece / 32; ++k)
        if (lane + 32 * k < n) atomicAdd(p.refs + row[lane + 32 * k], by);
    });
  };
  release(-1);
  // every entry's place among the copies
  int32_t* place = to + p.n_pages;
  int need = 0;
  for (int i0 = 0; i0 < p.B; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x, is = i < p.B && src.tokens(i) % kPage != 0;
    int n;
    const int r = need + block_scan(is, s, &n) - is;
    if (rank == 0 && i < p.B) place[i] = r;
    need += n;
  }
  plan_sync(C);
  if (!lowest_free(p, s, need, ids, C, rank)) {
    release(1);
    if (rank == 0 && threadIdx.x == 0) {
      p.ws[0] = 0;
      if (p.status != nullptr) atomicOr(p.status, ST_POOL_EXHAUSTED);
    }
    return plan_sync(C);
  }
  plan_sync(C);
  each_piece(
      p, p.B, w0, warps, [&](int i) { return max(pages_of(src.tokens(i)), pages_of(dst.tokens(i))); },
      [&](int i, int j0, int n) {
        const int len = src.tokens(i), whole = len / kPage, held = pages_of(len), slot = place[i];
        const int32_t* from_row = p.table + static_cast<long long>(src.x(i)) * p.max_pages + j0;
        int32_t* row = p.table + static_cast<long long>(dst.x(i)) * p.max_pages + j0;
        int id[kPiece / 32];
#pragma unroll
        for (int k = 0; k < kPiece / 32; ++k)
          id[k] = lane + 32 * k < n && j0 + lane + 32 * k < held ? from_row[lane + 32 * k] : -1;
#pragma unroll
        for (int k = 0; k < kPiece / 32; ++k) {
          const int j = j0 + lane + 32 * k;
          if (lane + 32 * k >= n) continue;
          if (j < whole) {
            atomicAdd(p.refs + id[k], 1);
          } else if (j < held) {
            from[slot] = id[k];
            to[slot] = id[k] = ids[slot];
            p.refs[id[k]] = 1;
          }
          row[lane + 32 * k] = id[k];
        }
      });
  // (lengths of targets once all of the cluster has read them)
  plan_sync(C);
  for (int i = rank * kPlanThreads + threadIdx.x; i < p.B; i += C * kPlanThreads) p.len[dst.x(i)] = src.tokens(i);
  if (rank == 0 && threadIdx.x == 0) p.ws[0] = need;
}

// Sequence seq[i] keeps its first new_len[i] tokens.
__global__ void __launch_bounds__(kPlanThreads, 1) k_plan_truncate(const PagesParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ PlanShared s;
  if (threadIdx.x == 0) s.bad = 0;
  pdl_wait();
  pdl_trigger();
  const int C = cluster_nctarank(), rank = cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = C * kPlanWarps, w0 = rank * kPlanWarps + warp;
  for (int i = threadIdx.x; i < (p.n_seqs + 31) / 32; i += kPlanThreads) bits[i] = 0;
  __syncthreads();
  int bad = mark(bits, p, s, 0, p.a, true);
  bad = __syncthreads_or(bad) ? ST_BAD_BLOCK : 0;
  const Entries seq{s, p.a, p.len, 0};
  const auto keep = [&](int i) { return p.b != nullptr ? p.b[i] : 0; };
  if (!bad) {
    for (int i = threadIdx.x; i < p.B; i += kPlanThreads) bad |= check_len(p, seq.tokens(i)) | (keep(i) < 0 ? ST_BAD_ROWS : 0);
    each_piece(p, p.B, w0, warps, [&](int i) { return check_len(p, seq.tokens(i)) ? 0 : pages_of(seq.tokens(i)); },
               [&](int i, int j0, int n) {
                 const int lo = keep(i) < 0 ? 0 : pages_of(keep(i));
                 if (lo < j0 + n) bad |= check_piece(p, seq.x(i), j0, n, lo);
               });
  }
  bad = cluster_or(s, bad, C, rank);
  if (bad) {
    if (rank == 0 && threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, bad);
    return plan_sync(C);
  }
  each_piece(p, p.B, w0, warps, [&](int i) { return pages_of(seq.tokens(i)); }, [&](int i, int j0, int n) {
    const int lo = pages_of(keep(i));
    if (lo >= j0 + n) return;
    int32_t* row = p.table + static_cast<long long>(seq.x(i)) * p.max_pages + j0;
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k) {
      const int j = lane + 32 * k;
      if (j >= n || j0 + j < lo) continue;
      atomicAdd(p.refs + row[j], -1);
      row[j] = -1;
    }
  });
  plan_sync(C);
  for (int i = rank * kPlanThreads + threadIdx.x; i < p.B; i += C * kPlanThreads)
    if (keep(i) < seq.tokens(i)) p.len[seq.x(i)] = keep(i);
}

// Sequence seq[i] gets room for n_rows[i] more tokens; a part-full last page that others hold is copied.
__global__ void __launch_bounds__(kPlanThreads, 1) k_plan_reserve(const PagesParams p) {
  extern __shared__ uint32_t bits[];
  __shared__ PlanShared s;
  if (threadIdx.x == 0) s.bad = 0;
  pdl_wait();
  pdl_trigger();
  const int C = cluster_nctarank(), rank = cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = C * kPlanWarps, w0 = rank * kPlanWarps + warp;
  int32_t *ids = p.ws + kWsHead, *from = ids + p.n_pages, *to = from + p.n_pages;
  for (int i = threadIdx.x; i < (p.n_seqs + 31) / 32; i += kPlanThreads) bits[i] = 0;
  __syncthreads();
  int bad = mark(bits, p, s, 0, p.a, true);
  bad = __syncthreads_or(bad) ? ST_BAD_BLOCK : 0;
  const Entries seq{s, p.a, p.len, 0};
  // Whether entry i can be (0, or what is wrong), the pages that it needs, and whether its last one is copied.
  const auto want = [&](int i, int& pages, int& copy) {
    const int len = seq.tokens(i), n = p.b[i];
    pages = copy = 0;
    int e = check_len(p, len);
    if (n < 0) e |= ST_BAD_ROWS;
    else if (!e && n > p.max_pages * kPage - len) e |= ST_SEQ_TOO_LONG;
    if (e) return e;
    if (n > 0 && len % kPage != 0) {
      const int id = p.table[static_cast<long long>(seq.x(i)) * p.max_pages + len / kPage];
      if (id < 0 || id >= p.n_pages) return static_cast<int>(ST_BAD_PAGE);
      const int held = __ldcg(p.refs + id);
      if (held < 1) return static_cast<int>(ST_BAD_PAGE);
      copy = held > 1;
    }
    pages = min(pages_of(len + n) - pages_of(len) + copy, p.n_pages + 1);
    return 0;
  };
  // every entry's first place among the new pages, and among the copies (-1: none), before any count changes
  int32_t* place = to + p.n_pages;
  // (all are looked at, even behind those that want more than there is: what is wrong with an entry comes before
  // pages that are missing for others)
  int need = 0, copies = 0;
  for (int i0 = 0; i0 < p.B; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int copy = 0, n = 0;
    if (i < p.B && !bad) bad |= want(i, n, copy);
    unsigned long long all;
    const unsigned long long mine = static_cast<unsigned long long>(copy) << 40 | static_cast<unsigned>(n);
    const unsigned long long upto = block_scan(mine, s, &all) - mine;
    if (rank == 0 && i < p.B) {
      place[2 * i] = need + static_cast<int>(upto & 0xffffffffffull);
      place[2 * i + 1] = copy ? copies + static_cast<int>(upto >> 40) : -1;
    }
    need = min(need + static_cast<int>(all & 0xffffffffffull), p.n_pages + 1);
    copies += static_cast<int>(all >> 40);
  }
  bad = cluster_or(s, bad, C, rank);
  if (!bad && (need > p.n_pages || !lowest_free(p, s, need, ids, C, rank))) bad = ST_POOL_EXHAUSTED;
  if (bad) {
    if (rank == 0 && threadIdx.x == 0) {
      p.ws[0] = 0;
      if (p.status != nullptr) atomicOr(p.status, bad);
    }
    return plan_sync(C);
  }
  plan_sync(C);
  for (int i = w0; i < p.B; i += warps) {
    const int len = seq.tokens(i), at = place[2 * i], slot = place[2 * i + 1];
    const int first = pages_of(len) - (slot >= 0), n = pages_of(len + p.b[i]) - first;
    int32_t* row = p.table + static_cast<long long>(seq.x(i)) * p.max_pages + first;
    for (int j = lane; j < n; j += 32) {
      const int id = ids[at + j];
      if (j == 0 && slot >= 0) {
        from[slot] = row[0];
        to[slot] = id;
        atomicAdd(p.refs + row[0], -1);
      }
      row[j] = id;
      p.refs[id] = 1;
    }
  }
  plan_sync(C);
  for (int i = rank * kPlanThreads + threadIdx.x; i < p.B; i += C * kPlanThreads) p.len[seq.x(i)] = seq.tokens(i) + p.b[i];
  if (rank == 0 && threadIdx.x == 0) p.ws[0] = copies;
}

// Where every page goes: those with a count, in order, to the lowest ids.  Pages
// that are there already stay; the r-th of the others goes to the r-th hole.
__global__ void __launch_bounds__(kPlanThreads, 1) k_plan_compact(const PagesParams p) {
  __shared__ PlanShared s;
  if (threadIdx.x == 0) s.bad = 0;
  pdl_wait();
  pdl_trigger();
  const int C = cluster_nctarank(), rank = cluster_ctarank();
  const int warp = threadIdx.x >> 5, warps = C * kPlanWarps, w0 = rank * kPlanWarps + warp;
  int32_t *map = p.ws + kWsHead, *from = map + p.n_pages, *to = from + p.n_pages;
  const int lo = static_cast<int>(static_cast<long long>(p.n_pages) * rank / C);
  const int hi = static_cast<int>(static_cast<long long>(p.n_pages) * (rank + 1) / C);
  __syncthreads();
  int bad = 0, mine = 0;
  for (int i = lo + threadIdx.x; i < hi; i += kPlanThreads) {
    const int r = p.refs[i];
    if (r < 0) bad = ST_BAD_PAGE;
    mine += r > 0;
  }
  for (int x = threadIdx.x; x < p.n_seqs; x += kPlanThreads) bad |= check_len(p, p.len[x]);
  each_piece(p, p.n_seqs, w0, warps, [&](int x) { return check_len(p, p.len[x]) ? 0 : pages_of(p.len[x]); },
             [&](int x, int j0, int n) { bad |= check_piece(p, x, j0, n, 0); });
  int own;
  block_scan(mine, s, &own);
  unsigned long long total;
  bad = cluster_or(s, bad, C, rank);
  if (bad) {
    if (rank == 0 && threadIdx.x == 0) {
      p.ws[0] = p.ws[1] = 0;
      if (p.status != nullptr) atomicOr(p.status, bad);
    }
    return plan_sync(C);
  }
  exchange(s, 1, own, C, rank, &total);
  const int used = static_cast<int>(total);
  // holes (low half) and movers of this CTA's share, and of those before
  const auto kind = [&](int i) -> unsigned long long {
    const bool is = p.refs[i] > 0;
    return !is && i < used ? 1ull : is && i >= used ? 1ull << 32 : 0ull;
  };
  unsigned long long hm = 0, at, all;
  for (int i = lo + threadIdx.x; i < hi; i += kPlanThreads) hm += kind(i);
  block_scan(hm, s, &hm);
  at = exchange(s, 2, hm, C, rank, &all);
  const int all_m = static_cast<int>(all >> 32);
  for (int i0 = lo; i0 < hi; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const unsigned long long k = i < hi ? kind(i) : 0;
    unsigned long long n;
    const unsigned long long r = at + block_scan(k, s, &n) - k;
    if (k == 1) to[r & 0xffffffffu] = i;
    if (k > 1) from[r >> 32] = i;
    if (i < hi) map[i] = p.refs[i] > 0 ? i : -1;  // (a mover's until its target is known)
    at += n;
  }
  plan_sync(C);
  // counts: one thread has a mover's and its hole's
  const int t = rank * kPlanThreads + threadIdx.x, step = C * kPlanThreads;
  for (int r = t; r < all_m; r += step) {
    const int a = __ldcg(from + r), b = __ldcg(to + r), n = p.refs[a];
    map[a] = b;
    p.refs_out[b] = n;
    p.refs_out[a] = 0;
    if (p.page_map != nullptr) p.page_map[a] = b;
  }
  for (int i = lo + threadIdx.x; i < hi; i += kPlanThreads) {
    const int to_i = __ldcg(map + i);
    // (at and past `used` only movers' entries are not negative, whether they are known yet or not)
    if (i >= used) {
      if (to_i < 0) {
        p.refs_out[i] = 0;
        if (p.page_map != nullptr) p.page_map[i] = -1;
      }
    } else {
      if (to_i == i) p.refs_out[i] = p.refs[i];
      if (p.page_map != nullptr) p.page_map[i] = to_i;
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.ws[0] = all_m;
    p.ws[1] = 1;
    if (p.n_used != nullptr) *p.n_used = used;
  }
}

// L: the most layers (4 KB of addresses a launch cost more than it for a pool of a few).
template <int L>
struct CopyParams {
  uint8_t* to[2 * L];                    // pages of layer l: keys 2 l, values 2 l + 1
  const uint8_t* from[2 * L];
  int arrays, bytes;                     // 2 x layers; a page's bytes in one of them
  int n_from, n_to;                      // pages of the pools
  const int32_t *count, *src, *dst;      // pairs (count null: n of them)
  int n;
  int* status;
  // compact: rows of the table through the map
  const int32_t *table, *len, *map, *go;
  int32_t* table_out;
  int n_seqs, max_pages;
};

// V bytes of a lane's access: 32 where all pages lie at whole 32 bytes (half the instructions), else 16.
template <int V>
struct Bytes {
  uint32_t w[V / 4];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (V == 32)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p)
                   : "memory");
    else
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p)
                   : "memory");
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
    if constexpr (V == 32)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                   "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    else
      asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
  }
};

// Bound by memory.  A warp takes pieces of 2 KB, 64 bytes a lane; the piece's page, layer and place step on
// by additions, since a division a vector takes longer than the copy.
template <int V, int L>
__global__ void __launch_bounds__(kCopyThreads) k_copy_pages(const __grid_constant__ CopyParams<L> p) {
  constexpr int N = kCopyBytes / V;
  const int lane = threadIdx.x & 31;
  const int per = (p.bytes + 32 * kCopyBytes - 1) / (32 * kCopyBytes);  // pieces a page
  const unsigned w0 = (blockIdx.x * kCopyThreads + threadIdx.x) / 32, warps = gridDim.x * (kCopyThreads / 32);
  int pair = w0 / (per * p.arrays), array = w0 / per % p.arrays, piece = w0 % per;
  const int d_pair = warps / (per * p.arrays), d_array = warps / per % p.arrays, d_piece = warps % per;
  pdl_wait();
  pdl_trigger();
  const int n = p.count != nullptr ? *p.count : p.n;
  while (pair < n) {
    const int a = p.src[pair], b = p.dst[pair];
    if (a < 0 || a >= p.n_from || b < 0 || b >= p.n_to) {
      if (array == 0 && piece == 0 && lane == 0 && p.status != nullptr) atomicOr(p.status, ST_BAD_PAGE);
    } else {
      const uint8_t* from = p.from[array] + static_cast<long long>(a) * p.bytes;
      uint8_t* to = p.to[array] + static_cast<long long>(b) * p.bytes;
      const int at = piece * (32 * kCopyBytes) + lane * V;
      Bytes<V> v[N];
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (at + 32 * V * k < p.bytes) v[k].load(from + at + 32 * V * k);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (at + 32 * V * k < p.bytes) v[k].store(to + at + 32 * V * k);
    }
    pair += d_pair;
    array += d_array;
    piece += d_piece;
    if (piece >= per) piece -= per, ++array;
    if (array >= p.arrays) array -= p.arrays, ++pair;
  }
  if (p.table_out != nullptr && *p.go != 0) {
    const long long entries = static_cast<long long>(p.n_seqs) * p.max_pages;
    for (long long e = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries;
         e += static_cast<long long>(gridDim.x) * kCopyThreads) {
      const int x = static_cast<int>(e / p.max_pages), j = static_cast<int>(e - static_cast<long long>(x) * p.max_pages);
      p.table_out[e] = j < pages_of(p.len[x]) ? p.map[p.table[e]] : -1;
    }
  }
}

bool off(const void* a, int n) { return reinterpret_cast<uintptr_t>(a) % n != 0; }

// Pointers, counts and alignment of a pool; its head_dim as the cache's other calls have it.
dflash_status pool_ok(const dflash_page_pool* p) {
  if (p == nullptr || p->k == nullptr || p->v == nullptr || p->page_table == nullptr || p->seq_len == nullptr ||
      p->refs == nullptr || p->n_layers < 1 || p->n_pages < 1 || p->n_seqs < 1 || p->max_pages < 1 ||
      p->n_kv_heads < 1 || p->head_dim < 1)
    return DFLASH_ERR_INVALID_ARG;
  if (p->elem != DFLASH_ELEM_F32 && p->elem != DFLASH_ELEM_BF16 && p->elem != DFLASH_ELEM_F16)
    return DFLASH_ERR_INVALID_ARG;
  if (off(p->page_table, 4) || off(p->seq_len, 4) || off(p->refs, 4)) return DFLASH_ERR_INVALID_ARG;
  if (p->n_layers > kMaxLayers || (p->head_dim != 32 && p->head_dim != 64 && p->head_dim != 128) ||
      p->n_seqs > kMaxSeqs || p->max_pages > INT32_MAX / (2 * kPage) || p->n_kv_heads > 1 << 16 || p->n_pages > kMaxPages)
    return DFLASH_ERR_UNSUPPORTED_SHAPE;
  for (int l = 0; l < p->n_layers; ++l)
    if (p->k[l] == nullptr || p->v[l] == nullptr || off(p->k[l], 16) || off(p->v[l], 16)) return DFLASH_ERR_INVALID_ARG;
  return DFLASH_OK;
}

int page_bytes(const dflash_page_pool& p) {
  return p.n_kv_heads * kPage * p.head_dim * (p.elem == DFLASH_ELEM_F32 ? 4 : 2);
}

PagesParams params(const dflash_page_pool& q, const int32_t* a, const int32_t* b, int B, void* ws, int* status) {
  PagesParams p{};
  p.table = q.page_table;
  p.len = q.seq_len;
  p.refs = q.refs;
  p.n_pages = q.n_pages;
  p.n_seqs = q.n_seqs;
  p.max_pages = q.max_pages;
  p.a = a;
  p.b = b;
  p.B = B;
  p.ws = static_cast<int32_t*>(ws);
  p.status = status;
  return p;
}

// The plan: one cluster, of more CTAs where tables and counts are long.
template <typename K>
cudaError_t launch_plan(K kernel, FuncAttr& attr, const PagesParams& p, long long entries, int bitmaps, cudaStream_t s) {
  const int smem = bitmaps * ((p.n_seqs + 31) / 32) * 4;
  const cudaError_t e = attr.ensure(std::max(smem, 1), [&](int v) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  int C = 1;
  while (C < kPlanCluster && entries > 1ll * kPlanThreads * C) C *= 2;
  return launch_cached(kernel, C, kPlanThreads, smem, s, C, p);
}

// The copies, at most `most` pages: started early, behind the plan.  `set` fills in the rest.
template <int L, typename Set>
cudaError_t launch_copy_l(const dflash_page_pool& to, const dflash_page_pool& from, long long most,
                          cudaStream_t s, Set&& set) {
  CopyParams<L> p{};
  bool wide = true;
  for (int l = 0; l < to.n_layers; ++l) {
    p.to[2 * l] = static_cast<uint8_t*>(to.k[l]);
    p.to[2 * l + 1] = static_cast<uint8_t*>(to.v[l]);
    p.from[2 * l] = static_cast<const uint8_t*>(from.k[l]);
    p.from[2 * l + 1] = static_cast<const uint8_t*>(from.v[l]);
    wide = wide && !off(to.k[l], 32) && !off(to.v[l], 32) && !off(from.k[l], 32) && !off(from.v[l], 32);
  }
  p.arrays = 2 * to.n_layers;
  p.bytes = page_bytes(to);
  p.n_from = from.n_pages;
  p.n_to = to.n_pages;
  set(p);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long blocks = (most * p.arrays * p.bytes + kCopyThreads * kCopyBytes - 1) / (kCopyThreads * kCopyBytes);
  // (far more blocks than run at once: 1 GB moved, 8 a SM 187 us with the plan, 32 177, 64 175)
  const long long grid = std::max(1ll, std::min(blocks, 64ll * sms));
  return launch_cached(wide ? k_copy_pages<32, L> : k_copy_pages<16, L>, static_cast<unsigned>(grid), kCopyThreads, 0, s, 1, p);
}

template <typename Set>
cudaError_t launch_copy(const dflash_page_pool& to, const dflash_page_pool& from, long long most, cudaStream_t s,
                        Set&& set) {
  return to.n_layers <= 8 ? launch_copy_l<8>(to, from, most, s, set)
                          : launch_copy_l<kMaxLayers>(to, from, most, s, set);
}

dflash_status answer(cudaError_t e) { return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA; }

// Whether a call's arrays lie apart from the pool's and from its workspace.  (Entries are read, checked and read again
// while tables, lengths, counts and lists are written.)
bool apart(const dflash_page_pool& q, const PagesParams& p, std::initializer_list<Span> arrays) {
  const Span own[] = {ints(q.page_table, static_cast<long long>(q.n_seqs) * q.max_pages), ints(q.seq_len, q.n_seqs),
                      ints(q.refs, q.n_pages)},
             ws = {p.ws, p.ws != nullptr ? 4 * ws_ints(q.n_pages, q.n_seqs) : 0};
  for (const Span& o : own) {
    if (!apart(ws, o)) return false;
    for (const Span& a : arrays)
      if (!apart(a, o)) return false;
  }
  for (const Span& a : arrays)
    if (!apart(a, ws)) return false;
  return true;
}

// (The lengths themselves, of entry i for sequence i: its thread reads them before it writes them.)
const int32_t* by_itself(const dflash_page_pool& q, const int32_t* seq, const int32_t* b) {
  return seq == nullptr && b == q.seq_len ? nullptr : b;
}

// Counts and workspace of a call on B sequences.
dflash_status call_ok(const dflash_page_pool* q, int B, const void* ws, size_t bytes, const int* status) {
  const dflash_status e = pool_ok(q);
  if (e != DFLASH_OK) return e;
  if (B < 1 || B > q->n_seqs || ws == nullptr || off(ws, 16) || off(status, 4)) return DFLASH_ERR_INVALID_ARG;
  if (bytes < static_cast<size_t>(ws_ints(q->n_pages, q->n_seqs)) * 4) return DFLASH_ERR_WORKSPACE;
  return DFLASH_OK;
}

}  // namespace

}  // namespace dflash

using namespace dflash;

extern "C" {

size_t dflash_pages_workspace(const dflash_page_pool* pool) {
  return pool_ok(pool) == DFLASH_OK ? static_cast<size_t>(ws_ints(pool->n_pages, pool->n_seqs)) * 4 : 0;
}

dflash_status dflash_pages_fork(const dflash_page_pool* pool, const int32_t* src, const int32_t* dst, int B,
                                void* workspace, size_t workspace_bytes, int* status, dflash_stream stream) {
  const dflash_status c = call_ok(pool, B, workspace, workspace_bytes, status);
  if (c != DFLASH_OK) return c;
  if (src == nullptr || dst == nullptr || off(src, 4) || off(dst, 4)) return DFLASH_ERR_INVALID_ARG;
  const PagesParams p = params(*pool, src, dst, B, workspace, status);
  if (!apart(*pool, p, {ints(src, B), ints(dst, B), ints(status, 1)})) return DFLASH_ERR_INVALID_ARG;
  static FuncAttr attr;
  cudaError_t e = launch_plan(k_plan_fork, attr, p, 2ll * B * pool->max_pages + pool->n_pages, 2, stream);
  if (e != cudaSuccess) return DFLASH_ERR_CUDA;
  return answer(launch_copy(*pool, *pool, B, stream, [&](auto& q) {
    q.count = p.ws;
    q.src = p.ws + kWsHead + pool->n_pages;
    q.dst = q.src + pool->n_pages;
  }));
}

dflash_status dflash_pages_truncate(const dflash_page_pool* pool, const int32_t* seq, const int32_t* new_len, int B,
                                    int* status, dflash_stream stream) {
  const dflash_status c = pool_ok(pool);
  if (c != DFLASH_OK) return c;
  if (B < 1 || B > pool->n_seqs || off(seq, 4) || off(new_len, 4) || off(status, 4)) return DFLASH_ERR_INVALID_ARG;
  const PagesParams p = params(*pool, seq, new_len, B, nullptr, status);
  if (!apart(*pool, p, {ints(seq, B), ints(by_itself(*pool, seq, new_len), B), ints(status, 1)})) return DFLASH_ERR_INVALID_ARG;
  static FuncAttr attr;
  return answer(launch_plan(k_plan_truncate, attr, p, static_cast<long long>(B) * pool->max_pages, 1, stream));
}

dflash_status dflash_pages_reserve(const dflash_page_pool* pool, const int32_t* seq, const int32_t* n_rows, int B,
                                   void* workspace, size_t workspace_bytes, int* status, dflash_stream stream) {
  const dflash_status c = call_ok(pool, B, workspace, workspace_bytes, status);
  if (c != DFLASH_OK) return c;
  if (n_rows == nullptr || off(seq, 4) || off(n_rows, 4)) return DFLASH_ERR_INVALID_ARG;
  const PagesParams p = params(*pool, seq, n_rows, B, workspace, status);
  if (!apart(*pool, p, {ints(seq, B), ints(by_itself(*pool, seq, n_rows), B), ints(status, 1)})) return DFLASH_ERR_INVALID_ARG;
  static FuncAttr attr;
  cudaError_t e = launch_plan(k_plan_reserve, attr, p, pool->n_pages, 1, stream);
  if (e != cudaSuccess) return DFLASH_ERR_CUDA;
  return answer(launch_copy(*pool, *pool, B, stream, [&](auto& q) {
    q.count = p.ws;
    q.src = p.ws + kWsHead + pool->n_pages;
    q.dst = q.src + pool->n_pages;
  }));
}

dflash_status dflash_pages_compact(const dflash_page_pool* pool, int32_t* table_out, int32_t* refs_out,
                                   int32_t* page_map, int32_t* n_used, void* workspace, size_t workspace_bytes,
                                   int* status, dflash_stream stream) {
  const dflash_status c = call_ok(pool, 1, workspace, workspace_bytes, status);
  if (c != DFLASH_OK) return c;
  if (off(table_out, 4) || off(refs_out, 4) || off(page_map, 4) || off(n_used, 4)) return DFLASH_ERR_INVALID_ARG;
  PagesParams p = params(*pool, nullptr, nullptr, 0, workspace, status);
  const long long entries = static_cast<long long>(pool->n_seqs) * pool->max_pages;
  // (the pool's own arrays may be named as outputs)
  if (table_out == pool->page_table) table_out = nullptr;
  if (refs_out == pool->refs) refs_out = nullptr;
  if (!apart(*pool, p, {ints(table_out, entries), ints(refs_out, pool->n_pages), ints(page_map, pool->n_pages), ints(n_used, 1),
                        ints(status, 1)}))
    return DFLASH_ERR_INVALID_ARG;
  p.table_out = table_out != nullptr ? table_out : pool->page_table;
  p.refs_out = refs_out != nullptr ? refs_out : pool->refs;
  p.page_map = page_map;
  p.n_used = n_used;
  static FuncAttr attr;
  cudaError_t e = launch_plan(k_plan_compact, attr, p, pool->n_pages + entries, 0, stream);
  if (e != cudaSuccess) return DFLASH_ERR_CUDA;
  // (at least as many threads as the table has entries, up to a full GPU)
  const long long rows = entries * kCopyBytes / (2ll * pool->n_layers * page_bytes(*pool)) + 1;
  return answer(launch_copy(*pool, *pool, std::max<long long>(pool->n_pages / 2, rows), stream, [&](auto& q) {
    q.count = p.ws;
    q.go = p.ws + 1;
    q.map = p.ws + kWsHead;
    q.src = q.map + pool->n_pages;
    q.dst = q.src + pool->n_pages;
    q.table = pool->page_table;
    q.len = pool->seq_len;
    q.table_out = p.table_out;
    q.n_seqs = pool->n_seqs;
    q.max_pages = pool->max_pages;
  }));
}

dflash_status dflash_pages_copy(const dflash_page_pool* to, const dflash_page_pool* from, const int32_t* dst,
                                const int32_t* src, int n, int* status, dflash_stream stream) {
  dflash_status c = pool_ok(to);
  if (c == DFLASH_OK) c = pool_ok(from);
  if (c != DFLASH_OK) return c;
  if (src == nullptr || dst == nullptr || off(src, 4) || off(dst, 4) || off(status, 4) || n < 1 || n > to->n_pages)
    return DFLASH_ERR_INVALID_ARG;
  if (to->n_layers != from->n_layers || to->n_kv_heads != from->n_kv_heads || to->head_dim != from->head_dim ||
      to->elem != from->elem)
    return DFLASH_ERR_INVALID_ARG;
  return answer(launch_copy(*to, *from, n, stream, [&](auto& q) {
    q.src = src;
    q.dst = dst;
    q.n = n;
    q.status = status;
  }));
}

}  // extern "C"
