// dflash_append_kv, dflash_extend and dflash_rope_table: keys and values that
// the caller has in hand into a paged cache, with the position rotation of
// the keys (and of the step's queries) applied on the way.
//
// A row (batch entry b, token i) stands at slot seq_len - n + i of its
// sequence; key and query elements x_i and x_{i+h} (h = head_dim / 2) rotate
// as a pair by the table's angle of the row's position.
#include "common.cuh"
#include "kernels.cuh"

namespace dflash {

namespace {

// Eight elements of a row in registers as fp32.  vec: the address is
// 16-byte aligned, so they come and go as 128-bit accesses.
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, float (&x)[8]) {
  if (vec) {
    constexpr int W = 16 / sizeof(T);  // elements per 128-bit access
#pragma unroll
    for (int j = 0; j < 8 / W; ++j) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + j * W);
      T t[W];
      memcpy(t, &u, 16);
#pragma unroll
      for (int k = 0; k < W; ++k) x[j * W + k] = to_f32<T>(t[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = to_f32<T>(p[k]);
  }
}

template <typename T>
__device__ __forceinline__ T round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half round_to<__half>(float v) { return __float2half_rn(v); }

// (the pool and q_out are 16-byte aligned, and so is every 8-element piece of a head)
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  constexpr int W = 16 / sizeof(T);
#pragma unroll
  for (int j = 0; j < 8 / W; ++j) {
    T t[W];
#pragma unroll
    for (int k = 0; k < W; ++k) t[k] = round_to<T>(x[j * W + k]);
    uint4 u;
    memcpy(&u, t, 16);
    *reinterpret_cast<uint4*>(p + j * W) = u;
  }
}

struct AppendParams {
  const void *k, *v, *q;
  long long ld_k, ld_v, ld_q;
  void *pool_k, *pool_v, *q_out;
  const int32_t *n_rows, *seq, *pos_base, *page_table, *seq_len;
  const float *rope_cos, *rope_sin;
  int rope_rows, B, T, Hq, Hkv, n_pages, n_seqs, max_pages;
  bool vec_k, vec_v, vec_q;
  int* status;
};

constexpr int kAppendThreads = 256;

// A unit is one head of one row: DH / 16 threads, each with eight elements
// of the head's first half and the eight they rotate with.
template <typename S, typename D, int DH>
__global__ void __launch_bounds__(kAppendThreads) k_append(const AppendParams p) {
  constexpr int TPU = DH / 16, HALF = DH / 2;
  const int heads = p.Hq + 2 * p.Hkv;
  const long long u = (static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x) / TPU;
  const int d = (threadIdx.x % TPU) * 8;
  const long long row = u / heads;
  if (row >= static_cast<long long>(p.B) * p.T) return;
  const int h = static_cast<int>(u - row * heads);
  const int b = static_cast<int>(row / p.T), i = static_cast<int>(row - static_cast<long long>(b) * p.T);
  const bool first = h == 0 && d == 0;  // the thread that reports
  auto flag = [&](int bit) {
    if (first && p.status != nullptr) atomicOr(p.status, bit);
  };
  const int n = p.n_rows != nullptr ? p.n_rows[b] : p.T;
  const int s = p.seq != nullptr ? p.seq[b] : b;
  int bad = 0;
  if (n < 0 || n > p.T) bad |= ST_BAD_ROWS;
  if (s < 0 || s >= p.n_seqs) bad |= ST_BAD_BLOCK;
  if (bad) return flag(bad);
  if (i >= n) return;
  const int len = p.seq_len[s];
  if (len < n) return flag(ST_BAD_ROWS);
  if (len > p.max_pages * kPage) return flag(ST_SEQ_TOO_LONG);
  const int slot = len - n + i;
  const bool rope = p.rope_cos != nullptr;
  const int page = p.page_table[static_cast<long long>(s) * p.max_pages + slot / kPage];
  const long long pos = static_cast<long long>(slot) + (p.pos_base != nullptr ? p.pos_base[b] : 0);
  if (page < 0 || page >= p.n_pages) return flag(ST_BAD_PAGE);
  if (rope && (pos < 0 || pos >= p.rope_rows)) return flag(ST_BAD_POS);

  const S* src;
  bool vec;
  D* dst;
  bool turn = rope;
  if (h < p.Hq) {
    src = static_cast<const S*>(p.q) + row * p.ld_q + h * DH;
    vec = p.vec_q;
    dst = static_cast<D*>(p.q_out) + (row * p.Hq + h) * DH;
  } else {
    const int hk = h - p.Hq;
    const bool is_v = hk >= p.Hkv;
    const int hh = is_v ? hk - p.Hkv : hk;
    src = static_cast<const S*>(is_v ? p.v : p.k) + row * (is_v ? p.ld_v : p.ld_k) + hh * DH;
    vec = is_v ? p.vec_v : p.vec_k;
    dst = static_cast<D*>(is_v ? p.pool_v : p.pool_k) +
          ((static_cast<long long>(page) * p.Hkv + hh) * kPage + slot % kPage) * DH;
    turn = rope && !is_v;
  }
  float x1[8], x2[8];
  load8<S>(src + d, vec, x1);
  load8<S>(src + HALF + d, vec, x2);
  if (turn) {
    float c[8], sn[8];
    load8<float>(p.rope_cos + pos * HALF + d, true, c);
    load8<float>(p.rope_sin + pos * HALF + d, true, sn);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = x1[k], e = x2[k];
      x1[k] = a * c[k] - e * sn[k];
      x2[k] = e * c[k] + a * sn[k];
    }
  }
  store8<D>(dst + d, x1);
  store8<D>(dst + HALF + d, x2);
}

template <typename S, typename D>
cudaError_t launch_append_t(const AppendParams& p, int dh, unsigned blocks, cudaStream_t s) {
  switch (dh) {
    case 32: k_append<S, D, 32><<<blocks, kAppendThreads, 0, s>>>(p); break;
    case 64: k_append<S, D, 64><<<blocks, kAppendThreads, 0, s>>>(p); break;
    default: k_append<S, D, 128><<<blocks, kAppendThreads, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

template <typename S>
cudaError_t launch_append_s(const AppendParams& p, int elem, int dh, unsigned blocks, cudaStream_t s) {
  if (elem == DFLASH_ELEM_F32) return launch_append_t<S, float>(p, dh, blocks, s);
  if (elem == DFLASH_ELEM_BF16) return launch_append_t<S, __nv_bfloat16>(p, dh, blocks, s);
  return launch_append_t<S, __half>(p, dh, blocks, s);
}

}  // namespace

}  // namespace dflash

using namespace dflash;

extern "C" {

dflash_status dflash_rope_table(float* rope_cos, float* rope_sin, int rows, int head_dim, double theta,
                                dflash_stream stream) {
  if (rope_cos == nullptr || rope_sin == nullptr || rows < 1 || !(theta > 0.0)) return DFLASH_ERR_INVALID_ARG;
  if (head_dim != 32 && head_dim != 64 && head_dim != 128) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<long long>(rows) * (head_dim / 2) > INT32_MAX) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (launch_rope_table(rope_cos, rope_sin, rows, head_dim, theta, stream) != cudaSuccess) return DFLASH_ERR_CUDA;
  return DFLASH_OK;
}

dflash_status dflash_append_kv(const dflash_paged_kv* kv, const void* k, long long ld_k, const void* v, long long ld_v,
                               int src_elem, const int32_t* n_rows, const int32_t* seq, const int32_t* pos_base,
                               int B, int T, const float* rope_cos, const float* rope_sin, int rope_rows,
                               const void* q, long long ld_q, int n_q_heads, void* q_out, int* status,
                               dflash_stream stream) {
  if (!paged_kv_ok(kv) || k == nullptr || v == nullptr || B < 1 || T < 1) return DFLASH_ERR_INVALID_ARG;
  if (src_elem != DFLASH_ELEM_F32 && src_elem != DFLASH_ELEM_BF16 && src_elem != DFLASH_ELEM_F16)
    return DFLASH_ERR_INVALID_ARG;
  if ((rope_cos == nullptr) != (rope_sin == nullptr) || (rope_cos != nullptr && rope_rows < 1))
    return DFLASH_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || (q != nullptr && n_q_heads < 1)) return DFLASH_ERR_INVALID_ARG;
  if (seq == nullptr && B > kv->n_seqs) return DFLASH_ERR_INVALID_ARG;
  const int dh = kv->head_dim, Hq = q != nullptr ? n_q_heads : 0;
  if (Hq > INT32_MAX / 2 / dh) return DFLASH_ERR_INVALID_ARG;
  const long long kvd = static_cast<long long>(kv->n_kv_heads) * dh;
  // (one token needs no stride between tokens)
  if (static_cast<long long>(B) * T > 1 &&
      (ld_k < kvd || ld_v < kvd || (q != nullptr && ld_q < static_cast<long long>(Hq) * dh)))
    return DFLASH_ERR_INVALID_ARG;
  if (dh != 32 && dh != 64 && dh != 128) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  const auto addr = [](const void* a) { return reinterpret_cast<uintptr_t>(a); };
  if (addr(rope_cos) % 16 || addr(rope_sin) % 16 || addr(q_out) % 16) return DFLASH_ERR_INVALID_ARG;
  const int size = src_elem == DFLASH_ELEM_F32 ? 4 : 2;
  if (addr(k) % size || addr(v) % size || addr(q) % size) return DFLASH_ERR_INVALID_ARG;
  AppendParams p{};
  p.k = k;
  p.v = v;
  p.q = q;
  p.ld_k = ld_k;
  p.ld_v = ld_v;
  p.ld_q = ld_q;
  p.pool_k = kv->k;
  p.pool_v = kv->v;
  p.q_out = q_out;
  p.n_rows = n_rows;
  p.seq = seq;
  p.pos_base = pos_base;
  p.page_table = kv->page_table;
  p.seq_len = kv->seq_len;
  p.rope_cos = rope_cos;
  p.rope_sin = rope_sin;
  p.rope_rows = rope_rows;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = kv->n_kv_heads;
  p.n_pages = kv->n_pages;
  p.n_seqs = kv->n_seqs;
  p.max_pages = kv->max_pages;
  p.vec_k = addr(k) % 16 == 0 && ld_k * size % 16 == 0;
  p.vec_v = addr(v) % 16 == 0 && ld_v * size % 16 == 0;
  p.vec_q = addr(q) % 16 == 0 && ld_q * size % 16 == 0;
  p.status = status;
  const unsigned long long threads =
      static_cast<unsigned long long>(B) * T * (Hq + 2ull * kv->n_kv_heads) * (dh / 16);
  const unsigned long long blocks = (threads + kAppendThreads - 1) / kAppendThreads;
  if (static_cast<long long>(B) * T > INT32_MAX || blocks > INT32_MAX) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  cudaError_t e;
  if (src_elem == DFLASH_ELEM_F32)
    e = launch_append_s<float>(p, kv->elem, dh, static_cast<unsigned>(blocks), stream);
  else if (src_elem == DFLASH_ELEM_BF16)
    e = launch_append_s<__nv_bfloat16>(p, kv->elem, dh, static_cast<unsigned>(blocks), stream);
  else
    e = launch_append_s<__half>(p, kv->elem, dh, static_cast<unsigned>(blocks), stream);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
