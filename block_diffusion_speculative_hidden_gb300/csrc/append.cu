// dflash_append_kv, dflash_extend and dflash_rope_table: keys and values that
// the caller has in hand into a paged cache, with the position rotation of
// the keys (and of the step's queries) applied on the way.
//
// A row (batch entry b, token i) stands at slot seq_len - n + i of its
// sequence; key and query elements x_i and x_{i+h} (h = head_dim / 2) rotate
// as a pair by the table's angle of the row's position.
#include "decode_common.cuh"
#include "kernels.cuh"

namespace dflash {

namespace {

// Eight elements of a row as they are stored.  VEC: the address is 16-byte
// aligned and they come as 128-bit loads, which stay where they are written:
// before the waits for what decides where the row goes.
template <typename T, bool VEC>
struct Raw8 {
  static constexpr int W = 16 / sizeof(T);  // elements per 128-bit access
  union {
    uint4 u[8 / W];
    T t[8];
  };
  __device__ __forceinline__ Raw8() {}
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < 8 / W; ++j)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u[j].x), "=r"(u[j].y), "=r"(u[j].z), "=r"(u[j].w)
                     : "l"(p + j * W));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = p[k];
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = to_f32<T>(t[k]);
  }
};

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
  int* status;
};

constexpr int kAppendThreads = 128;
constexpr int kAppendHeads = 2;  // (1: 9.2 us for verified blocks, 2: 8.3, 4: 9.6, for their registers)

// Bound by memory: every byte is read and written once (128 blocks of up to 17
// rows, 64 query and 8 kv heads of 64 from fp32 to fp16: 8.1 us, 4.4 TB/s, of
// which 2.5 us are a launch; 8 prompts of up to 4096 rows, 8 kv heads of 128:
// 33.5 us, 5.5 TB/s).
//
// DH / 16 threads take kAppendHeads heads of one row, each eight elements of
// the heads' first halves and the eight that they rotate with: the angles are
// read once for those heads, and their elements are on the way while the
// thread finds the row's slot.
template <typename S, typename D, int DH, bool VEC>
__global__ void __launch_bounds__(kAppendThreads) k_append(const AppendParams p) {
  constexpr int TPU = DH / 16, HALF = DH / 2;
  const int heads = p.Hq + 2 * p.Hkv, units = (heads + kAppendHeads - 1) / kAppendHeads;
  const long long u = (static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x) / TPU;
  const int d = (threadIdx.x % TPU) * 8;
  const long long row = u / units;
  if (row >= static_cast<long long>(p.B) * p.T) return;
  const int h0 = static_cast<int>(u - row * units) * kAppendHeads;
  const int b = static_cast<int>(row / p.T), i = static_cast<int>(row - static_cast<long long>(b) * p.T);
  const bool first = h0 == 0 && d == 0;  // the thread that reports
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
  Raw8<S, VEC> raw[kAppendHeads][2];
#pragma unroll
  for (int j = 0; j < kAppendHeads; ++j) {
    const int h = min(h0 + j, heads - 1), hk = h - p.Hq;
    const S* src = hk < 0        ? static_cast<const S*>(p.q) + row * p.ld_q + h * DH
                   : hk < p.Hkv ? static_cast<const S*>(p.k) + row * p.ld_k + hk * DH
                                : static_cast<const S*>(p.v) + row * p.ld_v + (hk - p.Hkv) * DH;
    raw[j][0].load(src + d);
    raw[j][1].load(src + HALF + d);
  }
  if (len < n) return flag(ST_BAD_ROWS);
  if (len > p.max_pages * kPage) return flag(ST_SEQ_TOO_LONG);
  const int slot = len - n + i;
  const bool rope = p.rope_cos != nullptr;
  const int page = p.page_table[static_cast<long long>(s) * p.max_pages + slot / kPage];
  const long long pos = static_cast<long long>(slot) + (p.pos_base != nullptr ? p.pos_base[b] : 0);
  const bool far = rope && (pos < 0 || pos >= p.rope_rows);
  float c[8] = {}, sn[8] = {};
  if (rope && !far && h0 < p.Hq + p.Hkv) {
    const float4 *pc = reinterpret_cast<const float4*>(p.rope_cos + pos * HALF + d),
                 *ps = reinterpret_cast<const float4*>(p.rope_sin + pos * HALF + d);
    *reinterpret_cast<float4*>(c) = pc[0];
    *reinterpret_cast<float4*>(c + 4) = pc[1];
    *reinterpret_cast<float4*>(sn) = ps[0];
    *reinterpret_cast<float4*>(sn + 4) = ps[1];
  }
  if (page < 0 || page >= p.n_pages) return flag(ST_BAD_PAGE);
  if (far) return flag(ST_BAD_POS);
#pragma unroll
  for (int j = 0; j < kAppendHeads; ++j) {
    const int h = h0 + j, hk = h - p.Hq;
    if (h >= heads) break;
    const bool is_v = hk >= p.Hkv;
    float x1[8], x2[8];
    raw[j][0].get(x1);
    raw[j][1].get(x2);
    if (rope && !is_v) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float a = x1[k], e = x2[k];
        x1[k] = a * c[k] - e * sn[k];
        x2[k] = e * c[k] + a * sn[k];
      }
    }
    D* dst = hk < 0 ? static_cast<D*>(p.q_out) + (row * p.Hq + h) * DH
                    : static_cast<D*>(is_v ? p.pool_v : p.pool_k) +
                          ((static_cast<long long>(page) * p.Hkv + (is_v ? hk - p.Hkv : hk)) * kPage + slot % kPage) * DH;
    store8<D>(dst + d, x1);
    store8<D>(dst + HALF + d, x2);
  }
}

template <typename S, typename D, bool VEC>
cudaError_t launch_append_t(const AppendParams& p, int dh, cudaStream_t s) {
  const long long units = (p.Hq + 2ll * p.Hkv + kAppendHeads - 1) / kAppendHeads;
  const long long threads = static_cast<long long>(p.B) * p.T * units * (dh / 16);
  const unsigned n = static_cast<unsigned>((threads + kAppendThreads - 1) / kAppendThreads);
  switch (dh) {
    case 32: k_append<S, D, 32, VEC><<<n, kAppendThreads, 0, s>>>(p); break;
    case 64: k_append<S, D, 64, VEC><<<n, kAppendThreads, 0, s>>>(p); break;
    default: k_append<S, D, 128, VEC><<<n, kAppendThreads, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

template <typename S, bool VEC>
cudaError_t launch_append_s(const AppendParams& p, int elem, int dh, cudaStream_t s) {
  if (elem == DFLASH_ELEM_F32) return launch_append_t<S, float, VEC>(p, dh, s);
  if (elem == DFLASH_ELEM_BF16) return launch_append_t<S, __nv_bfloat16, VEC>(p, dh, s);
  return launch_append_t<S, __half, VEC>(p, dh, s);
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
  p.status = status;
  if (static_cast<long long>(B) * T > INT32_MAX ||
      static_cast<unsigned long long>(B) * T * (Hq + 2ull * kv->n_kv_heads) * (dh / 16) / kAppendThreads > INT32_MAX)
    return DFLASH_ERR_UNSUPPORTED_SHAPE;
  const auto aligned = [&](const void* a, long long ld) { return addr(a) % 16 == 0 && ld * size % 16 == 0; };
  const bool vec = aligned(k, ld_k) && aligned(v, ld_v) && (q == nullptr || aligned(q, ld_q));
  const auto run = [&](auto t) {
    using S = decltype(t);
    return vec ? launch_append_s<S, true>(p, kv->elem, dh, stream) : launch_append_s<S, false>(p, kv->elem, dh, stream);
  };
  const cudaError_t e = src_elem == DFLASH_ELEM_F32    ? run(float{})
                        : src_elem == DFLASH_ELEM_BF16 ? run(__nv_bfloat16{})
                                                       : run(__half{});
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
