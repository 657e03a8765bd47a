// dflash_verify_tokens: which of a sequence's drafted tokens stand against the
// target's probabilities, and the token that follows them, from random numbers
// of the caller.
//
// Draft x_i stays while u_i q_i[x_i] < p_i[x_i].  At the first that does not, the
// next token comes from the weights max(p_i - q_i, 0), after all of them from
// the target's next row: the smallest index whose cumulated weight exceeds
// u * total.
//
// Only one row of p and q a sequence is read whole, so the work is bound by
// memory (128 rows of 201,088, fp32: 36.4 us, of which 12 before and after; one row of
// 151,936: 11.0 us, latencies).  A cluster of CTAs shares a row: units of 512 entries, a warp each,
// whose sums stay in shared memory; the CTA whose part holds u * total goes
// down to the unit and reads that one again.
//
// A unit's sum is a whole number of steps of 2^-38 of its largest weight m: added to
// s >= 32 m, a weight is rounded to s's last place and what that loses is exact
// (s' - s and x less it), so that the first parts add up in s's mantissa and the
// second in a small remainder.  Both are joined over lanes as integers, by one
// instruction each, and over units in double by one warp.  (Pairs of fp32 with
// an error-free sum for every weight took 20 instructions a pair of entries
// against 11, 47 us a batch of 128 rows against 42.4 then; doubles in every warp, 16 cycles of the SM for
// each instruction, 60.)  The order of additions is fixed.
#include <algorithm>

#include "decode_common.cuh"
#include "internal.h"

namespace dflash {

namespace {

constexpr int kVerifyLeast = 128, kVerifyWide = 512;  // threads a CTA
constexpr int kUnit = 512;              // entries of a unit: 16 a lane
constexpr int kVerifyMaxV = 1 << 22;
constexpr int kVerifyCluster = 8;

struct VerifyParams {
  const int32_t *tokens, *n_draft;
  const void *target, *draft;
  long long ld_t, ld_d;
  const float *u_accept, *u_sample;
  int32_t *out, *n_out;
  int* status;
  int K, V, units;
};

// A unit's sum: (hi 2^20 + lo) 2^(exp - 20).
struct UnitSum {
  int hi, lo, exp;
};
__device__ __forceinline__ double value_of(const UnitSum& s) {
  return static_cast<double>(static_cast<long long>(s.hi) * (1 << 20) + s.lo) * __hiloint2double((s.exp - 20 + 1023) << 20, 0);
}
// Weights are told apart down to about 2^-118 (and those of a unit below 2^-38 of its largest not at all).
constexpr uint32_t kLeastTop = (127u - 80u) << 23, kMostTop = (127u + 100u) << 23;

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    T t[4];
    memcpy(t, &v, 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = to_f32<T>(t[i]);
  }
}

// Entry l * 4 + e of each 128 of a unit: whole units of aligned rows come as vectors.
template <typename T>
__device__ __forceinline__ void load_unit(const T* row, int at, int V, int lane, float (&x)[16]) {
  if (at + kUnit <= V && reinterpret_cast<uintptr_t>(row) % (4 * sizeof(T)) == 0) {
    float v[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) load4<T>(row + at + j * 128 + lane * 4, v[j]);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = v[i / 4][i % 4];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = at + (i / 4) * 128 + lane * 4 + i % 4;
      x[i] = k < V ? to_f32<T>(row[k]) : 0.f;
    }
  }
}

// What is drawn from: p alone, p without one entry, or what p has over q.
enum Weights { kRow, kWithout, kResidual };

__device__ __forceinline__ bool weight_ok(float x) { return x >= 0.f && x <= 0x1p100f; }
__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }

template <typename P, typename Q>
__global__ void __launch_bounds__(kVerifyWide, 2) k_verify(const VerifyParams p) {
  extern __shared__ UnitSum sums[];  // of this CTA's units
  __shared__ double s_total;
  __shared__ int s_kept, s_bad, s_n, s_tok, s_next;
  const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int b = blockIdx.x / C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const P* const target = static_cast<const P*>(p.target) + static_cast<long long>(b) * (p.K + 1) * p.ld_t;
  const Q* const draft = p.draft != nullptr ? static_cast<const Q*>(p.draft) + static_cast<long long>(b) * p.K * p.ld_d : nullptr;
  const int32_t* const tok = p.tokens + static_cast<long long>(b) * p.K;

  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    // (tokens and random numbers come beside the count, whatever it is)
    int x = lane < p.K ? tok[lane] : 0;
    float u = lane < p.K ? p.u_accept[static_cast<long long>(b) * p.K + lane] : 0.f;
    const int n = p.n_draft != nullptr ? p.n_draft[b] : p.K;
    int kept = 0, bad = n < 0 || n > p.K ? ST_BAD_ROWS : 0, hit = -1;
    if (bad == 0) {
      kept = n;
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        int flag = 0, stop = 0;
        if (i < n) {
          if (i0 > 0) {
            x = tok[i];
            u = p.u_accept[static_cast<long long>(b) * p.K + i];
          }
          if (x < 0 || x >= p.V) flag = ST_BAD_TOKEN;
          if (!(u >= 0.f && u < 1.f)) flag |= ST_BAD_PROB;
          if (flag == 0) {
            const float pt = to_f32<P>(target[i * p.ld_t + x]), qt = draft != nullptr ? to_f32<Q>(draft[i * p.ld_d + x]) : 1.f;
            if (!weight_ok(pt) || !weight_ok(qt)) flag = ST_BAD_PROB;
            // (24 and 24 bits: the product is exact)
            stop = !(static_cast<double>(u) * qt < pt);
          }
        }
        const unsigned ends = __ballot_sync(0xffffffffu, flag != 0 || stop != 0);
        if (ends != 0) {
          const int at = __ffs(ends) - 1;
          bad = __shfl_sync(0xffffffffu, flag, at);
          hit = __shfl_sync(0xffffffffu, x, at);
          kept = i0 + at;
          break;
        }
      }
    }
    if (bad == 0) {
      const float u = p.u_sample[b];
      if (!(u >= 0.f && u < 1.f)) bad = ST_BAD_PROB;
    }
    if (lane == 0) {
      s_kept = kept;
      s_bad = bad;
      s_n = n;
      s_tok = hit;
    }
  }
  __syncthreads();
  const int kept = s_kept, without = s_tok;
  int bad = s_bad;
  const P* const row = target + kept * p.ld_t;
  const bool over = bad == 0 && kept < s_n;
  const Q* const qrow = over && draft != nullptr ? draft + kept * p.ld_d : nullptr;
  int mode = !over ? kRow : qrow != nullptr ? kResidual : kWithout;
  const int u0 = static_cast<int>(static_cast<long long>(p.units) * rank / C);
  const int u1 = static_cast<int>(static_cast<long long>(p.units) * (rank + 1) / C);
  int found = -1;
  // (a second time only where the residual weighs nothing)
  for (int pass = 0; pass < 2 && bad == 0; ++pass) {
    int fault = 0;
    for (int u = u0 + warp; u < u1; u += blockDim.x / 32) {
      float x[16], q[16];
      load_unit<P>(row, u * kUnit, p.V, lane, x);
      if (mode == kResidual) load_unit<Q>(qrow, u * kUnit, p.V, lane, q);
      // as integers, negative numbers and those that are none are above all others
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, bits_of(x[i]));
      if (mode == kResidual) {
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, bits_of(q[i]));
      }
      if (__any_sync(0xffffffffu, top > kMostTop)) {
        bool fine = true;  // (or a negative zero)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          fine = fine && weight_ok(x[i]) && (mode != kResidual || weight_ok(q[i]));
          x[i] = fabsf(x[i]);
          if (mode == kResidual) q[i] = fabsf(q[i]);
        }
        fault |= !fine;
      }
      // the weights in x, and in q what they lost: p - q = d + e exactly where p > q
      if (mode == kResidual) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float d = fmaxf(x[i] - q[i], 0.f), e = (x[i] - d) - q[i];
          x[i] = d;
          q[i] = d > 0.f ? e : 0.f;
        }
      } else if (mode == kWithout) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (u * kUnit + (i / 4) * 128 + lane * 4 + i % 4 == without) x[i] = 0.f;
      }
      // (of the weights that are summed: those of the row may be far larger)
      top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, bits_of(x[i]));
      top = min(__reduce_max_sync(0xffffffffu, top), kMostTop);
      // s0, a power of two of 32 to 64 times the largest
      const uint32_t s0 = (max(top, kLeastTop) & 0x7f800000u) + (6u << 23);
      float s = __uint_as_float(s0), lo = 0.f;
      const auto add = [&](float w) {
        const float t = s + w;
        lo += w - (t - s);
        s = t;
      };
#pragma unroll
      for (int i = 0; i < 16; ++i) add(x[i]);
      if (mode == kResidual) {
#pragma unroll
        for (int i = 0; i < 16; ++i) lo += q[i];
      }
      // s in units of its last place, g = s0 2^-23; the remainder, of at most 8 g, in 2^-20 of that
      const float per_g = __uint_as_float((254u << 23) - s0 + (43u << 23));
      const int hi = __reduce_add_sync(0xffffffffu, static_cast<int>(bits_of(s) - s0));
      const int rest = __reduce_add_sync(0xffffffffu, __float2int_rn(lo * per_g));
      if (lane == 0) sums[u - u0] = UnitSum{hi, rest, static_cast<int>(s0 >> 23) - 127 - 23};
    }
    fault = __syncthreads_or(fault);
    // From here on warp 0.  This CTA's total; lane l has the l-th share of its units.
    const int per = (u1 - u0 + 31) / 32, a0 = min(u1 - u0, lane * per), a1 = min(u1 - u0, a0 + per);
    const auto sum_of = [&](int i) { return value_of(sums[i]); };
    double mine = 0, upto = 0, own = 0;
    if (warp == 0) {
      for (int i = a0; i < a1; ++i) mine += sum_of(i);
      upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      own = __shfl_sync(0xffffffffu, upto, 31);
      if (lane == 0) s_total = fault ? __longlong_as_double(0x7ff8000000000000ll) : own;
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    double before = 0, total = 0;
    if (warp == 0) {
      double v = 0;
      if (lane < C)
        asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(dsmem_map(smem_u32(&s_total), lane)) : "memory");
#pragma unroll
      for (int r = 0; r < kVerifyCluster; ++r) {
        if (r == rank) before = total;
        total += __shfl_sync(0xffffffffu, v, r);
      }
      // 0: drawn; 1: the row itself, once more; 2: no weights
      if (lane == 0) s_next = !(total >= 0.0 && total <= 1.7e308) ? 2 : total > 0.0 ? 0 : mode == kRow ? 2 : 1;
    }
    // every CTA has read the totals before one leaves or writes its own again
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    const int next = s_next;
    if (next == 2) {
      bad = ST_BAD_PROB;
      break;
    }
    if (next == 1) {
      mode = kRow;
      __syncthreads();
      continue;
    }
    if (warp != 0) break;
    const double aim = static_cast<double>(p.u_sample[b]) * total;
    // the first CTA whose sum passes the aim
    if (before <= aim && before + own > aim) {
      // the lane, then its unit
      const unsigned pass_l = __ballot_sync(0xffffffffu, mine > 0 && before + upto > aim);
      const unsigned any_l = __ballot_sync(0xffffffffu, mine > 0);
      const int l = pass_l ? __ffs(pass_l) - 1 : 31 - __clz(any_l);
      int unit = -1;
      double at = before + __shfl_sync(0xffffffffu, upto - mine, l);
      if (lane == l) {
        for (int i = a0; i < a1; ++i) {
          const double v = sum_of(i);
          if (v > 0) {
            unit = i;
            if (at + v > aim) break;
          }
          at += v;
        }
        // (past the last unit by rounding: that unit, from its own start)
        if (unit >= 0 && !(at + sum_of(unit) > aim)) at -= sum_of(unit);
      }
      unit = u0 + __shfl_sync(0xffffffffu, unit, l);
      at = __shfl_sync(0xffffffffu, at, l);
      // its pieces of 16 entries, one a lane, then the entries of one; a piece's sum as a pair of fp32 (an error-free
      // sum and what it loses)
      const auto weight = [&](int k, float& e) {
        e = 0.f;
        if (k >= p.V || (mode == kWithout && k == without)) return 0.f;
        const float x = to_f32<P>(row[k]);
        if (mode != kResidual) return x;
        const float q = to_f32<Q>(qrow[k]), d = x - q;
        if (!(d > 0.f)) return 0.f;
        e = (x - d) - q;
        return d;
      };
      float s = 0.f, lo = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float e;
        const float x = weight(unit * kUnit + lane * 16 + i, e), t = s + x, z = t - s;
        lo += ((s - (t - z)) + (x - z)) + e;
        s = t;
      }
      double v = static_cast<double>(s) + static_cast<double>(lo);
      const auto scan = [&](double v, double& end) {  // the lane up to which, this one's included, v sums past the aim
        double run = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double w = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += w;
        }
        const unsigned past = __ballot_sync(0xffffffffu, v > 0 && at + run > aim), some = __ballot_sync(0xffffffffu, v > 0);
        end = run;
        return past ? __ffs(past) - 1 : 31 - __clz(some);
      };
      double end;
      const int f = scan(v, end);
      at += __shfl_sync(0xffffffffu, end - v, f);
      float e = 0.f;
      const float d = lane < 16 ? weight(unit * kUnit + f * 16 + lane, e) : 0.f;
      v = static_cast<double>(d) + static_cast<double>(e);
      found = unit * kUnit + f * 16 + scan(v, end);
    }
    break;
  }
  // the CTA that found the token writes the entry's row; the first one where there is nothing to say
  if (warp == 0 && (bad != 0 ? rank == 0 : found >= 0)) {
    int32_t* out = p.out + static_cast<long long>(b) * (p.K + 1);
    for (int i = lane; i <= p.K; i += 32) out[i] = bad != 0 ? -1 : i < kept ? tok[i] : i == kept ? found : -1;
    if (lane == 0) {
      p.n_out[b] = bad != 0 ? 0 : kept + 1;
      if (bad != 0 && p.status != nullptr) atomicOr(p.status, bad);
    }
  }
}

}  // namespace

}  // namespace dflash

namespace dflash {

namespace {

template <typename P, typename Q>
cudaError_t launch_verify(const VerifyParams& p, int B, int C, int threads, cudaStream_t s) {
  const int smem = ((p.units + C - 1) / C + 1) * static_cast<int>(sizeof(UnitSum));
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(smem, [](int v) {
    return cudaFuncSetAttribute(k_verify<P, Q>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  return launch_cached(k_verify<P, Q>, static_cast<unsigned>(B) * C, threads, smem, s, C, p);
}

}  // namespace

}  // namespace dflash

using namespace dflash;

extern "C" dflash_status dflash_verify_tokens(const int32_t* tokens, const int32_t* n_draft, const void* target,
                                              int target_elem, long long ld_t, const void* draft, int draft_elem,
                                              long long ld_d, const float* u_accept, const float* u_sample, int B, int K,
                                              int V, int32_t* out, int32_t* n_out, int* status, dflash_stream stream) {
  if (tokens == nullptr || target == nullptr || u_accept == nullptr || u_sample == nullptr || out == nullptr ||
      n_out == nullptr || B < 1 || K < 1 || V < 1)
    return DFLASH_ERR_INVALID_ARG;
  const auto size_of = [](int e) { return e == DFLASH_ELEM_F32 ? 4 : e == DFLASH_ELEM_BF16 || e == DFLASH_ELEM_F16 ? 2 : 0; };
  const int ts = size_of(target_elem), ds = draft != nullptr ? size_of(draft_elem) : 1;
  if (ts == 0 || ds == 0 || ld_t < V || (draft != nullptr && ld_d < V)) return DFLASH_ERR_INVALID_ARG;
  const auto off = [](const void* a, int n) { return reinterpret_cast<uintptr_t>(a) % n != 0; };
  if (off(target, ts) || off(draft, ds) || off(tokens, 4) || off(n_draft, 4) || off(u_accept, 4) || off(u_sample, 4) ||
      off(out, 4) || off(n_out, 4) || off(status, 4))
    return DFLASH_ERR_INVALID_ARG;
  if (V > kVerifyMaxV || B > 1 << 24 || K > 1 << 24) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  // (the last row's offset in bytes stays inside 63 bits)
  const long long rows = static_cast<long long>(B) * (K + 1ll);
  if (ld_t > INT64_MAX / 8 / rows || (draft != nullptr && ld_d > INT64_MAX / 8 / rows)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  // (a cluster's CTAs judge the drafts each by itself, while one of them may already write)
  const Span in[] = {ints(tokens, static_cast<long long>(B) * K), ints(n_draft, B), {u_accept, 4ll * B * K}, {u_sample, 4ll * B},
                     {target, ((rows - 1) * ld_t + V) * ts}, {draft, ((rows - B - 1) * ld_d + V) * ds}},
             outs[] = {ints(out, rows), ints(n_out, B), ints(status, 1)};
  for (const Span& o : outs)
    for (const Span& i : in)
      if (!apart(o, i)) return DFLASH_ERR_INVALID_ARG;
  if (!apart(outs[0], outs[1]) || !apart(outs[0], outs[2]) || !apart(outs[1], outs[2])) return DFLASH_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return DFLASH_ERR_CUDA;
  VerifyParams p{tokens, n_draft, target, draft, ld_t, ld_d, u_accept, u_sample, out, n_out, status, K, V,
                 (V + kUnit - 1) / kUnit};
  // A row's CTAs: as many as run at once (1024 threads a SM) with four units or more each, then their threads, a warp
  // a unit at most.  128 rows of 201,088: 2 CTAs of 512 threads a row 38.1 us, 4 of 256 37.4, 8 of 128 36.5, of 256
  // 41.4; one row, 8 of 256 11.8, of 512 11.0; 37 of 32,003, 8 of 128 9.4, of 256 8.8, of 512 12.9.
  const long long room = 1024ll * sms / B;
  int C = kVerifyCluster, threads = kVerifyWide;
  while (C > 1 && (C * kVerifyLeast > room || p.units < 4 * C)) C /= 2;
  while (threads > kVerifyLeast && (static_cast<long long>(C) * threads > room || threads / 32 > (p.units + C - 1) / C)) threads /= 2;
  const auto pick = [&](auto t, auto q) { return launch_verify<decltype(t), decltype(q)>(p, B, C, threads, stream); };
  const auto with = [&](auto t) {
    if (draft == nullptr) return pick(t, t);
    if (draft_elem == DFLASH_ELEM_F32) return pick(t, float{});
    if (draft_elem == DFLASH_ELEM_BF16) return pick(t, __nv_bfloat16{});
    return pick(t, __half{});
  };
  e = target_elem == DFLASH_ELEM_F32    ? with(float{})
      : target_elem == DFLASH_ELEM_BF16 ? with(__nv_bfloat16{})
                                        : with(__half{});
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
