// dflash_gemm_w4: products of a few activation rows with 4-bit weights under
// group scales,
//     out[m][n] = sum_k X[m][k] scale[n][k/g] (code[n][k] - zero[n][k/g]).
//
// The differences code - zero (and the E2M1 values) are exact in bf16 and
// fp16, so a block of 32 k enters the matrix instruction as it is, with fp32
// sums, and the scale multiplies the block's fp32 sum.  The order of k inside
// a block is free as long as weights and activations agree on it: thread t of
// a quad holds codes 8t .. 8t+7 of the block (one 32-bit word), whose halves
// come out of the word as pairs (k, k+4).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "tma_map.h"

namespace dflash {

namespace {

constexpr int kW4Warps = 8;      // each takes every eighth unit of k
constexpr int kW4Threads = kW4Warps * 32;
constexpr int kW4Unit = 128;     // k of a unit: 64 bytes of a weight row
constexpr int kW4Stages = 4;     // units in flight per warp
constexpr int kW4MaxM = 32;

template <typename X>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static constexpr uint32_t kMagic = 0x43004300u;  // 128 + code, exact
  static __device__ __forceinline__ uint32_t bias(int z) {  // 128 + z in both halves
    const __nv_bfloat162 b = __float2bfloat162_rn(static_cast<float>(128 + z));
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // E2M1: exponent and mantissa bits in place (exponent field 0..3, so the
  // value times 2^-126), the sign at bit 15, and one exact product by 2^126
  static __device__ __forceinline__ uint32_t e2m1(uint32_t q) {
    const uint32_t y = ((q & 0x00070007u) << 6) | ((q & 0x00080008u) << 12);
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(y), "r"(0x7E807E80u));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Half2<__half> {
  using V = __half2;
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024 + code, exact
  static __device__ __forceinline__ uint32_t bias(int z) {
    const __half2 b = __float2half2_rn(static_cast<float>(1024 + z));
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t e2m1(uint32_t q) {  // times 2^-14, as for bf16
    const uint32_t y = ((q & 0x00070007u) << 9) | ((q & 0x00080008u) << 12);
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(y), "r"(0x74007400u));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

struct W4Params {
  const void* scale;
  const uint8_t* zero;
  const void* X;
  float* out;
  int* status;
  int N, K, groups, M;
  int scale_elem;
  bool whole_units;  // scales and zeros of a unit may be read as one vector
};

// The scales of one weight row's NG groups from group g0 on, as fp32 (past the row's last group: 0).
template <int NG>
__device__ __forceinline__ void load_scales(const W4Params& p, long long row, int g0, float (&s)[NG]) {
  const long long at = row * p.groups + g0;
  if (p.scale_elem == DFLASH_ELEM_F32) {
    const float* src = static_cast<const float*>(p.scale) + at;
    if (NG == 4 && p.whole_units) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      s[0] = v.x, s[NG > 1 ? 1 : 0] = v.y, s[NG > 2 ? 2 : 0] = v.z, s[NG > 3 ? 3 : 0] = v.w;
      return;
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) s[j] = g0 + j < p.groups ? src[j] : 0.f;
    return;
  }
  const uint16_t* src = static_cast<const uint16_t*>(p.scale) + at;
  uint32_t h[(NG + 1) / 2];
  if (NG == 4 && p.whole_units) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    h[0] = v.x, h[NG > 2 ? 1 : 0] = v.y;
  } else if (NG == 2 && p.whole_units) {
    h[0] = *reinterpret_cast<const uint32_t*>(src);
  } else {
#pragma unroll
    for (int j = 0; j < NG; j += 2) {
      h[j / 2] = g0 + j < p.groups ? src[j] : 0u;
      if (j + 1 < NG && g0 + j + 1 < p.groups) h[j / 2] |= static_cast<uint32_t>(src[j + 1]) << 16;
    }
  }
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    const uint32_t b = j & 1 ? h[j / 2] >> 16 : h[j / 2] & 0xffffu;
    s[j] = p.scale_elem == DFLASH_ELEM_BF16 ? __uint_as_float(b << 16)
                                            : __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
  }
}

// Their zero points, a byte each (8 where there are none).
template <int NG>
__device__ __forceinline__ uint32_t load_zeros(const W4Params& p, long long row, int g0) {
  if (p.zero == nullptr) return 0x08080808u;
  const uint8_t* src = p.zero + row * p.groups + g0;
  if (NG == 4 && p.whole_units) return *reinterpret_cast<const uint32_t*>(src);
  uint32_t z = 0;
#pragma unroll
  for (int j = 0; j < NG; ++j) z |= g0 + j < p.groups ? static_cast<uint32_t>(src[j]) << (8 * j) : 0u;
  return z;
}

// Codes i and i + 4 of a word as a pair of 16-bit values.
template <typename X, bool E2M1>
__device__ __forceinline__ uint32_t widen(uint32_t w, int i, uint32_t bias) {
  const uint32_t q = w >> (4 * i);
  if constexpr (E2M1) return Half2<X>::e2m1(q);
  return Half2<X>::sub((q & 0x000F000Fu) | Half2<X>::kMagic, bias);
}

// mbar_wait (common.cuh) where no status word need be given.
__device__ __forceinline__ bool w4_wait(uint64_t* bar, uint32_t parity, int* status) {
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

template <int TILES, int NB>
struct W4Layout {
  static constexpr int ROWS = 16 * TILES;
  static constexpr int UNIT = ROWS * (kW4Unit / 2);   // bytes of a unit's codes
  static constexpr int WARP = kW4Stages * UNIT;       // a warp's ring; then its partial sums
  static constexpr int PART = ROWS * NB * 8 * 4;
  static constexpr int OFF_BAR = kW4Warps * (WARP > PART ? WARP : PART);
  static constexpr int STRIDE = WARP > PART ? WARP : PART;
  static constexpr int SMEM = 1024 + OFF_BAR + kW4Warps * kW4Stages * 8;
};

// One CTA: 16 * TILES weight rows.  Every warp streams units of its own (128
// k of all the CTA's rows) through a ring of TMA copies, keeps the unit's
// activations in registers over the row tiles, and adds up its units; the
// CTA joins the warps' sums in order at the end.  NB: blocks of 8 activation
// rows (the MMA's N).
//
// Within a group a thread of a quad takes 8 * GROUP / 32 adjacent codes (one
// 4, 8 or 16-byte read), so an MMA adds products of one group only.
template <typename X, bool E2M1, int GROUP, int TILES, int NB>
__global__ void __launch_bounds__(kW4Threads, NB == 1 ? 3 : NB == 2 ? 2 : 1)
    k_gemm_w4(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ W4Params p) {
  using H = Half2<X>;
  using L = W4Layout<TILES, NB>;
  constexpr int NG = kW4Unit / GROUP;  // groups of a unit
  constexpr int WPT = GROUP / 32;      // words a thread takes of a group
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
  const int n0 = blockIdx.x * L::ROWS;
  const int units = (p.K + kW4Unit - 1) / kW4Unit;
  const int mine = units > warp ? (units - warp + kW4Warps - 1) / kW4Warps : 0;
  uint8_t* ring = smem + warp * L::STRIDE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR) + warp * kW4Stages;
  auto issue = [&](int i) {  // (one thread)
    const int s = i % kW4Stages;
    mbar_arrive_expect_tx(&bars[s], L::UNIT);
    tma_load_2d(ring + s * L::UNIT, &tmW, &bars[s], (warp + i * kW4Warps) * (kW4Unit / 2), n0);
  };
  if (lane == 0) {
    for (int s = 0; s < kW4Stages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    for (int i = 0; i < min(mine, kW4Stages); ++i) issue(i);
  }
  __syncwarp();

  float acc[TILES][NB][4] = {};
  bool ok = true;
  for (int i = 0; i < mine; ++i) {
    const int s = i % kW4Stages, k0 = (warp + i * kW4Warps) * kW4Unit;
    // the unit's activations as B fragments, its scales and zero points
    uint4 x[NB][NG * WPT];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int w = 0; w < NG * WPT; ++w) {
        const int m = j * 8 + gr, k = k0 + w / WPT * GROUP + (t4 * WPT + w % WPT) * 8;
        x[j][w] = m < p.M && k < p.K
                      ? *reinterpret_cast<const uint4*>(static_cast<const X*>(p.X) + static_cast<long long>(m) * p.K + k)
                      : make_uint4(0, 0, 0, 0);
      }
    float sc[TILES][2][NG];
    uint32_t zr[TILES][2];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = min(n0 + t * 16 + h * 8 + gr, p.N - 1);
        load_scales<NG>(p, row, k0 / GROUP, sc[t][h]);
        zr[t][h] = E2M1 ? 0u : load_zeros<NG>(p, row, k0 / GROUP);
      }
    ok = ok && w4_wait(&bars[s], (i / kW4Stages) & 1, p.status);
    if (!__all_sync(0xffffffffu, ok)) break;
    const uint8_t* tile = ring + s * L::UNIT;
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t word[2][WPT], bias[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = t * 16 + h * 8 + gr, byte = g * (GROUP / 2) + t4 * WPT * 4;
          // (rows of 64 bytes, 16-byte pieces swizzled by the row's bits 1 and 2)
          const uint8_t* src = tile + r * 64 + (byte ^ ((r >> 1 & 3) << 4));
          if constexpr (WPT == 4) *reinterpret_cast<uint4*>(word[h]) = *reinterpret_cast<const uint4*>(src);
          else if constexpr (WPT == 2) *reinterpret_cast<uint2*>(word[h]) = *reinterpret_cast<const uint2*>(src);
          else word[h][0] = *reinterpret_cast<const uint32_t*>(src);
          bias[h] = E2M1 ? 0u : H::bias(min(static_cast<int>(zr[t][h] >> (8 * g) & 0xffu), 128));
        }
        float d[NB][4] = {};
#pragma unroll
        for (int w = 0; w < WPT; ++w) {
          uint32_t a[2][4];
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              a[q][h] = widen<X, E2M1>(word[h][w], 2 * q, bias[h]);
              a[q][2 + h] = widen<X, E2M1>(word[h][w], 2 * q + 1, bias[h]);
            }
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const uint4& v = x[j][g * WPT + w];
            H::mma(d[j], a[0], __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
            H::mma(d[j], a[1], __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
          }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][j][e] += sc[t][e >> 1][g] * d[j][e];
      }
    __syncwarp();
    if (lane == 0 && i + kW4Stages < mine) issue(i + kW4Stages);
  }
  if (!ok) {  // a wait gave up: copies still in flight get bounded waits of their own
    for (int s = 0; s < min(mine, kW4Stages); ++s) w4_wait(&bars[s], 0, p.status);
  }
  __syncwarp();
  float* part = reinterpret_cast<float*>(ring);  // [ROWS][NB * 8]
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(part + (t * 16 + h * 8 + gr) * (NB * 8) + j * 8 + 2 * t4) =
            make_float2(acc[t][j][2 * h], acc[t][j][2 * h + 1]);
  __syncthreads();
  for (int e = threadIdx.x; e < L::ROWS * NB * 8; e += kW4Threads) {
    const int r = e % L::ROWS, m = e / L::ROWS;
    if (n0 + r >= p.N || m >= p.M) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kW4Warps; ++w) v += reinterpret_cast<const float*>(smem + w * L::STRIDE)[r * (NB * 8) + m];
    p.out[static_cast<long long>(m) * p.N + n0 + r] = v;
  }
}

template <typename X, bool E2M1, int GROUP, int TILES, int NB>
cudaError_t launch_w4_t(const W4Params& p, const void* W, cudaStream_t s) {
  using L = W4Layout<TILES, NB>;
  // W as bytes [N][K / 2] in boxes of a unit (64 bytes) x the CTA's rows
  const auto encode = tensor_map_encoder();
  CUtensorMap map;
  const cuuint64_t gdim[2] = {static_cast<cuuint64_t>(p.K / 2), static_cast<cuuint64_t>(p.N)};
  const cuuint64_t pitch[1] = {static_cast<cuuint64_t>(p.K / 2)};
  const cuuint32_t box[2] = {kW4Unit / 2, L::ROWS}, es[2] = {1, 1};
  if (encode == nullptr ||
      encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(W), gdim, pitch, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(L::SMEM, [](int v) {
    return cudaFuncSetAttribute(k_gemm_w4<X, E2M1, GROUP, TILES, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  return launch_k(k_gemm_w4<X, E2M1, GROUP, TILES, NB>, dim3((p.N + L::ROWS - 1) / L::ROWS), dim3(kW4Threads), L::SMEM,
                  s, dim3(1), false, map, p);
}

// 32 weight rows a CTA where that still gives every SM about two CTAs, else 16.
template <typename X, bool E2M1, int GROUP, int NB>
cudaError_t launch_w4_n(const W4Params& p, const void* W, cudaStream_t s) {
  return p.N >= 2 * 32 * 152 ? launch_w4_t<X, E2M1, GROUP, 2, NB>(p, W, s)
                             : launch_w4_t<X, E2M1, GROUP, 1, NB>(p, W, s);
}

template <typename X, bool E2M1, int GROUP>
cudaError_t launch_w4_g(const W4Params& p, const void* W, cudaStream_t s) {
  switch ((p.M + 7) / 8) {
    case 1: return launch_w4_n<X, E2M1, GROUP, 1>(p, W, s);
    case 2: return launch_w4_n<X, E2M1, GROUP, 2>(p, W, s);
    case 3: return launch_w4_n<X, E2M1, GROUP, 3>(p, W, s);
    default: return launch_w4_n<X, E2M1, GROUP, 4>(p, W, s);
  }
}

template <typename X, bool E2M1>
cudaError_t launch_w4(const W4Params& p, const void* W, int group, cudaStream_t s) {
  if (group == 32) return launch_w4_g<X, E2M1, 32>(p, W, s);
  if (group == 64) return launch_w4_g<X, E2M1, 64>(p, W, s);
  return launch_w4_g<X, E2M1, 128>(p, W, s);
}

}  // namespace

}  // namespace dflash

using namespace dflash;

extern "C" dflash_status dflash_gemm_w4(const void* W, int format, const void* scale, int scale_elem, const void* zero,
                                        int N, int K, int group, const void* X, int x_elem, int M, float* out,
                                        int* status, dflash_stream stream) {
  if (W == nullptr || scale == nullptr || X == nullptr || out == nullptr || N < 1 || K < 1 || M < 1)
    return DFLASH_ERR_INVALID_ARG;
  if (format != DFLASH_W4_INT && (format != DFLASH_W4_E2M1 || zero != nullptr)) return DFLASH_ERR_INVALID_ARG;
  if (x_elem != DFLASH_ELEM_BF16 && x_elem != DFLASH_ELEM_F16) return DFLASH_ERR_INVALID_ARG;
  const int ss = scale_elem == DFLASH_ELEM_F32 ? 4 : 2;
  if (scale_elem != DFLASH_ELEM_F32 && scale_elem != DFLASH_ELEM_BF16 && scale_elem != DFLASH_ELEM_F16)
    return DFLASH_ERR_INVALID_ARG;
  if (M > kW4MaxM || K % 32 || (group != 32 && group != 64 && group != 128)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (reinterpret_cast<uintptr_t>(W) % 16 || reinterpret_cast<uintptr_t>(X) % 16 ||
      reinterpret_cast<uintptr_t>(scale) % ss || reinterpret_cast<uintptr_t>(out) % 4)
    return DFLASH_ERR_INVALID_ARG;
  W4Params p;
  p.scale = scale;
  p.zero = static_cast<const uint8_t*>(zero);
  p.X = X;
  p.out = out;
  p.status = status;
  p.N = N;
  p.K = K;
  p.groups = (K + group - 1) / group;
  p.M = M;
  p.scale_elem = scale_elem;
  p.whole_units = K % kW4Unit == 0 && reinterpret_cast<uintptr_t>(scale) % 16 == 0 &&
                  reinterpret_cast<uintptr_t>(zero) % 4 == 0;
  cudaError_t e;
  if (x_elem == DFLASH_ELEM_BF16)
    e = format == DFLASH_W4_E2M1 ? launch_w4<__nv_bfloat16, true>(p, W, group, stream)
                                 : launch_w4<__nv_bfloat16, false>(p, W, group, stream);
  else
    e = format == DFLASH_W4_E2M1 ? launch_w4<__half, true>(p, W, group, stream)
                                 : launch_w4<__half, false>(p, W, group, stream);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
