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

namespace dflash {

namespace {

constexpr int kW4Rows = 16;     // weight rows of a CTA (one MMA's rows)
constexpr int kW4Warps = 8;     // each takes every eighth 32-wide block of k
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
  const uint8_t* W;
  const void* scale;
  const uint8_t* zero;
  const void* X;
  float* out;
  int N, K, group, groups, M;
  int scale_elem;
};

__device__ __forceinline__ float load_scale(const void* s, int elem, long long i) {
  if (elem == DFLASH_ELEM_F32) return static_cast<const float*>(s)[i];
  if (elem == DFLASH_ELEM_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(s)[i]);
  return __half2float(static_cast<const __half*>(s)[i]);
}

// The four A registers of two k-steps from a thread's words of rows r and r + 8.
template <typename X, bool E2M1>
__device__ __forceinline__ uint32_t widen(uint32_t w, int i, uint32_t bias) {
  const uint32_t q = w >> (4 * i);
  if constexpr (E2M1) return Half2<X>::e2m1(q);
  return Half2<X>::sub((q & 0x000F000Fu) | Half2<X>::kMagic, bias);
}

// NB: 8-column blocks of activation rows.
template <typename X, bool E2M1, int NB>
__global__ void __launch_bounds__(kW4Warps * 32) k_gemm_w4(const W4Params p) {
  using H = Half2<X>;
  __shared__ float part[kW4Warps][NB][32][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
  const int n0 = blockIdx.x * kW4Rows;
  const int blocks = p.K / 32;
  const int rows[2] = {min(n0 + gr, p.N - 1), min(n0 + gr + 8, p.N - 1)};
  const uint32_t* w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = reinterpret_cast<const uint32_t*>(p.W + static_cast<long long>(rows[i]) * (p.K / 2)) + t4;
  float acc[NB][4] = {};
  for (int kb = warp; kb < blocks; kb += kW4Warps) {
    const int g = kb * 32 / p.group;
    float sc[2];
    uint32_t bias[2];
    uint32_t word[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long at = static_cast<long long>(rows[i]) * p.groups + g;
      word[i] = w[i][kb * 4];
      sc[i] = load_scale(p.scale, p.scale_elem, at);
      if constexpr (!E2M1) bias[i] = H::bias(p.zero != nullptr ? min(static_cast<int>(p.zero[at]), 128) : 8);
      else bias[i] = 0;
    }
    uint32_t a[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[s][i] = widen<X, E2M1>(word[i], 2 * s, bias[i]);
        a[s][2 + i] = widen<X, E2M1>(word[i], 2 * s + 1, bias[i]);
      }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int m = j * 8 + gr;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (m < p.M)
        x = *reinterpret_cast<const uint4*>(static_cast<const X*>(p.X) + static_cast<long long>(m) * p.K + kb * 32 +
                                            t4 * 8);
      float d[4] = {};
      H::mma(d, a[0], __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632));
      H::mma(d, a[1], __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
      acc[j][0] += sc[0] * d[0];
      acc[j][1] += sc[0] * d[1];
      acc[j][2] += sc[1] * d[2];
      acc[j][3] += sc[1] * d[3];
    }
  }
#pragma unroll
  for (int j = 0; j < NB; ++j)
    *reinterpret_cast<float4*>(part[warp][j][lane]) = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  for (int e = threadIdx.x; e < NB * 128; e += kW4Warps * 32) {
    const int j = e / 128, ln = e / 4 % 32, c = e % 4;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kW4Warps; ++q) v += part[q][j][ln][c];
    const int n = n0 + (ln >> 2) + 8 * (c >> 1), m = j * 8 + 2 * (ln & 3) + (c & 1);
    if (n < p.N && m < p.M) p.out[static_cast<long long>(m) * p.N + n] = v;
  }
}

template <typename X, bool E2M1>
cudaError_t launch_w4(const W4Params& p, cudaStream_t s) {
  const dim3 grid((p.N + kW4Rows - 1) / kW4Rows), block(kW4Warps * 32);
  switch ((p.M + 7) / 8) {
    case 1: k_gemm_w4<X, E2M1, 1><<<grid, block, 0, s>>>(p); break;
    case 2: k_gemm_w4<X, E2M1, 2><<<grid, block, 0, s>>>(p); break;
    case 3: k_gemm_w4<X, E2M1, 3><<<grid, block, 0, s>>>(p); break;
    default: k_gemm_w4<X, E2M1, 4><<<grid, block, 0, s>>>(p); break;
  }
  return cudaGetLastError();
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
  p.W = static_cast<const uint8_t*>(W);
  p.scale = scale;
  p.zero = static_cast<const uint8_t*>(zero);
  p.X = X;
  p.out = out;
  p.N = N;
  p.K = K;
  p.group = group;
  p.groups = (K + group - 1) / group;
  p.M = M;
  p.scale_elem = scale_elem;
  cudaError_t e;
  if (x_elem == DFLASH_ELEM_BF16)
    e = format == DFLASH_W4_E2M1 ? launch_w4<__nv_bfloat16, true>(p, stream) : launch_w4<__nv_bfloat16, false>(p, stream);
  else
    e = format == DFLASH_W4_E2M1 ? launch_w4<__half, true>(p, stream) : launch_w4<__half, false>(p, stream);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
