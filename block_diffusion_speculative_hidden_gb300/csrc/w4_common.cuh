// What the kernels of dflash_gemm_w4 share (gemm_w4.cu: the entry point;
// w4_resident.cuh, w4_stream.cu: the kernels).
#pragma once

#include <algorithm>

#include "decode_common.cuh"
#include "internal.h"
#include "tma_map.h"

namespace dflash {

// A call, its arguments checked.
struct W4Args {
  const void* W;
  const uint8_t* scale;
  const uint8_t* zero;
  const void* x;
  float* out;
  int* status;
  int N, K, groups, M, group;
  int scale_elem, scale_size, x_elem;
  int sms;
};
// w4_int.cu, w4_e2m1.cu (M <= kW4ResidentM), w4_stream.cu.  More activation
// rows leave the resident ones too little of k at a time (24576 x 4096 integer
// codes in groups of 64, resident / streaming: 25 / 33 us for 16 rows, 46 / 42
// for 24, 77 / 48 for 32).
constexpr int kW4ResidentM = 16;
cudaError_t launch_w4_int(const W4Args& a, cudaStream_t s);
cudaError_t launch_w4_e2m1(const W4Args& a, cudaStream_t s);
cudaError_t launch_w4_stream(const W4Args& a, bool e2m1, cudaStream_t s);

namespace {

constexpr int kW4Smem = 232448;

template <typename X>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
  // An 8-bit integer v as a bf16's bits is v 2^-133.  Products by 2^127 make v / 64
  // of it, exactly, and so are the differences code - zero that enter the MMA:
  // in 64ths, which kSum makes up for in the fp32 sum (activations below 2^-120
  // leave its normal range).  128 + v, with v in the mantissa, has no place for
  // zero points above 128, and its additions take longer: 24576 x 4096, one row,
  // groups of 32, 23.2 us against 21.3; 6144 x 4096 in groups of 128, 6.9 and 6.35.
  static constexpr float kSum = 64.f;
  // The zero point in byte g of z, for widen().
  static __device__ __forceinline__ uint32_t bias(uint32_t z, int g) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(__byte_perm(z, 0u, 0x4040 | g << 8 | g)), "r"(0xFF00FF00u));
    return d;
  }
  // Codes i and i + 4 of a word, less the zero point, in a[i].
  static __device__ __forceinline__ void widen(uint32_t w, uint32_t bias, uint32_t (&a)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(a[i]) : "r"((w >> (4 * i)) & 0x000F000Fu), "r"(0x7F007F00u), "r"(bias));
  }
  // an E2M1 code's value: its exponent and mantissa bits in place (an exponent
  // field of 0 .. 3, so the value times 2^-126), the sign at bit 15, and one
  // exact product by 2^126
  static __device__ __forceinline__ uint32_t e2m1(uint32_t c) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(((c & 7u) << 6) | ((c & 8u) << 12)), "r"(0x7E807E80u));
    return d;
  }
  // Two codes of a byte: a product puts them 16 bits apart, and so on as above.
  static __device__ __forceinline__ uint32_t e2m1x2(uint32_t c) {
    const uint32_t t = c * 0x1001u;
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"((t & 0x00070007u) * 64u + (t & 0x00080008u) * 4096u), "r"(0x7E807E80u));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  // d = a b
  static __device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
};
template <>
struct Half2<__half> {
  static constexpr uint32_t kMagic = 0x64006400u;  // kMagic + v is 1024 + v, exact
  static constexpr float kSum = 1.f;
  static __device__ __forceinline__ uint32_t bias(uint32_t z, int g) {
    return __byte_perm(z, kMagic, 0x5050 | g << 8 | g);  // 1024 + the zero point
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // Codes less the zero point; a nibble at bits 4 .. 7 stays there, as 1024 + 16 code, and an
  // exact product by 1/16 takes it down, so that two of the four need no shift.
  static __device__ __forceinline__ void widen(uint32_t w, uint32_t bias, uint32_t (&a)[4]) {
    const uint32_t low = sub(0x63806380u, bias);  // 960 - (1024 + zero) = -(64 + zero)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t v = w >> (4 * i);
      a[i] = sub((v & 0x000F000Fu) | kMagic, bias);
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(a[i + 1]) : "r"((v & 0x00F000F0u) | kMagic), "r"(0x2C002C00u), "r"(low));
    }
  }
  static __device__ __forceinline__ uint32_t e2m1(uint32_t c) {  // (by 2^-14 and 2^14)
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(((c & 7u) << 9) | ((c & 8u) << 12)), "r"(0x74007400u));
    return d;
  }
  static __device__ __forceinline__ uint32_t e2m1x2(uint32_t c) {
    const uint32_t t = c * 0x1001u;
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"((t & 0x00070007u) * 512u + (t & 0x00080008u) * 4096u), "r"(0x74007400u));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  // d = a b
  static __device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
};

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

// BYTES asynchronously, of which n come from src and the rest are zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes, int n) {
  if (bytes == 16) copy_async<16>(dst, src, n);
  else if (bytes == 8) copy_async<8>(dst, src, n);
  else copy_async<4>(dst, src, n);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// N words (1, 2, 4 or 8)
template <int N>
__device__ __forceinline__ void lds(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 8) {
    const uint4 u = lds128(a), v = lds128(a + 16);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
  } else if constexpr (N == 4) {
    const uint4 u = lds128(a);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = lds64(a);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = lds32(a);
  }
}

// E2M1 codes are widened through a table in shared memory: a byte (two codes)
// to its pair of 16-bit values, with a copy for every lane (entry e of lane l
// at 256 e + 4 l, so that one byte permutation makes the address and no two
// lanes share a bank).  Taking the codes apart with shifts and masks costs
// five instructions a pair against the table's two.
constexpr int kW4Table = 65536;  // its bytes, and what its address is a multiple of

// A matrix of `cols` columns of `size` bytes as boxes of box_rows x box_cols.
bool w4_map(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base, long long rows, long long cols,
            int box_rows, int box_cols, CUtensorMapSwizzle swizzle) {
  const auto encode = tensor_map_encoder();
  const cuuint64_t gdim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t pitch[1] = {static_cast<cuuint64_t>(cols) * size};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return encode != nullptr &&
         encode(map, type, 2, const_cast<void*>(base), gdim, pitch, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Bytes of the asynchronous copies that fetch `bytes` adjacent bytes of a row
// of `pitch` bytes at `base`, or 0 where none fits.
int w4_piece(int bytes, long long pitch, const void* base) {
  for (int n = 16; n >= 4; n /= 2)
    if (bytes % n == 0 && pitch % n == 0 && reinterpret_cast<uintptr_t>(base) % n == 0) return n;
  return 0;
}

}  // namespace

}  // namespace dflash
