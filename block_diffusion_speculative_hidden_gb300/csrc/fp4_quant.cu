// dflash_quantize_fp4, dflash_dequantize_fp4, dflash_fp4_tile_scales: rows of
// numbers to microscaled 4-bit floats and back.
//
// A group of 32 (MX) or 16 (NV) neighbours shares one step s: for MX the power
// of two 2^(floor(log2 max|x|) - 2), for NV an E4M3 number times the tensor's
// own fp32 scale g, s = e4m3(max|x| / 6g) g.  The code of an element is the
// E2M1 number nearest to |x| / s, ties to even, at most 6.
//
// Every border is decided as in real arithmetic, so that the codes are the
// same whoever computes them.  MX: s is a power of two and x / s is exact.  NV:
// a border m (an E2M1 or E4M3 midpoint) holds at x = m s, and the sign of
// fma(-m, s, x) is exact wherever the factor beside g has few bits; quotients in fp32 only
// propose the code.  16-bit inputs have few significant bits, so that a step has at most four numbers
// (and their powers of two) whose side of a border a quotient may miss: it is moved a little to the exact
// sides once for the step (with g = max|x| / 2688 half of all steps have such a number: 55.9 us where these groups'
// elements were looked at twice, 43.2).  In fp32, and where both sides are wanted, quotients that
// may lie within 2^-19 of a border are decided by the exact signs, element by element.
//
// Each element is read once, half a byte and its share of a scale are written.
// Both are bound by memory (8192 rows of 12,288 fp16, NV: 43.2 us, 6.0 TB/s; taking back 38.7 us, 6.7 TB/s).
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "fp4_common.cuh"

namespace dflash {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kPiece = 16;  // elements a thread: one NV group, half an MX group

// E2M1 codes of eight numbers, nearest, ties to even, at most 6.
__device__ __forceinline__ uint32_t e2m1x8(const float2 (&v)[4]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(w)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return w;
}

// Sixteen elements, as they are stored.
template <typename T>
struct Sixteen {
  union {
    uint4 u[kPiece * sizeof(T) / 16];
    uint32_t w[kPiece * sizeof(T) / 4];
    T t[kPiece];
  };
  __device__ __forceinline__ Sixteen() {}
  template <bool VEC>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
      // (32 bytes at a time: a lane's 16-byte halves of a sector would fetch it twice, 75 us against 45)
#pragma unroll
      for (int j = 0; j < static_cast<int>(kPiece * sizeof(T) / 4); j += 8)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[j]), "=r"(w[j + 1]), "=r"(w[j + 2]), "=r"(w[j + 3]), "=r"(w[j + 4]), "=r"(w[j + 5]),
                       "=r"(w[j + 6]), "=r"(w[j + 7])
                     : "l"(reinterpret_cast<const uint32_t*>(p) + j));
    } else {
#pragma unroll
      for (int k = 0; k < kPiece; ++k) t[k] = p[k];
    }
  }
  __device__ __forceinline__ float get(int k) const { return to_f32<T>(t[k]); }
  // x times f, eight from 8 h on, as codes.
  __device__ __forceinline__ uint32_t codes(int h, float f) const {
    float2 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = __fmul2_rn(make_float2(get(8 * h + 2 * k), get(8 * h + 2 * k + 1)), make_float2(f, f));
    return e2m1x8(v);
  }
  // x / sg, rounded to nearest, as codes; inv = 1 / sg, rounded to nearest: one step from x inv with the exact rest
  // (its negative, so that -0 stays -0).
  __device__ __forceinline__ uint32_t codes_of_quotients(int h, float inv, float sg) const {
    float2 v[4];
    const float2 i2 = make_float2(inv, inv), back = make_float2(-inv, -inv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 y = make_float2(get(8 * h + 2 * k), get(8 * h + 2 * k + 1)), q = __fmul2_rn(y, i2);
      v[k] = __ffma2_rn(__ffma2_rn(q, make_float2(sg, sg), make_float2(-y.x, -y.y)), back, q);
    }
    return e2m1x8(v);
  }
  // Bits (as fp32) of the largest magnitude; a NaN's are above infinity's.
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < kPiece; ++k) m = max(m, w[k] & 0x7fffffffu);
      return m;
    } else {
      using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
      T2 m;
      memcpy(&m, &w[0], 4);
      m = __habs2(m);
#pragma unroll
      for (int k = 1; k < kPiece / 2; ++k) {
        T2 v;
        memcpy(&v, &w[k], 4);
        m = __hmax2_nan(m, __habs2(v));
      }
      const uint32_t a = __float_as_uint(to_f32<T>(m.x)), b = __float_as_uint(to_f32<T>(m.y));
      return max(a & 0x7fffffffu, b & 0x7fffffffu);
    }
  }
};

// n / d for 32-bit n: d's rounded-up reciprocal from the host (a division takes as long as the rest of a piece's
// arithmetic).
struct Divisor {
  unsigned d, mul, shift;
  explicit Divisor(unsigned n) : d(n), mul(0), shift(0) {
    while (shift < 32 && (1ull << shift) < n) ++shift;
    mul = static_cast<unsigned>(((1ull << 32) * ((1ull << shift) - n)) / n + 1);
  }
  __device__ __forceinline__ unsigned divide(unsigned n) const {
    const unsigned t = __umulhi(n, mul);
    return static_cast<unsigned>((static_cast<unsigned long long>(t) + n) >> shift);
  }
};

// The value of E4M3 code c (0 .. 126, not negative).
__device__ __forceinline__ float e4m3_value(int c) {
  return c < 8 ? static_cast<float>(c) * 0x1p-9f : __int_as_float((((c >> 3) + 120) << 23) | ((c & 7) << 20));
}

// E2M1 code (without its sign) of a = |x| under the step s * g: the borders
// m s g one by one, their signs exact.
__device__ __noinline__ uint32_t e2m1_exact(float a, float s, float g) {
  constexpr float mid[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.f};
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const float d = fmaf(-(mid[i] * s), g, a);
    code += (i & 1) ? d >= 0.f : d > 0.f;  // a tie goes to the even code
  }
  return code;
}

// E4M3 code of top / (6 g), ties to even, at most 126 (448); per = 1 / (6 g).  The quotient need not be exact: it
// proposes a code (and is within 2^-20 of its size, so that the right one is that or a neighbour); the borders beside
// it are looked at where the quotient lies within 16 of its last places of one, or in E4M3's subnormal range, where
// borders are elsewhere.
__device__ __forceinline__ int e4m3_scale(float top, float g, float per) {
  const float t = top * per;
  int c = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3) & 0x7f;
  if (t >= 0x1p-6f && ((__float_as_uint(t) + 16u - (1u << 19)) & ((1u << 20) - 1)) > 32u) return c;
  c = min(c, 126);
  // the borders on both sides of the proposed code
  if (c > 0) {
    const float d = fmaf(-3.f * (e4m3_value(c - 1) + e4m3_value(c)), g, top);
    if (d < 0.f || (d == 0.f && (c & 1))) return c - 1;
  }
  if (c < 126) {
    const float d = fmaf(-3.f * (e4m3_value(c) + e4m3_value(c + 1)), g, top);
    if (d > 0.f || (d == 0.f && (c & 1))) return c + 1;
  }
  return c;
}

// What the elements of a group of step code sc (not 0) are multiplied by: 1 / (s g), moved a little where the code of
// a number of T's significant bits may hang on the quotient's error.  The borders are s g times 1, 3, 5 or 7 times a
// power of two; of numbers with T's bits only y, the one nearest to s g i, and its powers of two can lie that near to
// those of i, all on the same side, which one exact sign tells (on a border they go down for 1 and 5, up for 3 and
// 7: to the even code).  So the quotient is moved by 2^-21 = 8 u (u = 2^-24) to that side: with it the product is
// 4 u off at most, which leaves y on its side; farther numbers stay on theirs if they are more than 12 u from the
// border, and they are where s g i is 15 last places or more from a number of T (it is 1.5 off itself).
// Where borders want both sides: minus the quotient if each is a number of T (as with g a power of two: s g is one
// too, and the rounded quotients of these numbers are the borders themselves), else 0, as in fp32: the caller decides
// element by element (and where products may overflow, behind the largest step).
template <typename T>
__device__ __forceinline__ float nv_quotient(int sc, float g) {
  if constexpr (sizeof(T) == 4) return 0.f;
  const float s = e4m3_value(sc), sg = s * g, inv = __frcp_rn(sg);
  constexpr int kBits = std::is_same<T, __half>::value ? 13 : 16;  // of fp32's mantissa that T lacks
  bool up = false, down = false, beside = sc == 126;
#pragma unroll
  for (int i = 1; i < 8; i += 2) {
    const uint32_t v = __float_as_uint(sg * i);
    if (((v + 14u) & ((1u << kBits) - 1)) <= 28u) {
      const float y = __uint_as_float((v + (1u << (kBits - 1))) & ~((1u << kBits) - 1));
      const float d = fmaf(-(s * i), g, y);
      const bool below = d < 0.f || (d == 0.f && (i & 2) == 0);
      down = down || below;
      up = up || !below;
      beside = beside || d != 0.f;
    }
  }
  return up && down ? (beside ? 0.f : -inv) : up ? inv * (1.f + 0x1p-21f) : down ? inv * (1.f - 0x1p-21f) : inv;
}

struct QuantParams {
  const void* x;
  long long ld;
  const float* scale;
  uint8_t *codes, *scales;
  long long M;
  int K;
  Divisor pieces;  // of 16 elements a row, up to a whole 256 of k
  unsigned units;  // of a thread block
};

// One thread a piece (MANY: one after the other); two (MX) share a group's maximum.  Eight (MX) or four (NV)
// neighbours' scales make the 32-bit word that a row has in a scale tile.  With MANY a block holds the quotients of
// all 126 steps in shared memory.
template <typename T, bool NV, bool VEC, bool MANY>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 8 : 1) k_quantize_fp4(const QuantParams p) {
  constexpr bool TABLE = NV && MANY;
  pdl_wait();
  pdl_trigger();
  __shared__ float quotients[TABLE ? 128 : 1];
  float g = 1.f, per = 0.f;
  bool good = true;  // (the scale)
  if constexpr (NV) {
    if (p.scale != nullptr) g = *p.scale;
    good = g >= kFp4MinScale && g <= kFp4MaxScale;
    per = __fdividef(1.f, 6.f * g);
    if constexpr (TABLE) {
      if (threadIdx.x > 0 && threadIdx.x < 127) quotients[threadIdx.x] = nv_quotient<T>(threadIdx.x, g);
      __syncthreads();
    }
  }
  struct Place {
    long long row;
    int piece;
  };
  const auto place = [&](unsigned unit) {
    const unsigned u = unit * kQuantThreads + threadIdx.x, r = p.pieces.divide(u);
    return Place{r, static_cast<int>(u - r * p.pieces.d)};
  };
  const auto load = [&](const Place& at, Sixteen<T>& x) {
#pragma unroll
    for (auto& v : x.u) v = make_uint4(0, 0, 0, 0);
    if (at.row < p.M && at.piece * kPiece < p.K)
      x.template load<VEC>(static_cast<const T*>(p.x) + at.row * p.ld + at.piece * kPiece);
  };
  unsigned unit = blockIdx.x;
  Place at = place(unit);
  Sixteen<T> x;
  load(at, x);
#pragma unroll 1
  for (;;) {
    const bool more = MANY && unit + gridDim.x < p.units;
    const long long row = at.row;
    const int piece = at.piece, k0 = piece * kPiece;
    const bool live = row < p.M && k0 < p.K;
    uint32_t top = x.top();
    uint32_t sc;
    uint32_t w[2] = {};
    if constexpr (!NV) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const int e = static_cast<int>(top >> 23);
      sc = e == 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
      if (e != 255) {
        const float f = __uint_as_float((254u - sc) << 23);  // 1 / s
        w[0] = x.codes(0, f);
        w[1] = x.codes(1, f);
      }
    } else if (top >= 0x7f800000u || !good) {
      sc = 127u;  // NaN
    } else {
      sc = e4m3_scale(__uint_as_float(top), g, per);
      if (sc != 0) {
        const float q = TABLE ? quotients[sc] : nv_quotient<T>(sc, g);
        if (q > 0.f) {
          w[0] = x.codes(0, q);
          w[1] = x.codes(1, q);
        } else if (sizeof(T) == 2 && q < 0.f) {
          const float sg = e4m3_value(sc) * g;
          w[0] = x.codes_of_quotients(0, -q, sg);
          w[1] = x.codes_of_quotients(1, -q, sg);
        } else {
          const float s = e4m3_value(sc), inv = __frcp_rn(s * g);
          const float lo = inv * (1.f - 0x1p-19f), hi = inv * (1.f + 0x1p-19f);
          w[0] = x.codes(0, lo);
          w[1] = x.codes(1, lo);
          const uint32_t v[2] = {x.codes(0, hi), x.codes(1, hi)};
          if (w[0] != v[0] || w[1] != v[1]) {
#pragma unroll
            for (int k = 0; k < kPiece; ++k) {
              const int bit = 4 * (k & 7);
              if (((w[k >> 3] ^ v[k >> 3]) >> bit) & 15u) {
                const float y = x.get(k);
                const uint32_t c = e2m1_exact(fabsf(y), s, g) | ((__float_as_uint(y) >> 28) & 8u);
                w[k >> 3] = (w[k >> 3] & ~(15u << bit)) | (c << bit);
              }
            }
          }
        }
      }
    }
    if (live) *reinterpret_cast<uint2*>(p.codes + row * (p.K / 2) + k0 / 2) = make_uint2(w[0], w[1]);
    // (pieces behind K hold the zeros that fill a row's last tile)
    if (k0 >= p.K) sc = 0;
    constexpr int SPAN = NV ? 4 : 8;  // lanes of a word
    const int lane = threadIdx.x & 31, j = lane % SPAN, each = SPAN / 4;
    uint32_t word = sc << (8 * (j / each));
#pragma unroll
    for (int o = each; o < SPAN; o *= 2) word |= __shfl_xor_sync(0xffffffffu, word, o);
    if (row < p.M && j == 0)
      *reinterpret_cast<uint32_t*>(p.scales + fp4_scale_at(row, piece / SPAN, p.pieces.d / SPAN)) = word;
    if (!more) return;
    unit += gridDim.x;
    at = place(unit);
    load(at, x);
  }
}

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }

struct DequantParams {
  const uint8_t *codes, *scales;
  const float* scale;
  void* out;
  long long M;
  int K, words;
  Divisor pieces;
  bool wide;  // out is 32-byte aligned
};

// One thread 32 elements (16, with half the loads in flight: 46 us for 8192 rows of 12,288, 32: 40).
template <typename T, bool NV>
__global__ void __launch_bounds__(kQuantThreads) k_dequantize_fp4(const DequantParams p) {
  const unsigned u = blockIdx.x * kQuantThreads + threadIdx.x, r = p.pieces.divide(u);
  const long long row = r;
  pdl_wait();
  pdl_trigger();
  if (row >= p.M) return;
  const int piece = static_cast<int>(u - r * p.pieces.d);
  const uint4 c = *reinterpret_cast<const uint4*>(p.codes + row * (p.K / 2) + piece * 16);
  const int group = NV ? 2 * piece : piece;
  const uint8_t* at = p.scales + fp4_scale_at(row, group / 4, p.words) + group % 4;
  float s[2], g = 1.f;
  if constexpr (NV) {
    const uint32_t two = *reinterpret_cast<const uint16_t*>(at);
    if (p.scale != nullptr) g = *p.scale;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sc = two >> (8 * h) & 255u;
      s[h] = sc < 127u ? e4m3_value(sc) : sc == 128u ? 0.f : __int_as_float(0x7fc00000);
    }
  } else {
    const uint32_t sc = *at;
    s[0] = s[1] = sc == 255u ? __int_as_float(0x7fc00000) : sc == 0 ? 0x1p-127f : __uint_as_float(sc << 23);
  }
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  T* const out = static_cast<T*>(p.out) + row * p.K + piece * 32;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    T t[kPiece];
#pragma unroll
    for (int k = 0; k < kPiece; k += 2) {
      const __half2_raw v2 = __nv_cvt_fp4x2_to_halfraw2(w[2 * h + k / 8] >> (4 * (k & 7)) & 255u, __NV_E2M1);
      // (the product with s is exact)
      float2 v = __fmul2_rn(__half22float2(__half2(v2)), make_float2(s[h], s[h]));
      if constexpr (NV) v = __fmul2_rn(v, make_float2(g, g));
      t[k] = narrow<T>(v.x);
      t[k + 1] = narrow<T>(v.y);
    }
    // (rows of K elements are whole 32s, so that these lie at whole 32 bytes of a 32-byte aligned out)
    uint32_t q[kPiece * sizeof(T) / 4];
    memcpy(q, t, sizeof(t));
    uint32_t* d = reinterpret_cast<uint32_t*>(out + h * kPiece);
#pragma unroll
    for (int j = 0; j < static_cast<int>(kPiece * sizeof(T) / 4); j += 8) {
      if (p.wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d + j), "r"(q[j]), "r"(q[j + 1]),
                     "r"(q[j + 2]), "r"(q[j + 3]), "r"(q[j + 4]), "r"(q[j + 5]), "r"(q[j + 6]), "r"(q[j + 7])
                     : "memory");
      else
        for (int i = 0; i < 8; i += 4)
          *reinterpret_cast<uint4*>(d + j + i) = make_uint4(q[j + i], q[j + i + 1], q[j + i + 2], q[j + i + 3]);
    }
  }
}

// Row-major scales into tiles (a thread a 32-bit word of a row).  NV: the matrix unit's scales have no sign, so
// bytes that have one become 127 (NaN), -0 becomes 0.
__global__ void __launch_bounds__(kQuantThreads) k_fp4_tile_scales(const uint8_t* src, uint8_t* tiles, long long rows,
                                                                   int n, int words, bool nv) {
  const long long u = static_cast<long long>(blockIdx.x) * kQuantThreads + threadIdx.x;
  const long long row = u / words;
  const int word = static_cast<int>(u - row * words);
  if (row >= (rows + 127) / 128 * 128) return;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (row < rows && word * 4 + j < n) {
      uint32_t sc = src[row * n + word * 4 + j];
      if (nv && sc > 127u) sc = sc == 128u ? 0u : 127u;
      w |= sc << (8 * j);
    }
  *reinterpret_cast<uint32_t*>(tiles + fp4_scale_at(row, word, words)) = w;
}

bool elem_ok(int e) { return e == DFLASH_ELEM_F32 || e == DFLASH_ELEM_BF16 || e == DFLASH_ELEM_F16; }
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Thread blocks for all pieces, or 0 where these are too many to be counted in 32 bits.
unsigned blocks_of(long long rows, long long per_row) {
  const long long n = (rows * per_row + kQuantThreads - 1) / kQuantThreads;
  return n > INT32_MAX / kQuantThreads ? 0u : static_cast<unsigned>(n);
}

}  // namespace

}  // namespace dflash

using namespace dflash;

extern "C" {

size_t dflash_fp4_scales_size(int format, long long rows, int K) {
  if ((format != DFLASH_FP4_MX && format != DFLASH_FP4_NV) || !fp4_shape_ok(rows, K)) return 0;
  return static_cast<size_t>((rows + 127) / 128) * fp4_words(format, K) * 512;
}

dflash_status dflash_fp4_tile_scales(const void* scales, int format, long long rows, int K, void* tiles,
                                     dflash_stream stream) {
  if (scales == nullptr || tiles == nullptr || (format != DFLASH_FP4_MX && format != DFLASH_FP4_NV) || rows < 1 ||
      K < 1 || !aligned(tiles, 16))
    return DFLASH_ERR_INVALID_ARG;
  if (!fp4_shape_ok(rows, K)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  const int words = fp4_words(format, K);
  const unsigned blocks = blocks_of((rows + 127) / 128 * 128, words);
  if (blocks == 0) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  k_fp4_tile_scales<<<blocks, kQuantThreads, 0, stream>>>(static_cast<const uint8_t*>(scales),
                                                          static_cast<uint8_t*>(tiles), rows, K / fp4_group(format),
                                                          words, format == DFLASH_FP4_NV);
  return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

dflash_status dflash_quantize_fp4(const void* X, int x_elem, long long ld_x, long long M, int K, int format,
                                  const float* scale, void* codes, void* scales, dflash_stream stream) {
  if (X == nullptr || codes == nullptr || scales == nullptr || M < 1 || K < 1 || !elem_ok(x_elem))
    return DFLASH_ERR_INVALID_ARG;
  if ((format != DFLASH_FP4_MX && format != DFLASH_FP4_NV) || (format == DFLASH_FP4_MX && scale != nullptr))
    return DFLASH_ERR_INVALID_ARG;
  const int size = x_elem == DFLASH_ELEM_F32 ? 4 : 2;
  if ((M > 1 && ld_x < K) || !aligned(X, size) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(scale, 4))
    return DFLASH_ERR_INVALID_ARG;
  if (!fp4_shape_ok(M, K) || ld_x > INT64_MAX / 8 / M) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  QuantParams p{X, ld_x, scale, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), M, K,
                Divisor(static_cast<unsigned>(K + 255) / 256 * 16), 0};
  const unsigned blocks = blocks_of(M, p.pieces.d);
  if (blocks == 0) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  const bool vec = aligned(X, 32) && (M == 1 || ld_x * size % 32 == 0);
  p.units = blocks;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return DFLASH_ERR_CUDA;
  // Blocks that go from piece to piece and hold the steps' quotients, for 16-bit NV from 16 units an SM on (2176 x 6144
  // fp16: 8.8 us, one unit a block 10.9; 2176 x 4096 as long either way, 1024 x 4096 4.1 against 4.0), 32 blocks an SM at
  // most (8 to 64: 43.1, 43.6, 43.0, 42.6, 42.9 us).  In fp32 memory is the bound (8192 x 12,288: 68.5 us either way).
  const unsigned many = static_cast<unsigned>(sms) * 16, grid = std::min(many * 2, blocks / 2);
  const auto run = [&](auto t, auto nv, auto v) {
    using T = decltype(t);
    constexpr bool NV = decltype(nv)::value, VEC = decltype(v)::value, MANY = NV && sizeof(T) == 2;
    const bool go = MANY && blocks >= many;
    e = launch_cached(go ? k_quantize_fp4<T, NV, VEC, MANY> : k_quantize_fp4<T, NV, VEC, false>, go ? grid : blocks,
                      kQuantThreads, 0, stream, 1, p);
  };
  const auto pick = [&](auto t) {
    if (format == DFLASH_FP4_NV) vec ? run(t, std::true_type{}, std::true_type{}) : run(t, std::true_type{}, std::false_type{});
    else vec ? run(t, std::false_type{}, std::true_type{}) : run(t, std::false_type{}, std::false_type{});
  };
  if (x_elem == DFLASH_ELEM_F32) pick(float{});
  else if (x_elem == DFLASH_ELEM_BF16) pick(__nv_bfloat16{});
  else pick(__half{});
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

dflash_status dflash_dequantize_fp4(const void* codes, const void* scales, int format, const float* scale, long long M,
                                    int K, void* out, int out_elem, dflash_stream stream) {
  if (out == nullptr || codes == nullptr || scales == nullptr || M < 1 || K < 1 || !elem_ok(out_elem))
    return DFLASH_ERR_INVALID_ARG;
  if ((format != DFLASH_FP4_MX && format != DFLASH_FP4_NV) || (format == DFLASH_FP4_MX && scale != nullptr))
    return DFLASH_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(scale, 4))
    return DFLASH_ERR_INVALID_ARG;
  if (!fp4_shape_ok(M, K)) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  DequantParams p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), scale, out, M, K,
                  fp4_words(format, K), Divisor(static_cast<unsigned>(K / 32)), aligned(out, 32)};
  const unsigned blocks = blocks_of(M, p.pieces.d);
  if (blocks == 0) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  cudaError_t e = cudaSuccess;
  const auto pick = [&](auto t) {
    using T = decltype(t);
    e = launch_cached(format == DFLASH_FP4_NV ? k_dequantize_fp4<T, true> : k_dequantize_fp4<T, false>, blocks, kQuantThreads, 0,
                      stream, 1, p);
  };
  if (out_elem == DFLASH_ELEM_F32) pick(float{});
  else if (out_elem == DFLASH_ELEM_BF16) pick(__nv_bfloat16{});
  else pick(__half{});
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
