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

constexpr int kW4Unit = 128;     // k of a unit: 64 bytes of a weight row, 256 of an activation row
constexpr int kW4MaxM = 32;

template <typename X>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
  // 128 + v for v = 0 .. 128 is kMagic + v, exact
  static constexpr uint32_t kMagic = 0x43004300u;
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // an E2M1 code's value: its exponent and mantissa bits in place (an exponent
  // field of 0 .. 3, so the value times 2^-126), the sign at bit 15, and one
  // exact product by 2^126
  static __device__ __forceinline__ uint32_t e2m1(uint32_t c) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(((c & 7u) << 6) | ((c & 8u) << 12)), "r"(0x7E807E80u));
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
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024 + v, likewise
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t e2m1(uint32_t c) {  // (by 2^-14 and 2^14)
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(((c & 7u) << 9) | ((c & 8u) << 12)), "r"(0x74007400u));
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

struct W4Params {
  const uint8_t* scale;
  const uint8_t* zero;
  float* out;
  int* status;
  int N, K, groups, M;
  int scale_elem, scale_size;
  int panel;               // units of a panel
  int piece_s, piece_z;    // bytes of an asynchronous copy of scales, of zero points (0: element by element)
  int row_warps;           // warps that share a k-group's activations, each with rows of its own
  int x_bytes, stage_bytes, stages;
};

// Integer codes i and i + 4 of a word, less the zero point, as a pair of 16-bit values.
template <typename X>
__device__ __forceinline__ uint32_t widen(uint32_t w, int i, uint32_t bias) {
  return Half2<X>::sub(((w >> (4 * i)) & 0x000F000Fu) | Half2<X>::kMagic, bias);
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

__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes, bool there) {
  const uint32_t d = smem_u32(dst);
  const int n = there ? bytes : 0;  // (what is not there reads as zeros)
  if (bytes == 16) asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
  else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

constexpr int kW4MaxStages = 8;

// E2M1 codes are widened through a table in shared memory: a byte (two codes)
// to its pair of 16-bit values, with a copy for every lane (entry e of lane l
// at 256 e + 4 l, so that one byte permutation makes the address and no two
// lanes share a bank).  Taking the codes apart with shifts and masks costs
// five instructions a pair against the table's two, and the kernel is bound by
// its instructions.
constexpr int kW4Table = 65536;

template <int GROUP, int TILES, int NB>
struct W4Layout {
  // (with more than 16 activation rows a thread needs over 128 registers)
  static constexpr int WARPS = NB <= 2 ? 16 : 8, THREADS = WARPS * 32;
  static constexpr int NG = kW4Unit / GROUP;           // groups of a unit
  static constexpr int ROWS = 16 * TILES;              // weight rows of a warp
  static constexpr int BYTES_W = ROWS * (kW4Unit / 2); // their codes of a unit
  // scales and zero points of a panel, a row's together: at most PANEL units of
  // 16-bit scales (half as many of 32-bit ones)
  static constexpr int PANEL = NG == 4 ? 2 : 4;
  static constexpr int PITCH_S = PANEL * NG * 2, PITCH_Z = PANEL * NG;  // (16 or 8 bytes: no two of 8 rows share a bank)
  static constexpr int BYTES_P = ROWS * (PITCH_S + PITCH_Z);
  // a warp's sums, [activation row][weight row]
  static constexpr int PITCH_O = ROWS + 4;
  static constexpr int BYTES_O = NB * 8 * PITCH_O * 4;
  static constexpr int FIXED = 1024 + WARPS * (2 * BYTES_P + BYTES_O) + WARPS * 2 * kW4MaxStages * 8;
};

// Persistent CTAs, one an SM, over tiles of weight rows.  The
// warps form k-groups: group g takes panels g, g + groups, .. of k (a panel:
// a few units of 128 k), and each of its row_warps warps 16 * TILES rows of
// the tile.  A group streams its units (the codes of its warps' rows and the
// activations, which they share) through a ring of TMA copies that runs on
// over the tiles; a warp keeps a unit's activations in registers over its row
// tiles.  Scales and zero points come a panel ahead, a lane copying a row's
// piece (read per unit, a warp would touch every row's line for a few bytes).
// At the end of a tile the CTA adds the groups' sums in order.  NB: blocks of
// 8 activation rows (the MMA's N).
//
// Within a scale group a thread of a quad takes 8 * GROUP / 32 adjacent codes
// (one 4, 8 or 16-byte read), so an MMA adds products of one group only.
template <typename X, bool E2M1, int GROUP, int TILES, int NB>
__global__ void __launch_bounds__(W4Layout<GROUP, TILES, NB>::THREADS, 1)
    k_gemm_w4(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
              const __grid_constant__ W4Params p) {
  using H = Half2<X>;
  using L = W4Layout<GROUP, TILES, NB>;
  constexpr int NG = L::NG;
  constexpr int WPT = GROUP / 32;      // words a thread takes of a group
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + (E2M1 ? kW4Table : 0) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t4 = lane & 3;
  const int kgroups = L::WARPS / p.row_warps, kg = warp / p.row_warps, rw = warp % p.row_warps;
  const int tile_rows = p.row_warps * L::ROWS, tiles = (p.N + tile_rows - 1) / tile_rows;
  const int units = (p.K + kW4Unit - 1) / kW4Unit, panels = (units + p.panel - 1) / p.panel;
  uint8_t* ring = smem + kg * p.stages * p.stage_bytes;
  uint8_t* fixed = smem + kgroups * p.stages * p.stage_bytes;
  float* sums = reinterpret_cast<float*>(fixed);                              // [warp][NB * 8][PITCH_O]
  uint8_t* panel_buf = fixed + L::WARPS * L::BYTES_O + warp * 2 * L::BYTES_P; // [2]: scales, then zero points
  uint64_t* full = reinterpret_cast<uint64_t*>(fixed + L::WARPS * (L::BYTES_O + 2 * L::BYTES_P)) +
                   kg * 2 * kW4MaxStages;
  int* through = reinterpret_cast<int*>(full + kW4MaxStages);  // per slot: warps of the group that are done with its unit

  // The group's next unit to fetch: every warp counts along, the last one
  // through with a slot refills it (lane 0).
  int f_tile = kg < panels ? blockIdx.x : tiles, f_panel = kg, f_unit = 0;
  int fetched = 0;
  auto next_unit = [&](bool issue, int s) {
    const int unit = f_panel * p.panel + f_unit, k = unit * kW4Unit;
    if (issue) {
      uint8_t* dst = ring + s * p.stage_bytes;
      mbar_arrive_expect_tx(&full[s], p.row_warps * L::BYTES_W + p.M * 256);
      tma_load_2d(dst, &tmX, &full[s], k, 0);
      tma_load_2d(dst + p.M * 128, &tmX, &full[s], k + 64, 0);
      tma_load_2d(dst + p.x_bytes, &tmW, &full[s], k / 2, f_tile * tile_rows);
    }
    ++fetched;
    if (++f_unit == p.panel || unit + 1 == units) {
      f_unit = 0;
      f_panel += kgroups;
      if (f_panel >= panels) {
        f_panel = kg;
        f_tile += gridDim.x;
      }
    }
  };
  if (rw == 0 && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      through[s] = 0;
    }
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (lane == 0)
    for (int s = 0; s < p.stages && f_tile < tiles; ++s) next_unit(rw == 0, s);

  // scales and zero points of a panel into buffer b
  auto fetch_panel = [&](int tile, int panel, int b) {
    if (lane < L::ROWS) {
      const int per = p.panel * NG, left = min(per, p.groups - panel * per);  // groups; past the last one: zeros
      const long long at = static_cast<long long>(min(tile * tile_rows + rw * L::ROWS + lane, p.N - 1)) * p.groups +
                           panel * per;
      uint8_t* ds = panel_buf + b * L::BYTES_P + lane * L::PITCH_S;
      const uint8_t* ss = p.scale + at * p.scale_size;
      if (p.piece_s != 0) {
        for (int o = 0; o < per * p.scale_size; o += p.piece_s)
          copy_async(ds + o, o < left * p.scale_size ? ss + o : p.scale, p.piece_s, o < left * p.scale_size);
      } else {
        for (int j = 0; j < per; ++j) {
          if (p.scale_size == 4)
            reinterpret_cast<uint32_t*>(ds)[j] = j < left ? reinterpret_cast<const uint32_t*>(ss)[j] : 0u;
          else
            reinterpret_cast<uint16_t*>(ds)[j] = j < left ? reinterpret_cast<const uint16_t*>(ss)[j] : uint16_t(0);
        }
      }
      if (!E2M1 && p.zero != nullptr) {
        uint8_t* dz = panel_buf + b * L::BYTES_P + L::ROWS * L::PITCH_S + lane * L::PITCH_Z;
        const uint8_t* sz = p.zero + at;
        if (p.piece_z != 0) {
          for (int o = 0; o < per; o += p.piece_z) copy_async(dz + o, o < left ? sz + o : p.zero, p.piece_z, o < left);
        } else {
          for (int j = 0; j < per; ++j) dz[j] = j < left ? sz[j] : uint8_t(0);
        }
      }
    }
    copies_commit();
  };
  if (kg < panels && blockIdx.x < static_cast<unsigned>(tiles)) fetch_panel(blockIdx.x, kg, 0);
  if constexpr (E2M1) {
    for (int e = warp; e < 256; e += L::WARPS)
      *reinterpret_cast<uint32_t*>(smem_raw + e * 256 + lane * 4) = H::e2m1(e & 15) | H::e2m1(e >> 4) << 16;
  }
  __syncthreads();  // the rings' barriers (and the table) are set up
  // two E2M1 codes: byte i of a word
  const uint32_t lane4 = lane * 4, table = smem_u32(smem_raw);
  auto look_up = [&](uint32_t w, int i) {
    uint32_t v;
    asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(__byte_perm(w, lane4, 0x5504 | i << 4) + table));
    return v;
  };

  // where a thread finds its 16-byte pieces of the activations: 64 k to a
  // 128-byte row, pieces swizzled by the row's place (columns past M are not kept)
  int xoff[NB][NG * WPT];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int w = 0; w < NG * WPT; ++w) {
      const int piece = w / WPT * (GROUP / 8) + t4 * WPT + w % WPT;  // 8 k each
      const int row = min(j * 8 + gr, p.M - 1) + (piece >> 3) * p.M;
      xoff[j][w] = row * 128 + (((piece ^ row) & 7) << 4);
    }
  // and its codes: rows of 64 bytes, pieces swizzled by the row's bits 1 and 2
  const int wrow = p.x_bytes + (rw * L::ROWS + gr) * 64, wswz = (gr >> 1 & 3) << 4;

  bool ok = true;
  int s = 0, b = 0;
  uint32_t parity = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    float acc[TILES][NB][4] = {};
    for (int panel = kg; panel < panels; panel += kgroups, b ^= 1) {
      const bool more = panel + kgroups < panels;
      if (more || tile + static_cast<int>(gridDim.x) < tiles) {
        fetch_panel(more ? tile : tile + gridDim.x, more ? panel + kgroups : kg, b ^ 1);
        copies_wait<1>();
      } else {
        copies_wait<0>();
      }
      __syncwarp();
      const uint8_t* bs = panel_buf + b * L::BYTES_P + gr * L::PITCH_S;
      const uint8_t* bz = panel_buf + b * L::BYTES_P + L::ROWS * L::PITCH_S + gr * L::PITCH_Z;
      const int count = min(p.panel, units - panel * p.panel);
      for (int u = 0; u < count; ++u) {
        ok = ok && w4_wait(&full[s], parity, p.status);
        const uint8_t* xs = ring + s * p.stage_bytes;
        // B fragments: pairs (k, k + 1) for E2M1, (k, k + 4) for integers
        uint32_t xb[NB][NG * WPT][4];
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int w = 0; w < NG * WPT; ++w) {
            const uint4 v = *reinterpret_cast<const uint4*>(xs + xoff[j][w]);
            xb[j][w][0] = E2M1 ? v.x : __byte_perm(v.x, v.z, 0x5410);
            xb[j][w][1] = E2M1 ? v.y : __byte_perm(v.x, v.z, 0x7632);
            xb[j][w][2] = E2M1 ? v.z : __byte_perm(v.y, v.w, 0x5410);
            xb[j][w][3] = E2M1 ? v.w : __byte_perm(v.y, v.w, 0x7632);
          }
        // the unit's scales
        float sc[TILES][2][NG];
        auto scales = [&](auto&& read) {
#pragma unroll
          for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) read(bs + (t * 16 + h * 8) * L::PITCH_S + u * NG * p.scale_size, sc[t][h]);
        };
        auto scales16 = [&](auto&& as_float) {
          scales([&](const uint8_t* src, float (&v)[NG]) {
            uint32_t w[(NG + 1) / 2];
            if constexpr (NG == 4) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(src);
            else if constexpr (NG == 2) w[0] = *reinterpret_cast<const uint32_t*>(src);
            else w[0] = *reinterpret_cast<const uint16_t*>(src);
#pragma unroll
            for (int g = 0; g < NG; ++g) v[g] = as_float(w[g / 2], g & 1);
          });
        };
        if (p.scale_elem == DFLASH_ELEM_BF16)
          scales16([](uint32_t w, int hi) { return __uint_as_float(hi ? w & 0xffff0000u : w << 16); });
        else if (p.scale_elem == DFLASH_ELEM_F16)
          scales16([](uint32_t w, int hi) {
            return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> (16 * hi))));
          });
        else
          scales([](const uint8_t* src, float (&v)[NG]) {
            if constexpr (NG == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
            else if constexpr (NG == 2) *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
            else v[0] = *reinterpret_cast<const float*>(src);
          });
        uint32_t z[TILES][2];
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            z[t][h] = 0x08080808u;
            if (!E2M1 && p.zero != nullptr) {
              const uint8_t* src = bz + (t * 16 + h * 8) * L::PITCH_Z + u * NG;
              if constexpr (NG == 4) z[t][h] = *reinterpret_cast<const uint32_t*>(src);
              else if constexpr (NG == 2) z[t][h] = *reinterpret_cast<const uint16_t*>(src);
              else z[t][h] = *src;
            }
          }
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            uint32_t word[2][WPT], bias[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint8_t* src = xs + wrow + (t * 16 + h * 8) * 64 + ((g * (GROUP / 2) + t4 * WPT * 4) ^ wswz);
              if constexpr (WPT == 4) *reinterpret_cast<uint4*>(word[h]) = *reinterpret_cast<const uint4*>(src);
              else if constexpr (WPT == 2) *reinterpret_cast<uint2*>(word[h]) = *reinterpret_cast<const uint2*>(src);
              else word[h][0] = *reinterpret_cast<const uint32_t*>(src);
              bias[h] = E2M1 ? 0u : H::kMagic + (z[t][h] >> (8 * g) & 0xffu) * 0x00010001u;
            }
            float d[NB][4];
#pragma unroll
            for (int w = 0; w < WPT; ++w) {
              uint32_t a[2][4];
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  a[q][h] = E2M1 ? look_up(word[h][w], 2 * q) : widen<X>(word[h][w], 2 * q, bias[h]);
                  a[q][2 + h] = E2M1 ? look_up(word[h][w], 2 * q + 1) : widen<X>(word[h][w], 2 * q + 1, bias[h]);
                }
#pragma unroll
              for (int j = 0; j < NB; ++j) {
                const uint32_t* v = xb[j][g * WPT + w];
                if (w == 0) H::mma0(d[j], a[0], v[0], v[1]);
                else H::mma(d[j], a[0], v[0], v[1]);
                H::mma(d[j], a[1], v[2], v[3]);
              }
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              acc[t][j][0] += sc[t][0][g] * d[j][0];
              acc[t][j][1] += sc[t][0][g] * d[j][1];
              acc[t][j][2] += sc[t][1][g] * d[j][2];
              acc[t][j][3] += sc[t][1][g] * d[j][3];
            }
          }
        __syncwarp();
        if (lane == 0 && f_tile < tiles) {
          __threadfence_block();
          const bool last = atomicAdd(&through[s], 1) == p.row_warps - 1;
          if (last) {
            __threadfence_block();
            through[s] = 0;
          }
          next_unit(last && ok, s);
        }
        if (++s == p.stages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    float* mine = sums + warp * (L::BYTES_O / 4);
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(j * 8 + 2 * t4 + (e & 1)) * L::PITCH_O + t * 16 + (e >> 1) * 8 + gr] = acc[t][j][e];
    __syncthreads();
    for (int e = threadIdx.x; e < tile_rows * p.M; e += L::THREADS) {
      const int m = e / tile_rows, r = e - m * tile_rows, n = tile * tile_rows + r;
      if (n >= p.N) continue;
      const float* src = sums + r / L::ROWS * (L::BYTES_O / 4) + m * L::PITCH_O + r % L::ROWS;
      float v = 0.f;
      for (int g = 0; g < kgroups; ++g) v += src[g * p.row_warps * (L::BYTES_O / 4)];
      p.out[static_cast<long long>(m) * p.N + n] = v;
    }
    __syncthreads();
  }
  if (lane == 0 && !ok) {  // a wait gave up: copies still in flight get bounded waits before the CTA leaves
    for (int i = max(0, fetched - p.stages); i < fetched; ++i)
      w4_wait(&full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1, p.status);
  }
}

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

int w4_x_bytes(int M) { return (M * 256 + 1023) / 1024 * 1024; }

// Units that the rings can hold per k-group (0 or 1: too few).
template <int GROUP, int TILES, int NB>
int w4_stages(int M, int row_warps, bool e2m1) {
  using L = W4Layout<GROUP, TILES, NB>;
  return std::min(kW4MaxStages, (232448 - L::FIXED - (e2m1 ? kW4Table : 0)) /
                                    (L::WARPS / row_warps * (w4_x_bytes(M) + row_warps * L::BYTES_W)));
}

template <typename X, bool E2M1, int GROUP, int TILES, int NB>
cudaError_t launch_w4_t(W4Params p, const void* W, const void* x, int row_warps, int sms, cudaStream_t s) {
  using L = W4Layout<GROUP, TILES, NB>;
  const int tile_rows = row_warps * L::ROWS, kgroups = L::WARPS / row_warps;
  CUtensorMap tw, tx;
  if (!w4_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, W, p.N, p.K / 2, tile_rows, kW4Unit / 2,
              CU_TENSOR_MAP_SWIZZLE_64B) ||
      !w4_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, x, p.M, p.K, p.M, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  p.row_warps = row_warps;
  // the longest panel that leaves every k-group one
  const int units = (p.K + kW4Unit - 1) / kW4Unit;
  p.panel = p.scale_size == 4 ? L::PANEL / 2 : L::PANEL;
  while (p.panel > 1 && units < p.panel * kgroups) p.panel /= 2;
  const int per = p.panel * L::NG;
  p.piece_s = w4_piece(per * p.scale_size, static_cast<long long>(p.groups) * p.scale_size, p.scale);
  p.piece_z = w4_piece(per, p.groups, p.zero);
  p.x_bytes = w4_x_bytes(p.M);
  p.stage_bytes = p.x_bytes + row_warps * L::BYTES_W;
  p.stages = w4_stages<GROUP, TILES, NB>(p.M, row_warps, E2M1);
  const int smem = L::FIXED + (E2M1 ? kW4Table : 0) + kgroups * p.stages * p.stage_bytes;
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(smem, [](int v) {
    return cudaFuncSetAttribute(k_gemm_w4<X, E2M1, GROUP, TILES, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  const int tiles = (p.N + tile_rows - 1) / tile_rows;
  return launch_k(k_gemm_w4<X, E2M1, GROUP, TILES, NB>, dim3(std::min(tiles, sms)), dim3(L::THREADS), smem, s, dim3(1),
                  false, tw, tx, p);
}

// Rows of a tile: tall ones read the activations fewer times and share the
// cost of a tile's end (about that of kTileEnd rows); short ones spread few
// rows over the SMs.
template <typename X, bool E2M1, int GROUP, int NB>
cudaError_t launch_w4_n(const W4Params& p, const void* W, const void* x, int sms, cudaStream_t s) {
  constexpr int kTileEnd = 24;
  int best = 128;
  long long cost = INT64_MAX;
  for (int rows = 128; rows >= 16; rows /= 2) {
    if ((rows == 16 ? w4_stages<GROUP, 1, NB>(p.M, 1, E2M1) : w4_stages<GROUP, 2, NB>(p.M, rows / 32, E2M1)) < 2)
      continue;  // (the rings of so many groups do not fit)
    const long long tiles = (p.N + rows - 1) / rows, c = (tiles + sms - 1) / sms * (rows + kTileEnd);
    if (c < cost) {
      cost = c;
      best = rows;
    }
  }
  if (best == 16) return launch_w4_t<X, E2M1, GROUP, 1, NB>(p, W, x, 1, sms, s);
  return launch_w4_t<X, E2M1, GROUP, 2, NB>(p, W, x, best / 32, sms, s);
}

template <typename X, bool E2M1, int GROUP>
cudaError_t launch_w4_g(const W4Params& p, const void* W, const void* x, int sms, cudaStream_t s) {
  switch ((p.M + 7) / 8) {
    case 1: return launch_w4_n<X, E2M1, GROUP, 1>(p, W, x, sms, s);
    case 2: return launch_w4_n<X, E2M1, GROUP, 2>(p, W, x, sms, s);
    case 3: return launch_w4_n<X, E2M1, GROUP, 3>(p, W, x, sms, s);
    default: return launch_w4_n<X, E2M1, GROUP, 4>(p, W, x, sms, s);
  }
}

template <typename X, bool E2M1>
cudaError_t launch_w4(const W4Params& p, const void* W, const void* x, int group, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (group == 32) return launch_w4_g<X, E2M1, 32>(p, W, x, sms, s);
  if (group == 64) return launch_w4_g<X, E2M1, 64>(p, W, x, sms, s);
  return launch_w4_g<X, E2M1, 128>(p, W, x, sms, s);
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
  W4Params p{};
  p.scale = static_cast<const uint8_t*>(scale);
  p.zero = static_cast<const uint8_t*>(zero);
  p.out = out;
  p.status = status;
  p.N = N;
  p.K = K;
  p.groups = (K + group - 1) / group;
  p.M = M;
  p.scale_elem = scale_elem;
  p.scale_size = ss;
  cudaError_t e;
  if (x_elem == DFLASH_ELEM_BF16)
    e = format == DFLASH_W4_E2M1 ? launch_w4<__nv_bfloat16, true>(p, W, X, group, stream)
                                 : launch_w4<__nv_bfloat16, false>(p, W, X, group, stream);
  else
    e = format == DFLASH_W4_E2M1 ? launch_w4<__half, true>(p, W, X, group, stream)
                                 : launch_w4<__half, false>(p, W, X, group, stream);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}
