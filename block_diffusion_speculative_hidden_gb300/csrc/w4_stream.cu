// The kernel of dflash_gemm_w4 for 17 to 32 activation rows, which streams the
// activations beside the weights.
#include "w4_common.cuh"

namespace dflash {

namespace {

constexpr int kW4Unit = 128;     // k of a unit: 64 bytes of a weight row, 256 of an activation row
constexpr int kW4MaxStages = 8;

struct StreamParams {
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

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

template <int GROUP, int TILES, int NB>
struct StreamLayout {
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
//
// Bound by instructions as w4_resident.cuh is, and by what a tile's end costs
// (24576 x 4096 in groups of 64: 24 rows 42 us, 32 rows 48; 2880 x 2880 in
// groups of 32, 17 rows 9.6).
template <typename X, bool E2M1, int GROUP, int TILES, int NB>
__global__ void __launch_bounds__(StreamLayout<GROUP, TILES, NB>::THREADS, 1)
    k_gemm_w4_stream(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
              const __grid_constant__ StreamParams p) {
  using H = Half2<X>;
  using L = StreamLayout<GROUP, TILES, NB>;
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
          copy_async(smem_u32(ds + o), o < left * p.scale_size ? ss + o : p.scale, p.piece_s,
                     o < left * p.scale_size ? p.piece_s : 0);
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
          for (int o = 0; o < per; o += p.piece_z)
            copy_async(smem_u32(dz + o), o < left ? sz + o : p.zero, p.piece_z, o < left ? p.piece_z : 0);
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
              bias[h] = E2M1 ? 0u : H::bias(z[t][h], g);
            }
            float d[NB][4];
#pragma unroll
            for (int w = 0; w < WPT; ++w) {
              uint32_t a[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t v[4];
                if constexpr (E2M1) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) v[i] = look_up(word[h][w], i);
                } else {
                  H::widen(word[h][w], bias[h], v);
                }
                a[0][h] = v[0];
                a[0][2 + h] = v[1];
                a[1][h] = v[2];
                a[1][2 + h] = v[3];
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
      p.out[static_cast<long long>(m) * p.N + n] = v * (E2M1 ? 1.f : H::kSum);
    }
    __syncthreads();
  }
  if (lane == 0 && !ok) {  // a wait gave up: copies still in flight get bounded waits before the CTA leaves
    for (int i = max(0, fetched - p.stages); i < fetched; ++i)
      w4_wait(&full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1, p.status);
  }
}

int w4_x_bytes(int M) { return (M * 256 + 1023) / 1024 * 1024; }

// Units that the rings can hold per k-group (0 or 1: too few).
template <int GROUP, int TILES, int NB>
int w4_stages(int M, int row_warps, bool e2m1) {
  using L = StreamLayout<GROUP, TILES, NB>;
  return std::min(kW4MaxStages, (kW4Smem - L::FIXED - (e2m1 ? kW4Table : 0)) /
                                    (L::WARPS / row_warps * (w4_x_bytes(M) + row_warps * L::BYTES_W)));
}

template <typename X, bool E2M1, int GROUP, int TILES, int NB>
cudaError_t launch_w4_t(const W4Args& a, int row_warps, cudaStream_t s) {
  using L = StreamLayout<GROUP, TILES, NB>;
  const int tile_rows = row_warps * L::ROWS, kgroups = L::WARPS / row_warps;
  StreamParams p{};
  p.scale = a.scale;
  p.zero = a.zero;
  p.out = a.out;
  p.status = a.status;
  p.N = a.N;
  p.K = a.K;
  p.groups = a.groups;
  p.M = a.M;
  p.scale_elem = a.scale_elem;
  p.scale_size = a.scale_size;
  CUtensorMap tw, tx;
  if (!w4_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.W, p.N, p.K / 2, tile_rows, kW4Unit / 2,
              CU_TENSOR_MAP_SWIZZLE_64B) ||
      !w4_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.x, p.M, p.K, p.M, 64, CU_TENSOR_MAP_SWIZZLE_128B))
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
    return cudaFuncSetAttribute(k_gemm_w4_stream<X, E2M1, GROUP, TILES, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  const int tiles = (p.N + tile_rows - 1) / tile_rows;
  return launch_k(k_gemm_w4_stream<X, E2M1, GROUP, TILES, NB>, dim3(std::min(tiles, a.sms)), dim3(L::THREADS), smem, s, dim3(1),
                  false, tw, tx, p);
}

// Rows of a tile: tall ones read the activations fewer times and share the
// cost of a tile's end (about that of kTileEnd rows); short ones spread few
// rows over the SMs.
template <typename X, bool E2M1, int GROUP, int NB>
cudaError_t launch_w4_n(const W4Args& a, cudaStream_t s) {
  constexpr int kTileEnd = 24;
  int best = 128;
  long long cost = INT64_MAX;
  for (int rows = 128; rows >= 16; rows /= 2) {
    if ((rows == 16 ? w4_stages<GROUP, 1, NB>(a.M, 1, E2M1) : w4_stages<GROUP, 2, NB>(a.M, rows / 32, E2M1)) < 2)
      continue;  // (the rings of so many groups do not fit)
    const long long tiles = (a.N + rows - 1) / rows, c = (tiles + a.sms - 1) / a.sms * (rows + kTileEnd);
    if (c < cost) {
      cost = c;
      best = rows;
    }
  }
  if (best == 16) return launch_w4_t<X, E2M1, GROUP, 1, NB>(a, 1, s);
  return launch_w4_t<X, E2M1, GROUP, 2, NB>(a, best / 32, s);
}

template <typename X, bool E2M1>
cudaError_t launch_w4_x(const W4Args& a, cudaStream_t s) {
  const bool three = a.M <= 24;  // blocks of 8 activation rows
  if (a.group == 32) return three ? launch_w4_n<X, E2M1, 32, 3>(a, s) : launch_w4_n<X, E2M1, 32, 4>(a, s);
  if (a.group == 64) return three ? launch_w4_n<X, E2M1, 64, 3>(a, s) : launch_w4_n<X, E2M1, 64, 4>(a, s);
  return three ? launch_w4_n<X, E2M1, 128, 3>(a, s) : launch_w4_n<X, E2M1, 128, 4>(a, s);
}

}  // namespace

cudaError_t launch_w4_stream(const W4Args& a, bool e2m1, cudaStream_t s) {
  if (a.x_elem == DFLASH_ELEM_BF16)
    return e2m1 ? launch_w4_x<__nv_bfloat16, true>(a, s) : launch_w4_x<__nv_bfloat16, false>(a, s);
  return e2m1 ? launch_w4_x<__half, true>(a, s) : launch_w4_x<__half, false>(a, s);
}

}  // namespace dflash
