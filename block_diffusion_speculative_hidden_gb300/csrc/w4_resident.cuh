// The kernel of dflash_gemm_w4 for up to 16 activation rows, which keeps the
// activations in shared memory.
#pragma once

#include "w4_common.cuh"

namespace dflash {

namespace {

constexpr int kW4Unit = 256;     // k of a unit: 128 bytes of a weight row, 512 of an activation row
constexpr int kW4Rows = 16;      // weight rows of a tile (an MMA's)
constexpr int kW4Warps = 16;
constexpr int kW4Threads = kW4Warps * 32;
constexpr int kW4MaxStages = 4;
constexpr int kW4Reserved = 1024;  // the system's bytes before a CTA's shared memory

struct W4Params {
  const uint8_t* scale;
  const uint8_t* zero;
  const uint4* x;
  float* out;
  int* status;
  int N, K, groups, M;
  int piece_s, piece_z;    // bytes of an asynchronous copy of scales, of zero points (0: element by element)
  int chunk, chunks;       // units of k whose activations shared memory holds, and how often that changes
  int share, extra;        // tiles of a CTA, and how many have one more
  int pitch;               // bytes of an activation row there
  int stages;              // units in flight per warp
  int off_scale, off_zero, off_sum, off_ring, off_high;  // shared memory
  int low_warps;           // warps whose ring is at off_ring, the others' are at off_high
};

// One arrival at bar once this thread's asynchronous copies so far are there.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Persistent CTAs, one an SM, each with a run of tiles of 16 weight rows.  The
// activations of a chunk of k (all of k where they fit) lie in shared memory,
// in the order of the MMA's fragments; the CTA's tiles x units of that chunk
// are a line that its warps share evenly, each with a ring of TMA copies
// (codes) and asynchronous copies (scales, zero points) of its own that runs
// on over tiles and chunks, so that nothing but the ends of a chunk makes
// warps wait for one another.  A tile that several warps share is summed by
// the first of them, in the order of k.  With several chunks the sums go
// through `out`.  NB: blocks of 8 activation rows (the MMA's N).
//
// Bound by the instructions that widen codes: a warp takes some 400 for a unit
// (16 x 256 codes: of 32 MMAs, 64 pairs of codes masked, less their zero points,
// a third of them shifted, 8 to 24 reads of activations, and its share of the ring),
// four warps a scheduler issue 0.6 to 0.7 of them a cycle, and half to two
// thirds of the integer pipe's and of shared memory's cycles are taken.  More
// and smaller warps spill (20 warps: 41 us for the first of these).  Measured:
// 24576 x 4096 in groups of 64 with zero points, 16 rows 22.2 us (2.5 TB/s of
// codes, scales and zero points), one row 18.4; 6144 x 4096 in groups of 128,
// one row 6.9; E2M1 codes, 151936 x 4096 in groups of 32, one row 80 us (4.4
// TB/s).  Per-CTA k-groups that stream the activations as well (w4_stream.cu)
// took 32.6, 26.1, 9.3 and 108.
//
// Within a scale group a thread of a quad takes 8 * GROUP / 32 adjacent codes
// (one 4, 8 or 16-byte read), so an MMA adds products of one group only.
template <typename X, bool E2M1, int GROUP, int NB, int SCALE>
__global__ void __launch_bounds__(kW4Threads, 1)
    k_gemm_w4(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ W4Params p) {
  using H = Half2<X>;
  constexpr int SS = SCALE == DFLASH_ELEM_F32 ? 4 : 2;
  constexpr int NG = kW4Unit / GROUP;  // groups of a unit
  constexpr int WPT = GROUP / 32;      // words a thread takes of a group
  constexpr int ZB = NG < 4 ? 4 : NG;  // bytes kept of a row's zero points
  constexpr int SUM = NB * 4 * 33;     // floats of a warp's sums, [4 NB][33]
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int gr = lane >> 2, t4 = lane & 3;
  const bool elected = elect_one();
  uint64_t* full = reinterpret_cast<uint64_t*>(smem) + warp * kW4MaxStages;
  uint64_t* x_full = reinterpret_cast<uint64_t*>(smem) + kW4Warps * kW4MaxStages;
  uint8_t* xs = smem + 1024;
  const uint32_t ring = smem_u32(smem) + (warp < p.low_warps ? p.off_ring + warp * p.stages * 2048
                                                             : p.off_high + (warp - p.low_warps) * p.stages * 2048);
  const int bytes_s = kW4Rows * NG * SS;
  const uint32_t ring_s = smem_u32(smem) + p.off_scale + warp * p.stages * bytes_s;
  const uint32_t ring_z = smem_u32(smem) + p.off_zero + warp * p.stages * (kW4Rows * ZB);
  float* sums = reinterpret_cast<float*>(smem + p.off_sum);

  const int units = (p.K + kW4Unit - 1) / kW4Unit, block = blockIdx.x;
  const int tile0 = p.share * block + min(block, p.extra), tiles = p.share + (block < p.extra ? 1 : 0);
  // warp w's share of a chunk's line of tiles x n units starts at unit share(n, w)
  auto share = [&](int n, int w) { return tiles * n * w / kW4Warps; };
  auto chunk_units = [&](int c) { return min(p.chunk, units - c * p.chunk); };

  if (lane == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 33);  // (the TMA copy's arrival and the lanes')
    mbar_init(&x_full[warp], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();

  bool ok = true;
  // The warp's next unit to fetch.
  int f_chunk = -1, f_n = 0, f_at = 0, f_end = 0, f_tile = 0, f_unit = 0;
  auto f_settle = [&]() {  // on to the next chunk where this one's share is done
    while (f_at == f_end && ++f_chunk < p.chunks) {
      f_n = chunk_units(f_chunk);
      f_at = share(f_n, warp);
      f_end = share(f_n, warp + 1);
      f_tile = f_at / f_n;
      f_unit = f_at - f_tile * f_n;
    }
  };
  f_settle();
  // Lanes 0 .. 15 copy a row's scales each, lanes 16 .. 31 its zero points.
  const bool c_zero = lane >= kW4Rows, c_any = !c_zero || (!E2M1 && p.zero != nullptr);
  const int c_row = lane & (kW4Rows - 1), c_size = c_zero ? 1 : SS, c_piece = c_zero ? p.piece_z : p.piece_s;
  // (of two zero points the aligned four bytes that hold them)
  const int c_bytes = c_zero && NG == 2 && c_piece != 0 ? 4 : NG * c_size;
  const uint32_t c_dst = c_zero ? ring_z + c_row * ZB : ring_s + c_row * (NG * SS);
  const int c_slot = c_zero ? kW4Rows * ZB : bytes_s;
  const uint8_t* c_src = nullptr;  // this lane's row
  auto c_locate = [&]() {
    const long long row = min((tile0 + f_tile) * kW4Rows + c_row, p.N - 1);
    c_src = (c_zero ? p.zero : p.scale) + row * p.groups * c_size;
  };
  bool c_new = true;
  auto fetch = [&](int s) {
    if (c_new) c_locate();
    const int unit = f_chunk * p.chunk + f_unit;
    if (elected) {
      mbar_arrive_expect_tx(&full[s], 2048);
      tma_load_2d_to(ring + s * 2048, &tmW, &full[s], unit * (kW4Unit / 2), (tile0 + f_tile) * kW4Rows);
    }
    if (c_any) {
      const int at = c_zero && NG == 2 && c_piece != 0 ? unit * 2 & ~3 : unit * NG * c_size;
      const int left = p.groups * c_size - at;  // bytes of the row; past the last group: zeros
      const uint32_t dst = c_dst + s * c_slot;
      if (c_piece == c_bytes) {
        copy_async(dst, c_src + at, c_piece, min(left, c_piece));
      } else if (c_piece != 0) {
        for (int o = 0; o < c_bytes; o += c_piece)
          copy_async(dst + o, o < left ? c_src + at + o : c_src, c_piece, o < left ? c_piece : 0);
      } else {
        for (int o = 0; o < c_bytes; o += c_size) {
          const int to = dst + o + (c_zero && NG == 2 ? (unit & 1) * 2 : 0);
          const uint8_t* src = c_src + at + o;
          if (c_size == 4)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(o < left ? *reinterpret_cast<const uint32_t*>(src) : 0u)
                         : "memory");
          else if (c_size == 2)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(to),
                         "h"(o < left ? *reinterpret_cast<const uint16_t*>(src) : uint16_t(0))
                         : "memory");
          else
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(to), "r"(o < left ? static_cast<uint32_t>(*src) : 0u) : "memory");
        }
      }
    }
    copies_arrive(&full[s]);
    ++f_at;
    c_new = ++f_unit == f_n || f_at == f_end;
    if (c_new) {
      f_unit = 0;
      ++f_tile;
      f_settle();
    }
  };
  // A chunk's activations: warps 0 .. M - 1 fetch a row each
  auto fetch_x = [&](int c) {
    const int k0 = c * p.chunk * kW4Unit, bytes = min(chunk_units(c) * kW4Unit, p.K - k0) * 2;
    if (warp < p.M && elected) {
      mbar_arrive_expect_tx(&x_full[warp], bytes);
      bulk_load_global(smem_u32(xs) + warp * p.pitch, p.x + (static_cast<long long>(warp) * p.K + k0) / 8, bytes,
                       &x_full[warp]);
    }
    __syncwarp();
  };
  fetch_x(0);
  int fetched = 0;
  for (; fetched < p.stages && f_chunk < p.chunks; ++fetched) fetch(fetched);

  const uint32_t table = (smem_u32(smem_raw) + kW4Table) & ~(kW4Table - 1u);
  if constexpr (E2M1) {
    for (int e = warp; e < 256; e += kW4Warps) {
      const uint32_t v = H::e2m1x2(e);
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(table + e * 256 + lane * 4), "r"(v) : "memory");
    }
  }
  // two E2M1 codes: byte i of a word
  const uint32_t lane4 = lane * 4 | table >> 8;  // (a byte permutation makes the entry's address)
  auto look_up = [&](uint32_t w, int i) {
    uint32_t v;
    asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(__byte_perm(w, lane4, 0x6504 | i << 4)));
    return v;
  };
  // All warps put the activations in place: within a unit, thread t4's 8 k of word q go
  // to 64 q + 16 t4, as the pairs (k, k + 1) for E2M1, (k, k + 4) for integers
  auto place_x = [&](int c) {
    const int n = chunk_units(c), left = (p.K - c * p.chunk * kW4Unit) / 8 - lane;
    const int g = lane / (GROUP / 8), r = lane % (GROUP / 8), to = (g * WPT + r % WPT) * 64 + r / WPT * 16;
    const int parts = kW4Warps / p.M, part = warp / p.M, m = warp - part * p.M;
    if (part >= parts) return;
    ok = w4_wait(&x_full[m], c & 1, p.status) && ok;
    __syncwarp();
    const uint32_t row = smem_u32(xs) + m * p.pitch;
#pragma unroll 4
    for (int u = part; u < n; u += parts) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (u * 32 < left) v = lds128(row + u * 512 + lane * 16);
      if constexpr (!E2M1)
        v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                       __byte_perm(v.y, v.w, 0x7632));
      __syncwarp();
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + u * 512 + to), "r"(v.x), "r"(v.y), "r"(v.z),
                   "r"(v.w)
                   : "memory");
    }
  };
  __syncthreads();  // (the barriers of the activations are set up)
  place_x(0);
  __syncthreads();  // the activations (and the table) are there

  // (rows past M are not kept: their columns of the sums are not either)
  uint32_t xrow[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) xrow[j] = smem_u32(xs) + min(j * 8 + gr, p.M - 1) * p.pitch + t4 * 16;
  const bool xlast = (NB - 1) * 8 + gr < p.M;
  // where a thread finds its codes: rows of 128 bytes, 16-byte pieces swizzled by the row
  int woff[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int o = g * (GROUP / 2) + t4 * WPT * 4;
    woff[g] = gr * 128 + (((o >> 4) ^ gr) << 4) + (o & 15);
  }

  int s = 0;
  uint32_t parity = 0;
  for (int c = 0; c < p.chunks; ++c) {
    const int n = chunk_units(c), end = share(n, warp + 1);
    int at = share(n, warp), tile = at / n, unit = at - tile * n;
    float acc[NB][4];
    // the sums of tile `t` into out
    auto leave = [&](int t) {
      const int row = (tile0 + t) * kW4Rows + gr;
      float* o = p.out + 2ll * t4 * p.N + row;
#pragma unroll
      for (int j = 0; j < NB; ++j, o += 8ll * p.N)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j * 8 + 2 * t4 + (e & 1) < p.M && row + (e >> 1) * 8 < p.N) {
            float* to = o + (e & 1 ? p.N : 0) + (e >> 1) * 8;
            *to = acc[j][e] * (E2M1 ? 1.f : H::kSum) + (c > 0 ? *to : 0.f);
          }
    };
    bool open = false;  // a tile that this warp begins and others end
    while (at < end) {
      const int u0 = unit, u1 = min(n, unit + end - at);
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
      for (; unit < u1; ++unit, ++at) {
        ok = ok && w4_wait(&full[s], parity, p.status);
        __syncwarp();  // (elements that were copied one by one)
        const uint32_t ws = ring + s * 2048, xu = unit * 512;
        // the unit's scales
        float sc[2][NG];
        const uint32_t at_s = ring_s + s * bytes_s + gr * (NG * SS), next_s = 8 * NG * SS;
        auto scales16 = [&](auto&& as_float) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[NG / 2];
            lds(at_s + h * next_s, w);
#pragma unroll
            for (int g = 0; g < NG; ++g) sc[h][g] = as_float(w[g / 2], g & 1);
          }
        };
        if constexpr (SCALE == DFLASH_ELEM_BF16)
          scales16([](uint32_t w, int hi) { return __uint_as_float(hi ? w & 0xffff0000u : w << 16); });
        else if constexpr (SCALE == DFLASH_ELEM_F16)
          scales16([](uint32_t w, int hi) {
            return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> (16 * hi))));
          });
        else
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[NG];
            lds(at_s + h * next_s, w);
#pragma unroll
            for (int g = 0; g < NG; ++g) sc[h][g] = __uint_as_float(w[g]);
          }
        uint32_t z[2][ZB / 4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int g = 0; g < ZB / 4; ++g) z[h][g] = 0x08080808u;
          if (!E2M1 && p.zero != nullptr) {
            lds(ring_z + s * (kW4Rows * ZB) + (gr + h * 8) * ZB, z[h]);
            if (NG == 2) z[h][0] >>= ((c * p.chunk + unit) & 1) * 16;
          }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint32_t word[2][WPT];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            lds(ws + woff[g] + h * 1024, word[h]);
          }
          float d[NB][4];
#pragma unroll
          for (int w = 0; w < WPT; ++w) {
            uint32_t a[2][4];  // [k half][row half + 2 x k quarter]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[4];
              if constexpr (E2M1) {
#pragma unroll
                for (int i = 0; i < 3; ++i) v[i] = look_up(word[h][w], i);
                v[3] = H::e2m1x2(word[h][w] >> 24);
              } else {
                H::widen(word[h][w], H::bias(z[h][g / 4], g & 3), v);
              }
              a[0][h] = v[0];
              a[0][2 + h] = v[1];
              a[1][h] = v[2];
              a[1][2 + h] = v[3];
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              // (lanes of rows past M read nothing: a read takes as long as the lanes that take part)
              uint4 v = make_uint4(0, 0, 0, 0);
              if (!E2M1 || j < NB - 1 || xlast) v = lds128(xrow[j] + xu + (g * WPT + w) * 64);
              if (w == 0) H::mma0(d[j], a[0], v.x, v.y);
              else H::mma(d[j], a[0], v.x, v.y);
              H::mma(d[j], a[1], v.z, v.w);
            }
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            acc[j][0] += sc[0][g] * d[j][0];
            acc[j][1] += sc[0][g] * d[j][1];
            acc[j][2] += sc[1][g] * d[j][2];
            acc[j][3] += sc[1][g] * d[j][3];
          }
        }
        __syncwarp();
        if (ok && f_chunk < p.chunks) {
          fetch(s);
          ++fetched;
        }
        if (++s == p.stages) {
          s = 0;
          parity ^= 1;
        }
      }
      if (u0 > 0) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sums[warp * SUM + (j * 4 + e) * 33 + lane] = acc[j][e];
      } else if (u1 == n) {
        leave(tile);
      } else {
        open = true;
      }
      if (u1 == n) {
        unit = 0;
        ++tile;
      }
    }
    __syncthreads();  // the warps' sums are there, and the activations done with
    if (open) {
      for (int w = warp + 1; w < kW4Warps; ++w) {
        const int a0 = share(n, w);
        if (a0 >= (tile + 1) * n) break;
        if (a0 == share(n, w + 1)) continue;
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] += sums[w * SUM + (j * 4 + e) * 33 + lane];
      }
      leave(tile);
    }
    if (c + 1 < p.chunks) {
      fence_proxy_async_smem();
      fetch_x(c + 1);
      place_x(c + 1);
      __syncthreads();
    }
  }
  if (!ok) {  // a wait gave up: copies still in flight get bounded waits before the CTA leaves
    if (warp < p.M) w4_wait(&x_full[warp], (p.chunks - 1) & 1, p.status);
    for (int i = max(0, fetched - p.stages); i < fetched; ++i)
      w4_wait(&full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1, p.status);
  }
}

template <typename X, bool E2M1, int GROUP, int NB, int SCALE>
cudaError_t launch_w4_n(const W4Args& a, cudaStream_t s) {
  constexpr int NG = kW4Unit / GROUP, ZB = NG < 4 ? 4 : NG;
  W4Params p{};
  p.scale = a.scale;
  p.zero = a.zero;
  p.x = static_cast<const uint4*>(a.x);
  p.out = a.out;
  p.status = a.status;
  p.N = a.N;
  p.K = a.K;
  p.groups = a.groups;
  p.M = a.M;
  CUtensorMap tw;
  if (!w4_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.W, p.N, p.K / 2, kW4Rows, kW4Unit / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  p.piece_s = w4_piece(NG * a.scale_size, static_cast<long long>(p.groups) * a.scale_size, p.scale);
  p.piece_z = w4_piece(ZB, p.groups, p.zero);
  // Where things lie in shared memory, with `stages` units in flight per warp
  // beside the activations of n units.  (The E2M1 table takes a multiple of 64
  // KB; what is before it and behind it are two places.)
  const int units = (p.K + kW4Unit - 1) / kW4Unit;
  const auto lay_out = [&](int stages, int n) {
    int at[2] = {1024, kW4Smem}, end[2] = {kW4Smem, kW4Smem};
    if (E2M1) {
      end[0] = kW4Table - kW4Reserved;
      at[1] = end[0] + kW4Table;
    }
    bool fits = true;
    const auto take = [&](int bytes, int first) {
      bytes = (bytes + 1023) / 1024 * 1024;
      const int k = end[first] - at[first] >= bytes ? first : 1 - first;
      fits = fits && end[k] - at[k] >= bytes;
      const int o = at[k];
      at[k] += bytes;
      return o;
    };
    const int ring = stages * 2048;
    p.low_warps = E2M1 ? kW4Warps - std::min(kW4Warps, (end[1] - at[1]) / ring) : kW4Warps;
    p.off_high = at[1];
    at[1] += (kW4Warps - p.low_warps) * ring;
    if (take(p.M * (n * 512 + 64), 0) != 1024) fits = false;
    p.off_ring = take(p.low_warps * ring, 0);
    if (p.low_warps > 0 && p.off_ring >= end[0]) fits = false;
    p.off_sum = take(kW4Warps * NB * 4 * 33 * 4, 1);
    p.off_scale = take(kW4Warps * stages * kW4Rows * NG * a.scale_size, 1);
    p.off_zero = p.zero != nullptr ? take(kW4Warps * stages * kW4Rows * ZB, 1) : 0;
    p.stages = stages;
    p.chunk = n;
    p.pitch = n * 512 + 64;
    return fits;
  };
  // the activations of all of k if two units in flight fit beside them, else of a part of k
  const auto plan = [&]() {
    for (int stages = kW4MaxStages; stages >= 2; --stages)
      if (lay_out(stages, units)) return true;
    for (int least = 2; least >= 1; --least)
      for (int stages = kW4MaxStages; stages >= 2; --stages) {
        if (!lay_out(stages, least)) continue;
        int most = least;
        while (lay_out(stages, most + 1)) ++most;
        const int chunks = (units + most - 1) / most;
        return lay_out(stages, (units + chunks - 1) / chunks);
      }
    return false;
  };
  if (!plan()) return cudaErrorInvalidConfiguration;
  p.chunks = (units + p.chunk - 1) / p.chunk;
  const int all = (p.N + kW4Rows - 1) / kW4Rows, ctas = std::min(all, a.sms);
  p.share = all / ctas;
  p.extra = all % ctas;
  static FuncAttr attr;
  const cudaError_t e = attr.ensure(kW4Smem, [](int v) {
    return cudaFuncSetAttribute(k_gemm_w4<X, E2M1, GROUP, NB, SCALE>, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
  });
  if (e != cudaSuccess) return e;
  return launch_k(k_gemm_w4<X, E2M1, GROUP, NB, SCALE>, dim3(ctas), dim3(kW4Threads),
                  kW4Smem, s, dim3(1), false, tw, p);
}

template <typename X, bool E2M1, int GROUP, int NB>
cudaError_t launch_w4_s(const W4Args& a, cudaStream_t s) {
  if (a.scale_elem == DFLASH_ELEM_F32) return launch_w4_n<X, E2M1, GROUP, NB, DFLASH_ELEM_F32>(a, s);
  if (a.scale_elem == DFLASH_ELEM_BF16) return launch_w4_n<X, E2M1, GROUP, NB, DFLASH_ELEM_BF16>(a, s);
  return launch_w4_n<X, E2M1, GROUP, NB, DFLASH_ELEM_F16>(a, s);
}

template <typename X, bool E2M1, int GROUP>
cudaError_t launch_w4_g(const W4Args& a, cudaStream_t s) {
  return a.M <= 8 ? launch_w4_s<X, E2M1, GROUP, 1>(a, s) : launch_w4_s<X, E2M1, GROUP, 2>(a, s);
}

template <typename X, bool E2M1>
cudaError_t launch_w4_x(const W4Args& a, cudaStream_t s) {
  int dev = 0, reserved = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e != cudaSuccess) return e;
  if (reserved != kW4Reserved) return cudaErrorInvalidConfiguration;
  if (a.group == 32) return launch_w4_g<X, E2M1, 32>(a, s);
  if (a.group == 64) return launch_w4_g<X, E2M1, 64>(a, s);
  return launch_w4_g<X, E2M1, 128>(a, s);
}

}  // namespace

}  // namespace dflash
