// How a product of two microscaled 4-bit matrices is cut into tiles, CTAs,
// stages and TMEM columns (fp4_gemm.cu).  Plain host code, without CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

namespace dflash {

constexpr int kOutWarps = 8;            // that read accumulators out, two a quarter of the lanes
constexpr int kOutRows = 32;            // rows of out a block
constexpr int kFp4Smem = 232448;
constexpr int kFp4Head = 232;           // bytes of the barriers in front of the ring
constexpr int kRows = 128;              // rows of W a tile
constexpr int kMaxBn = 256;             // the MMA's; scales from two tiles
constexpr int kCodeRow = 128;           // bytes of 256 codes
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;

struct Fp4Plan {
  int bn, m_tiles, split, stages, smem, second, shared_last, shared_first, sc_first, cols, x_tiles, blocks;
  unsigned grid;
  bool pair;
};

// Rows of X a tile, CTAs a tile, stages: the cheapest by a rough count of cycles.
// clusters(n): how many clusters of n CTAs run at once on `sms` SMs.
template <typename Clusters>
Fp4Plan fp4_plan(bool nv, int M, int N, int kt, int sms, int out_size, Clusters&& clusters) {
  const int chunks = nv ? 4 : 2;
  const long long n_tiles = (N + kRows - 1) / kRows;
  Fp4Plan best{};
  double best_cost = 0;
  const auto consider = [&](int bn, int split, bool pair) {
    const long long m_tiles = (M + bn - 1) / bn, tiles = (pair ? (n_tiles + 1) / 2 : n_tiles) * m_tiles;
    if (split > 1 && tiles * split > 4ll * sms) return;
    Fp4Plan c{};
    c.bn = bn;
    c.m_tiles = static_cast<int>(m_tiles);
    c.split = split;
    c.pair = pair;
    // 128-row scale tiles that BN rows lie in, wherever they start
    const int at = m_tiles > 1 ? 128 - std::min(128, bn & -bn) : 0;
    c.x_tiles = (at + bn + 127) / 128;
    if (pair && c.x_tiles != 2) return;
    const int own = pair ? bn / 2 : bn;
    const int stage = (kRows * kCodeRow + own * kCodeRow + chunks * 512 * (1 + c.x_tiles) + 1023) & ~1023;
    // (a second block of out a warp, so that a copy is read while the next is written, where it costs no stage)
    const int block = kOutWarps * kOutRows * 32 * out_size, room = kFp4Smem - 1024 - kFp4Head;
    c.stages = std::min(kMaxStages, (room - block) / stage);
    c.blocks = std::min(kMaxStages, (room - 2 * block) / stage) == c.stages ? 2 : 1;
    const int fixed = kFp4Smem - room + c.blocks * block;
    // Two accumulators where a CTA has several tiles; where they do not fit beside the scales they share columns.
    const int sets = c.stages * chunks * 4 * (1 + c.x_tiles);
    const int team = pair ? 2 : split;
    const long long at_once = team == 1 ? sms : clusters(team), rounds = (tiles + at_once - 1) / at_once;
    const bool one = split > 1 || tiles <= at_once;
    c.sc_first = one ? bn : std::min(2 * bn, 512 - sets);
    c.second = one ? 0 : c.sc_first - bn;
    // The second one's blocks of 32 columns that lie on the first one's last columns, and the first one's on which they
    // lie: one more where the first one's last block is a half (bn = 240: columns 80 to 239, blocks 0 to 4 and 7 to 2).
    const bool overlap = !one && c.second < bn;
    c.shared_first = overlap ? (bn - c.second + kOutRows - 1) / kOutRows : 0;
    c.shared_last = overlap ? (bn + kOutRows - 1) / kOutRows - c.second / kOutRows : 0;
    c.cols = 32;
    while (c.cols < c.sc_first + sets) c.cols *= 2;
    if (c.sc_first < bn || c.cols > 512 || (split > 1 && bn * kRows * 4 > c.stages * stage)) return;
    c.smem = fixed + c.stages * stage;
    c.grid = static_cast<unsigned>((split > 1 ? tiles : std::min(tiles, at_once)) * team);
    // (16 x 6144 x 4096: one CTA a tile 6.8 us, two 6.2, three, whose clusters do not run all at once, 10.6; 17 x 2560 x 9728: one
    // 11.8, five 6.5)
    // a stage: issuing it, shared memory's reads and writes, W's bytes from memory (once for all tiles beside each other)
    const double per_k =
        std::max({500., (4. * (4096 + 32 * own) + stage) / 128, 17408. / (23. * std::min<long long>(m_tiles, 8))});
    double cost = 1500 + rounds * per_k * ((kt + split - 1) / split) + 300 + 8. * bn + (pair ? 1000 : 0);
    cost += (rounds - 1) * (c.shared_first + 1) / 2 * 500.;
    if (split > 1) cost += 1500 + (rounds - 1) * 2000 + 10. * bn;
    if (best.bn == 0 || cost < best_cost) best = c, best_cost = cost;
  };
  for (int bn = 16; bn <= kMaxBn && bn < M + 16; bn += 16) {
    // (a column of X's scales holds 32 rows, and the MMA takes them from an even column on)
    if (bn < M && bn % 64) continue;
    for (int split = 1; split <= kMaxSplit && split <= kt; ++split) consider(bn, split, false);
  }
  // (the lines of the scales are counted in 32 bits)
  const bool lines = std::max<long long>(n_tiles + 2, M / kRows + 4) * kt * 8 < INT32_MAX;
  for (int bn = 192; bn <= kMaxBn && lines && n_tiles > 1 && M > bn - 64; bn += 64) consider(bn, 1, true);
  return best;
}

}  // namespace dflash
