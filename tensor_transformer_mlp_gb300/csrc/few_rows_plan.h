// How the products of few tokens (gemm_few_rows.cu) are cut into tiles and splits, and when they are taken instead of the SM-pair
// GEMM: sizes in, a Plan out. Plain C++, so that the choice can be looked at without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#ifdef __CUDACC__
#define TPMLP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TPMLP_HOST_DEVICE inline
#endif

namespace tpmlp {
namespace few_rows {

constexpr int kTileCols = 256;          // weight columns of a tile: two blocks of 128
constexpr int kBlock = 128;
constexpr int kBK = 64;
constexpr int kMaxTokens = 256;         // tokens of a tile
constexpr int kWeightBytes = kTileCols * kBK * 2;
constexpr int kBoxBytes = 64 * kBK * 2;  // one 64 x 64 box of weights stored [K][cols]
constexpr int kMaxStages = 6;
constexpr int kSmemBudget = 220 * 1024;
constexpr int kBarrierBytes = 256;
constexpr int kSms = 152;               // what splits and workspaces are chosen for, with or without a device

struct Plan {
  int n, cols, num_kb;   // tokens, output columns (of Y for the gate), k-blocks
  int nt, token_tiles;   // tokens of a tile (a multiple of 16, on a pair of 32) and tiles of them
  int col_tiles, tiles, splits, items, ctas;  // items = tiles * splits
  int shard, unit;       // the gated block's columns (EpiParams), 0: plain
  int ranks;             // CTAs of a tile: 2 are a pair of SMs that take half of the tokens in each (FC1 with one split)
  int stages;
};

TPMLP_HOST_DEVICE int plan_stage_bytes(const Plan& p) { return kWeightBytes + p.nt / p.ranks * kBK * 2; }

// Tile -> its first column (and token: tile % token_tiles). Tiles of the same columns are neighbours: their weights meet in L2. A
// CTA of a tile takes 256 columns of the weights: 256 of the output, or 128 (gate and up) of Y.
TPMLP_HOST_DEVICE int cta_columns(const Plan& p) { return p.shard ? kBlock : kTileCols; }
TPMLP_HOST_DEVICE int tile_column(const Plan& p, int tile) {
  const int ct = tile / p.token_tiles, w = cta_columns(p) * p.ranks;
  if (!p.shard) return ct * w;
  const int per = (p.unit + w - 1) / w;
  return ct / per * p.unit + ct % per * w;
}

// Estimated time of a product, in us: rounds of items, each k-block at the slowest of the weights' share of HBM (7.2 TB/s, what
// reads alone reach), an SM's weights from HBM (70 KB a us) and all that it takes in (110), and the tensor core (15 TFLOP/s
// an SM); what a launch (FC1: no kernel in front) and a round cost beside the k-blocks; the shares' way to L2 and back
// (9.3 TB/s) and the second kernel. Measured / estimated:
//   FC1, one split, m16384: d1024, 4 tokens 18.0 / 17.7, 200 22.4 / 24.9; d4096, 4 46 / 46, 64 46 / 47, 128 48 / 49, 200 51 / 53,
//   256 52 / 54; d8192, 4 84 / 82, 200 88 / 90, 256 91 / 91; d4096 m11008, 200 45 / 47
//   splits, from the end of the kernel in front: 4 tokens K16384 4096 columns, 4 splits 37 / 36, 8 27 / 26, 9 28 / 25; 200
//   tokens there, 5 40 / 42, 9 33 / 34; n512 K8192 1024 columns, 4 29 / 27, 9 22 / 21, 19 21 / 22; 37 tokens K4096, 19 9 / 9
inline double plan_time(const Plan& p) {
  const double ctas = static_cast<double>(p.items) * p.ranks, busy = std::min<double>(ctas, kSms);
  const double kb = std::max({kWeightBytes * busy / 7.2e6, kWeightBytes / 70e3, plan_stage_bytes(p) / 110e3, 2.0 * kTileCols * p.nt * kBK / 15e6});
  const double rounds = std::ceil(ctas / kSms), blocks = std::ceil(static_cast<double>(p.num_kb) / p.splits);
  if (p.splits == 1) {
    const double tokens = p.ranks == 1 ? std::max(0, p.nt - kBlock) * 7e-4 : 0.0;  // beyond 128 a ring of 3 stages falls behind
    return rounds * (blocks * (kb + tokens) + 3.3 + p.nt / 30.0) + 4.5 + (p.ranks - 1) * 0.3;
  }
  return rounds * (blocks * kb + 2.5 + p.nt / 100.0) + 3.8 + (p.shard ? 5.0 : 0.0) + ctas * p.nt * kTileCols * 8.0 / 9.3e6;
}

// The plan with the least estimated time over the number of splits and, for FC1 without a split, single CTAs and pairs (whose split
// sums were slower than single CTAs' at every size: n200 K16384 4096 columns 34.9 us against 33.2, n512 K8192 1024 columns 22.8
// against 21.0).
inline Plan make_plan(int64_t n, int64_t cols, int64_t k, int64_t m, int t, bool gate) {
  Plan best{};
  double best_time = 0;
  for (int ranks = 1; ranks <= (gate ? 2 : 1); ++ranks) {
    Plan p{};
    p.n = static_cast<int>(n);
    p.cols = static_cast<int>(cols);
    p.num_kb = static_cast<int>((k + kBK - 1) / kBK);
    p.token_tiles = static_cast<int>((n + kMaxTokens - 1) / kMaxTokens);
    // the tensor core's instruction takes N in steps of 16 (M = 128, one SM) or of 32 (M = 256, a pair)
    const int64_t step = 16 * ranks;
    p.nt = static_cast<int>(((n + p.token_tiles - 1) / p.token_tiles + step - 1) / step * step);
    p.ranks = ranks;
    if (gate) {
      p.shard = static_cast<int>(m / t);
      p.unit = p.shard % 64 == 0 ? static_cast<int>(m) : p.shard;
    }
    const int64_t w = static_cast<int64_t>(cta_columns(p)) * ranks;
    p.col_tiles = static_cast<int>(gate ? m / p.unit * ((p.unit + w - 1) / w) : (cols + w - 1) / w);
    p.tiles = p.col_tiles * p.token_tiles;
    p.stages = std::min<int>(kMaxStages, (kSmemBudget - kBarrierBytes - 1024) / plan_stage_bytes(p));
    // one split, and the numbers that fill one, two and three waves of CTAs or parts of the first
    const int wave = kSms / (p.tiles * ranks);
    for (const int splits : {1, wave / 4, wave / 2, 3 * wave / 4, wave - 1, wave, 2 * kSms / (p.tiles * ranks), 3 * kSms / (p.tiles * ranks)}) {
      p.splits = std::min(splits, p.num_kb);
      if (p.splits < 1 || (p.splits > 1 && ranks > 1)) continue;
      p.items = p.tiles * p.splits;
      const double time = plan_time(p);
      if (best.tiles == 0 || time < best_time) {
        best = p;
        best_time = time;
      }
    }
  }
  return best;
}

inline size_t slot_bytes(const Plan& p) {
  return p.splits > 1 ? static_cast<size_t>(p.items) * p.nt * kTileCols * sizeof(float) : 0;
}

// Against the SM-pair GEMM (gemm_tc.cu): for each wave of 256 x 256 accumulators over 76 pairs some 0.32 us a k-block (FC1:
// 0.35, 0.29 in a single wave) beside 6 us (7.5). Measured here and there:
//   FC1, m16384: d4096, 4 tokens 46 and 64 us, 64 46 and 52, 128 48 and 51, 200 51 and 51, 256 52 and 51; d1024, 4 18 and 25,
//   128 20 and 19.6, 200 22 and 20; d8192, 200 88 and 96; m4096 d4096, 4 21 and 25.5, 64 24 and 26, 200 29 and 26; a forward of
//   d8192 m8448 in 32 ragged shards, 4 tokens 95 and 121, 128 100 and 121
//   others: n200 K16384 4096 columns 33 and 87, n512 1024 columns K4096 19 and 24, K8192 21 and 43, n1111 1000 columns K2736 18
//   and 20
inline bool pays(const Plan& p, int64_t pair_tiles) {
  const double waves = std::ceil(static_cast<double>(pair_tiles) / (kSms / 2)), blocks = p.num_kb * waves;
  return plan_time(p) < (p.shard ? 7.5 + (waves > 1 ? 0.35 : 0.29) * blocks : 6.0 + 0.32 * blocks);
}

inline bool gemm_pays(int64_t n, int64_t cols, int64_t k) {
  const int64_t tiles = (n + 255) / 256 * ((cols + 255) / 256);
  return tiles <= kSms && pays(make_plan(n, cols, k, 0, 1, false), tiles);
}
inline bool gated_fc1_pays(int64_t n, int64_t d, int64_t m, int t) {
  if (n > kMaxTokens) return false;
  const Plan p = make_plan(n, m, d, m, t, true);
  return pays(p, m / p.unit * ((p.unit + kBlock - 1) / kBlock));  // that GEMM's tiles divide runs of `unit` columns too
}

}  // namespace few_rows
}  // namespace tpmlp
