// int8_plan.cuh — which form a product of moe_int8_product takes, and the layout of its
// workspace: host code from the sizes alone, without CUDA headers.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {
namespace i8 {

constexpr int BK = 128;              // K per stage: 128 bytes = one swizzle row
constexpr int PAIR_ROWS = 256;       // rows of one MMA of a CTA pair
constexpr int kMaxExperts = 1024;
constexpr int kMaxCtas = 160;        // product CTAs at most (workspace sizing; 148 SMs on B200)
// Split form: CTAs per tile, and the clusters of that many that run at once with a margin
// of one (one CTA per SM: 15, 22, 26, 33, 45 and 74 fit on the eight GPCs of a B200). One
// cluster more is a second wave: 16 x 4096 x 4096, 16 tiles in clusters of 8: 18 us, of 4: 9.
constexpr int kSplits[6][2] = {{8, 14}, {6, 21}, {5, 25}, {4, 32}, {3, 44}, {2, 73}};

// Tile schedule in the workspace, made by the prepare kernel.
struct Sched {
  int32_t off[kMaxExperts + 1];  // first row of each expert, and the end of the last one
  int32_t pre[kMaxExperts + 1];  // row tiles before each expert, and all of them
};

struct Layout {
  size_t status, sched, counters, q, a, part, total;
  int32_t tile_rows;  // rows of a tile: 64 or 128 (stream and split form), 256 or 512 (pair form)
  int32_t split;      // CTAs per tile of the split form, 0: another form
};

// Row tiles of `rows` rows that R rows of n experts make: exact for one expert, else the
// expectation for counts close to normal with mean and variance R / n.
inline double row_tiles(int64_t R, int32_t n, int rows) {
  if (n == 1) return static_cast<double>((R + rows - 1) / rows);
  const double m = static_cast<double>(R) / n, sd = std::sqrt(m);
  double total = 0.0, weight = 0.0;
  for (int i = -40; i <= 40; ++i) {
    const double z = i / 10.0, c = std::max(m + z * sd, 0.0), w = std::exp(-0.5 * z * z);
    total += w * std::ceil(c / rows);
    weight += w;
  }
  return n * total / weight;
}

// Pair form: whether tiles of 512 rows end sooner than tiles of 256. In units of one
// 256-row tile: a full tall tile takes 1.76, one with rows in its first half alone 1.15 (a
// shorter ring); a wave counts half of its last tile as lost, and fewer tiles than
// pairs take one tile's time. Measured, us, 512 against 256: Grok-1 gate/up, 287, 437
// and 1024 rows per expert 1117 and 1238, 1140 and 1248, 2184 and 2382; 256 rows 753 and
// 712; down, 437 and 525 rows 561 and 616, 950 and 852; 571 x 8400 x 304 gated, 104 and 67.
inline bool tall_tiles(int64_t R, int32_t n, int64_t nt) {
  constexpr double kPairs = 74.0, kFull = 1.76, kHalf = 1.15;
  const double t256 = row_tiles(R, n, 256) * nt, t512 = row_tiles(R, n, 512) * nt;
  const double full = t256 - t512, half = t512 - full;
  const double low = t256 <= kPairs ? 1.0 : t256 / kPairs + 0.5;
  const double tall = t512 <= kPairs ? kFull : (full * kFull + half * kHalf) / kPairs + 0.5 * kFull;
  return tall < low;
}

// Which form, from the sizes alone (the rows of each expert are only known on the device):
// - split form if the tiles there can be at most leave room for two CTAs or more each (us,
//   split against stream or pair form: 16 x 4096 x 4096 9.0 and 11.6, 64 rows 10.7 and
//   20-25, 128 rows 13.1 and 28-39, 333 rows 18.4 and 33.8), unless few CTAs would have
//   long runs (16 x 14336 x 4096: 28 K blocks on 64 CTAs 19.2, stream form 17.5);
// - else by the rows an expert has on average: up to 48 the stream form in tiles of 64, up
//   to 128 in tiles of 128, above them the pair form in tiles of 256 or 512. Measured at
//   the Grok-1 shape, gate/up and down, us: 128 rows per expert, stream 612 and 259, pair
//   698 and 339; 192 rows, gate/up, stream 1078, pair 705.
inline Layout plan(int64_t R, int64_t K, int64_t N, int32_t n_experts, moe_dtype_t x_dtype, bool dual) {
  Layout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  const int64_t kb = (K + BK - 1) / BK, nt = (N + (dual ? 127 : 255)) / (dual ? 128 : 256);
  L.tile_rows = R <= 48 * static_cast<int64_t>(n_experts) || R <= 64 ? 64 : 128;
  // an expert's last tile may be short: at most one more row tile for each but one
  const int64_t tiles = std::min<int64_t>(R, (R + L.tile_rows - 1) / L.tile_rows + n_experts - 1) * nt;
  for (const auto& s : kSplits)
    if (L.split == 0 && tiles <= s[1] && kb >= 2 * s[0]) L.split = s[0];
  if (L.split > 0 && tiles * L.split < 96 && kb > 24 * L.split && R <= 128 * static_cast<int64_t>(n_experts))
    L.split = 0;
  if (L.split == 0 && R > 128 * static_cast<int64_t>(n_experts))
    L.tile_rows = tall_tiles(R, n_experts, nt) ? 2 * PAIR_ROWS : PAIR_ROWS;
  L.status = take(256);
  L.sched = take(sizeof(Sched));
  L.counters = take(sizeof(int32_t) * kMaxCtas);
  if (x_dtype != MOE_INT8) {
    L.q = take(static_cast<size_t>(R) * K);
    L.a = take(sizeof(float) * R);
  }
  L.part = o;
  if (L.tile_rows < PAIR_ROWS && L.split == 0) take(sizeof(int32_t) * 2 * kMaxCtas * 256 * static_cast<size_t>(L.tile_rows));
  L.total = o;
  return L;
}

}  // namespace i8
}  // namespace moe
