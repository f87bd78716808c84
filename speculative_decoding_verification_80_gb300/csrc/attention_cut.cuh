// attention_cut.cuh — how spec_attention's list of tiles is cut into equal
// parts, one for each CTA.  Host and device: the test of the cut compiles it
// without nvcc.
//
// The list is cut by cost: a tile costs 4 to 6 units by its rows' 16s, and an
// item (a row group of a head) kItemCost more, half before and half after its
// tiles.  (Measured when the costs were set: 0.64, 0.72 and 0.98 us a tile of
// 16, 32 and 48 rows of D = 128, 2 us an item; a tile takes 0.67, 0.74 and 1.09
// now.)  A cut within an item falls between tiles; one near
// its start or end moves there, so the CTAs at an item's ends may have units of
// it and no tile: as many as two at its start, since its first tile ends at
// kItemCost / 2 + 6 units and a CTA's part may be kLeastCost.  (An item's cost
// of 12, 20, 32 and 44 units: 158, 160, 163 and 167 us on 64 requests, 64, 62,
// 63 and 62 us on one long one, 296, 299, 309 and 312 us on 256.)
#pragma once
#include <stdint.h>

#if defined(__CUDACC__)
#define SPECDEC_CUT_FN __host__ __device__ __forceinline__
#else
#define SPECDEC_CUT_FN inline
#endif

namespace specdec {

constexpr int kItemCost = 12;
constexpr int kMostTileCost = 6;
constexpr int kLeastCost = 10;  // of a CTA's part
static_assert(kLeastCost >= kMostTileCost, "between two CTAs with tiles of an item there is none without");

SPECDEC_CUT_FN uint32_t tile_cost(int rows) { return rows <= 32 ? 4 : (rows <= 48 ? 5 : kMostTileCost); }

// Tiles of an item that lie before `cost` units of it.
SPECDEC_CUT_FN int tiles_before(uint32_t cost, uint32_t per_tile, int tiles) {
  if (cost <= kItemCost / 2) return 0;
  const uint32_t n = (cost - kItemCost / 2) / per_tile;
  return n < static_cast<uint32_t>(tiles) ? static_cast<int>(n) : tiles;
}

// The CTAs that have tiles of the item of units [first, end), first to last of
// them, and the one that its first unit falls to; `chunk` units go to each.
struct ItemCtas {
  uint32_t home, c0, c1;
};
SPECDEC_CUT_FN ItemCtas item_ctas(uint32_t first, uint32_t end, uint32_t per_tile, int tiles, uint32_t chunk) {
  ItemCtas p;
  p.home = p.c0 = first / chunk;
  p.c1 = (end - 1) / chunk;
  while (p.c0 < p.c1 && tiles_before((p.c0 + 1) * chunk - first, per_tile, tiles) == 0) ++p.c0;
  while (p.c1 > p.c0 && tiles_before(p.c1 * chunk - first, per_tile, tiles) == tiles) --p.c1;
  return p;
}

}  // namespace specdec
