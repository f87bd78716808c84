// Test helper (host code): replays the cut of spec_attention's list of tiles
// (csrc/attention_cut.cuh) and compares the CTAs that have tiles of an item with
// those that the join expects.
#include "attention_cut.cuh"

using namespace specdec;

// One item whose first unit is `first`; 0 where all is well, else what is not.
extern "C" int cut_of_item(uint32_t first, int rows, int tiles, uint32_t chunk) {
  const uint32_t per_tile = tile_cost(rows), cost = tiles * per_tile + kItemCost, end = first + cost;
  const ItemCtas on = item_ctas(first, end, per_tile, tiles, chunk);
  if (on.home != first / chunk) return 1;
  int done = 0;
  uint32_t c0 = 0, c1 = 0;
  for (uint32_t c = first / chunk; c * chunk < end; ++c) {
    const uint32_t from = c * chunk > first ? c * chunk - first : 0, to = (c + 1) * chunk - first;
    const int tile0 = tiles_before(from, per_tile, tiles), tile1 = tiles_before(to < cost ? to : cost, per_tile, tiles);
    if (tile0 >= tile1) continue;
    if (tile0 != done) return 2;            // a tile of no one, or of two
    if (done > 0 && c != c1 + 1) return 3;  // the records of a join are neighbours'
    if (done == 0) c0 = c;
    c1 = c;
    done = tile1;
  }
  if (done != tiles) return 4;
  return on.c0 == c0 && on.c1 == c1 ? 0 : 5;
}

// All items of 1 to `most_tiles` tiles, from every unit of a CTA's part, for parts of
// kLeastCost to `most_chunk` units: how many fail; `where` gets the first.
extern "C" long long cut_of_all(int most_tiles, uint32_t most_chunk, int* where) {
  long long bad = 0;
  for (uint32_t chunk = kLeastCost; chunk <= most_chunk; ++chunk)
    for (int rows = 16; rows <= 64; rows += 16)
      for (int tiles = 1; tiles <= most_tiles; ++tiles)
        for (uint32_t first = 3 * chunk; first < 4 * chunk; ++first)
          if (const int what = cut_of_item(first, rows, tiles, chunk)) {
            if (bad++ == 0) where[0] = static_cast<int>(first), where[1] = rows, where[2] = tiles, where[3] = static_cast<int>(chunk), where[4] = what;
          }
  return bad;
}
