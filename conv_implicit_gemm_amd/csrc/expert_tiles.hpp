// expert_tiles.hpp -- the integer arithmetic of the search for a block's tile
// of rows grouped by expert, for the host and the device alike.
//
// The offsets come from device memory and may hold anything.  Whatever they
// hold, a tile that these functions hand out lies inside its expert's rows, and
// those lie inside [0, T): a block either gets such a tile or none.
#pragma once

#include <stdint.h>

namespace ox {

// n / d rounded up, for 0 <= n < 2^31 and a small d: the sum needs the 32nd bit.
constexpr int ceil_div(int n, int d) { return (int)(((uint32_t)n + (uint32_t)d - 1) / (uint32_t)d); }

struct ExpertTile {
  int e, row0, rows;   // expert, first row of the tile, rows in it (<= BM)
};

// The most row tiles that offsets which do not decrease can give: T / BM full
// ones and one partial tile for every expert with rows.
constexpr int64_t expert_tile_bound(int64_t T, int64_t E, int BM) { return T / BM + (E < T ? E : T); }

// Whether block b has a tile among `total` row tiles x NT column tiles.  More
// than the bound come only from offsets that decrease; their product with NT
// need not fit 32 bits, and no block takes a tile.
constexpr bool block_has_tile(int64_t b, int64_t total, int64_t NT, int64_t bound) {
  return total <= bound && b < total * NT;
}

// Place u of the order that takes bands of four row tiles and walks the
// columns inside a band: row tile t, column tile nt (0 <= u < total * NT).
constexpr void tile_order(int u, int total, int NT, int& t, int& nt) {
  const int band = u / (4 * NT), in = u - band * 4 * NT;
  const int h = total - band * 4 < 4 ? total - band * 4 : 4;
  nt = in / h;
  t = band * 4 + in - nt * h;
}

// Tile `skip` of an expert's rows [lo, hi); false if it has no such tile (a
// count over decreasing offsets that left 32 bits on the way).
constexpr bool expert_tile_rows(int lo, int hi, int64_t skip, int BM, ExpertTile& r) {
  if (skip < 0 || lo + skip * BM >= hi) return false;
  r.row0 = (int)(lo + skip * BM);
  r.rows = hi - r.row0 < BM ? hi - r.row0 : BM;
  return true;
}

}  // namespace ox
