// Which rows a work-group of the attention kernels takes: index arithmetic alone, the same on the
// device and in a host program.
//
// Row tiles of graph g (rows first(g) .. first(g + 1)) take the slots first(g) / tile + g
// and on: enough for ceil(rows / tile) tiles, without a host-side list of lengths.  A
// slot belongs to the last graph whose first slot is not beyond it, and may hold no tile.
#pragma once

#include <cstdint>

namespace e3c {
namespace attn {

// An offset of a segment table, kept inside [0, n] whatever the table holds.
constexpr int clamp_offset(int v, long n) { return v < 0 ? 0 : (v > n ? (int)n : v); }

// First slot of graph g, whose first row (of mult for each entry of the table) is `first`.
constexpr int slot_at(int first, int g, int mult, int tile) { return first * mult / tile + g; }

// The graph of a slot among `graphs`.  64 graphs lo, lo + step, .. (below lo + count) are tried at a
// time: hits(lo, step, count) is how many of them have a first slot not beyond it.
template <class Hits>
constexpr int search_graph(int graphs, Hits hits) {
  int lo = 0, count = graphs;
  while (count > 1) {
    const int step = (count + 63) >> 6, found = hits(lo, step, count), n = found > 1 ? found : 1;
    lo += (n - 1) * step;
    count = step < count - (n - 1) * step ? step : count - (n - 1) * step;
  }
  return lo;
}

// Row of a graph's rows where the tile of a slot starts, or -1 where its nrows rows have no such tile.
// A table that does not begin at 0 or decreases gives slots before the graph's first.
constexpr int tile_start(int slot, int first_slot, int tile, int nrows) {
  const int64_t row = (int64_t)(slot - first_slot) * tile;
  return row >= 0 && row < nrows ? (int)row : -1;
}

// r / group for 0 <= r < 2^31: ceil(2^(31 + l) / group) with 2^l >= group, by a product.
struct GroupDiv {
  unsigned magic;
  int shift, log2;      // log2: of a power of two, else 31 (a shift that leaves nothing of a step of rows)
};
constexpr GroupDiv group_div(int group) {
  int l = 0;
  while ((1 << l) < group) ++l;
  return {(unsigned)((((uint64_t)1 << (31 + l)) + group - 1) / group), l - 1, 1 << l == group ? l : 31};
}
constexpr int div_group(int r, int group, unsigned magic, int shift) {
  return group == 1 ? r : (int)((unsigned)(((uint64_t)(unsigned)r * magic) >> 32) >> shift);
}

}  // namespace attn
}  // namespace e3c
