// How a decode call's work is shared out: plain integer arithmetic, used by the
// kernels and by the tests on the host.
//
// An entry is one line of the page table (a sequence, or a sequence's choice of
// pages for one cached head); it has `copies` items (its cached heads and, for
// more than 16 query heads to a cached head, blocks of those).  An item is one
// pass over the entry's positions in tiles of kDecodeTile; an empty entry has
// one (empty) tile, so that its output is written.  The tiles of all items form
// one line, entry by entry and item by item, and every thread block takes the
// same number of adjacent ones, whatever the lengths are: blocks finish
// together, and long sequences are split while short ones share a block.
#pragma once

#ifndef __CUDACC__
#define FAT_HD inline
#else
#define FAT_HD __host__ __device__ __forceinline__
#endif

namespace fat {

constexpr int kDecodeTile = 64;
constexpr int kDirectTiles = 8;
constexpr int kDecodeMaxBlocks = 640;  // what the workspace has room for

FAT_HD int decode_tiles(int len) {
  return len > kDecodeTile ? (len - 1) / kDecodeTile + 1 : 1;
}

// The positions that are seen of a sequence of `len`: the last `window` of them and
// the first `sinks`; window 0 stands for all.  They are walked tile by tile, the
// tiles between the two left out.
struct DecodeSpan {
  int lo, sink;     // seen: [0, sink) and [lo, len)
  int heads, skip;  // tiles ahead of the gap, and tiles in it
  int tiles;        // tiles walked (one empty one if there is nothing to see)
};

FAT_HD DecodeSpan decode_span(int len, int window, int sinks, int tile) {
  DecodeSpan s;
  s.lo = window > 0 && len > window ? len - window : 0;
  s.sink = sinks < len ? sinks : len;
  if (s.sink >= s.lo) s.lo = s.sink = 0;  // one range
  s.heads = s.sink > 0 ? (s.sink - 1) / tile + 1 : 0;
  s.skip = s.lo / tile > s.heads ? s.lo / tile - s.heads : 0;
  s.tiles = (len > tile ? (len - 1) / tile + 1 : 1) - s.skip;
  return s;
}

// The tile of the sequence that is walked i-th.
FAT_HD int decode_span_tile(const DecodeSpan& s, int i) { return i < s.heads ? i : i + s.skip; }

FAT_HD bool decode_span_sees(const DecodeSpan& s, int at) { return at < s.sink || at >= s.lo; }

// The most tiles that a sequence of at most `positions` can have.
FAT_HD long long decode_span_most(long long positions, int window, int sinks, int tile) {
  const long long all = positions > tile ? (positions - 1) / tile + 1 : 1;
  if (window <= 0) return all;
  const long long seen = (static_cast<long long>(sinks) + tile - 1) / tile +
                         (static_cast<long long>(window) + tile - 1) / tile + 1;
  return seen < all ? seen : all;
}

// Tiles of one block: an equal share, but at least `least` (a split costs the
// join of its parts).
template <typename T>
FAT_HD T decode_share(T total, int blocks, int least) {
  const T n = (total + blocks - 1) / blocks;
  return n > least ? n : least;
}

// A place on the line of tiles: tile `tile` of item `item` of entry `entry`.
struct DecodePlace {
  int entry, item, tile, tiles;  // tiles: of this entry's items
};

// The place `offset` tiles into an entry whose items have `tiles` tiles.
FAT_HD DecodePlace decode_place(int entry, long long offset, int tiles) {
  DecodePlace p;
  p.entry = entry;
  p.tiles = tiles;
  p.item = offset <= 0x7fffffff ? static_cast<int>(offset) / tiles
                                : static_cast<int>(offset / tiles);
  p.tile = static_cast<int>(offset - static_cast<long long>(p.item) * tiles);
  return p;
}

// One tile on; true where that is a new entry (whose `tiles` the caller sets).
FAT_HD bool decode_advance(DecodePlace& p, int copies) {
  if (++p.tile < p.tiles) return false;
  p.tile = 0;
  if (++p.item < copies) return false;
  p.item = 0;
  ++p.entry;
  return true;
}

// A block keeps at most two unfinished items: the one that its range starts in
// (part 0) and the one that it ends in (part 1).  `first`: the item's first
// tile on the line, `begin`: the block's.
FAT_HD int decode_part(long long first, long long begin) { return first <= begin ? 0 : 1; }

}  // namespace fat
