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
