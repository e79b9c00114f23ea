// How the warps of the attention of drafted tokens wait for an item's queries over an e4m3
// cache: plain integers, used by the kernel and by the test of its waits on the host.
//
// The queries of a block's items (those with drafted tokens, counted from 0) come one item after
// the other, and each completes a phase of a barrier.  The MMA issuer waits for every item; the
// converters of K, whose type follows the queries', for the items that they have tiles of.  Two
// teams of them take tiles in turn, so that a team has no tile of an item of one tile that is the
// other's, and nothing holds that item up for it: by the time it looks, the item's phase and the
// next one may be over.  On one barrier the parity of the first would then read as not yet there,
// and the wait would not end.  So there are two, for even and odd items, and a team waits only for
// its own tile's: its tiles are two apart, so it passes over one item at most and has seen, or knows
// from the item behind it, that the phase before the one it waits for is over; and the one behind
// that needs the team's own keys.
#pragma once

#ifndef FAT_HD
#ifndef __CUDACC__
#define FAT_HD inline
#else
#define FAT_HD __host__ __device__ __forceinline__
#endif
#endif

namespace fat {

constexpr int kTreeQueryBars = 2;

// The barrier of item j, and the parity of its phase.
FAT_HD int tree_query_bar(unsigned j) { return static_cast<int>(j % kTreeQueryBars); }
FAT_HD unsigned tree_query_parity(unsigned j) { return j / kTreeQueryBars & 1u; }

}  // namespace fat
