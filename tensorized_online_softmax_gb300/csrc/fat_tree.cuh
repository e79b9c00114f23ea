// Attention of drafted tokens over the paged cache: what its kernels are given, what a
// row sees, and how the work is cut.
#pragma once

#include "fat_cache.cuh"
#include "fat_decode_plan.h"
#include "fat_tree_sync.h"

namespace fat {

constexpr int kTreeTokens = 64;   // drafted tokens of a sequence: bits of a mask
constexpr int kTreeTile = 128;    // positions of a tile
constexpr int kTreeBlockRows = 128;
constexpr int kTreeMaxBlocks = 160;  // what the workspace has room for
// Items are not split, where a block is there for each, if they have up to kTreeDirect tiles (as the
// table and the window bound them); or up to kTreeWhole (under a window, where most sequences have
// as many, kTreeWholeWindow) and blocks without an item cost less than the plan, the join and a
// block's second item: tiles * (blocks - items) <= 6 * blocks.  8 heads of 32 rows, split and not,
// us: one sequence of 6, 7 and 8 tiles 11.8, 12.0, 12.5 and 11.9, 12.8, 13.6 (e4m3, where 5 tiles
// are the border, 15.2, 15.1, 15.2 and 16.5, 17.8, 18.9), four 13.8, 14.7, 14.9 and 12.0, 12.8,
// 13.7; 19 of 50 to 2048 (16 tiles) 29.0 and 23.7, 8 of 50 to 4096 28.0 and 34.7; window 1000 (10
// tiles), 19 sequences 31.2 and 23.4, 4 of them 16.0 and 17.7; where there are more items than
// blocks neither way is better for all.
constexpr int kTreeDirect = 6, kTreeWhole = 16, kTreeWholeWindow = 24;

struct TreeParams {
  CacheView c;
  TableView t;
  const uint8_t* q;
  uint32_t q_batch, q_token, q_head;  // bytes
  int tokens;                         // drafted tokens of a sequence, at most
  int group;                          // query heads per cached head
  const long long* tree;              // a mask for each (sequence, drafted token)
  long long tree_stride;              // masks between sequences
  const int* draft_lens;              // null: `tokens` everywhere
  int window, sinks;                  // window 0: the whole context
  float scale_log2;                   // scale * log2(e)
  uint8_t* o;                         // [batch, tokens, q_heads, d]
  float* lse;                         // [batch, tokens, q_heads]
  uint8_t* workspace;
  // Rows of a cached head: blocks of `block_tokens` tokens by `block_heads` of the group's
  // heads (row = token * block_heads + head), one or two blocks along the tokens to an item.
  int block_tokens, block_heads;
  int token_items, head_items;  // items along the tokens and along the group's heads
  int item_rows;                // rows of an item
  int copies;                   // (e4m3) of an item's rows among the 128 of a block: 2 if they fit
  int direct;       // items are not split
  int item_cost;    // what an item costs besides its tiles, in tiles
  unsigned long long timeout_ns;  // of a wait on the device
  uint32_t suspend_ns;            // of one poll of it, about
  unsigned int* error_word;
};

// A sequence's length and how many of its last positions are drafted tokens.
struct TreeLens {
  int len, drafted;
};
__device__ __forceinline__ TreeLens tree_lens(const TreeParams& p, int b) {
  TreeLens n;
  n.len = table_length(p.t, p.c.page_shift, b);
  n.drafted = p.draft_lens ? p.draft_lens[b] : p.tokens;
  const int most = min(n.len, p.tokens);
  if (n.drafted < 0 || n.drafted > most) {
    atomicOr(p.t.error_word, kErrIndex);
    n.drafted = n.drafted < 0 ? 0 : most;
  }
  return n;
}

// What drafted token t sees: of the context the positions below `sinks` and from `lo`
// on, of the drafted tokens those in `mask`.  Its own position is the context's length
// plus the drafted tokens that it sees, itself among them, less one.
struct TreeRow {
  unsigned long long mask;
  int lo;
};
__device__ __forceinline__ TreeRow tree_row(const TreeParams& p, const TreeLens& n, int b, int t) {
  TreeRow r;
  r.mask = static_cast<unsigned long long>(p.tree[b * p.tree_stride + t]);
  if (n.drafted < 64) r.mask &= (1ull << n.drafted) - 1ull;
  r.lo = 0;
  if (p.window > 0) r.lo = max(0, n.len - n.drafted + __popcll(r.mask) - p.window);
  return r;
}

// The tiles that are walked for a sequence: those with a position that some row may see
// (a row that sees no drafted token sees the window one further back than the others).
__device__ __forceinline__ DecodeSpan tree_span(const TreeParams& p, const TreeLens& n) {
  const int len = n.drafted > 0 ? n.len : 0;
  const int window = p.window > 0 ? min(p.window, 1 << 30) + n.drafted : 0;
  return decode_span(len, window, p.sinks, kTreeTile);
}

// An item costs as much as `item_cost` tiles besides its own: its queries, the first scores and
// the last O += P V, which nothing overlaps, its end.  (An entry without drafted tokens costs
// next to nothing.)
__device__ __forceinline__ int tree_cost(const TreeParams& p, const TreeLens& n) {
  return n.drafted > 0 ? p.item_cost : 0;
}

size_t tree_workspace_bytes(int tokens, int group, int d);
int launch_tree(const TreeParams& p, int d, bool e4m3, bool bf16, int dev, int sms,
                cudaStream_t stream);

}  // namespace fat
