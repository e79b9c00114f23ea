// Attention of drafted tokens over the paged cache: what its kernels are given, and
// what a row sees.
#pragma once

#include "fat_cache.cuh"

namespace fat {

constexpr int kTreeTokens = 64;  // drafted tokens of a sequence: bits of a mask

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

// What drafted token t sees: of the context the positions below `sink` and from `lo`
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

size_t tree_workspace_bytes(int tokens, int group, int d);
int launch_tree(const TreeParams& p, int d, bool e4m3, bool bf16, int dev, cudaStream_t stream);

}  // namespace fat
