// Attention of drafted tokens over the paged cache: the choice of the kernel, the cut of
// the rows, and the tensor maps of the cache.
#include "fat_tree_kernel.cuh"

namespace fat {

namespace tree {

int launch_d64(const KernelParams& kp, int type, int blocks, int dev, int sms,
               cudaStream_t stream);
int launch_d128(const KernelParams& kp, int type, int blocks, int dev, int sms,
                cudaStream_t stream);

namespace {

// K or V as [page, head, token, d], in boxes of as many tokens as a tile has of a page: 64
// columns of 16 bits, 128-byte swizzle (the layout of the MMA's operands), or whole rows of
// codes (swizzled alike where they have 128 bytes).  A dimension whose stride is 0 becomes one
// of size 1, and its coordinates are multiplied by 0.
bool cache_map(CUtensorMap* tm, void* ptr, const CacheView& c, int d, bool e4m3, uint32_t page,
               uint32_t head, uint32_t token, int* by_page, int* by_head) {
  *by_page = page != 0 && c.num_pages > 1;
  *by_head = head != 0 && c.heads > 1;
  const uint32_t row = static_cast<uint32_t>(d) * (e4m3 ? 1 : 2);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(*by_head ? c.heads : 1),
                              static_cast<cuuint64_t>(*by_page ? c.num_pages : 1)};
  const cuuint64_t strides[3] = {token, *by_head ? head : row, *by_page ? page : row};
  const cuuint32_t rows = c.page_size < kTreeTile ? c.page_size : kTreeTile;
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(e4m3 ? d : 64), rows, 1, 1};
  return encode_tensor_map(tm,
                           e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                           4, ptr, dims, strides, box,
                           e4m3 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_NONE
                                           : CU_TENSOR_MAP_SWIZZLE_128B);
}

// The queries as [sequence, token, head, d], in boxes of a block of rows.
bool query_map(CUtensorMap* tm, const TreeParams& p, int d, int* by_batch) {
  *by_batch = p.q_batch != 0 && p.t.batch > 1;
  const int heads = p.group * p.c.heads;
  const uint32_t row = static_cast<uint32_t>(d) * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(p.tokens),
                              static_cast<cuuint64_t>(*by_batch ? p.t.batch : 1)};
  const cuuint64_t strides[3] = {heads > 1 ? p.q_head : row, p.tokens > 1 ? p.q_token : row,
                                 *by_batch ? p.q_batch : row};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.block_heads),
                             static_cast<cuuint32_t>(p.block_tokens), 1};
  return encode_tensor_map(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<uint8_t*>(p.q), dims,
                           strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The cut of a cached head's rows into items of one block of at most 128 rows or of two: as few
// blocks as hold them, shared out evenly.
void cut_rows(int tokens, int group, int blocks, TreeParams* p) {
  p->head_items = (group + kTreeBlockRows - 1) / kTreeBlockRows;
  p->block_heads = (group + p->head_items - 1) / p->head_items;
  const int most = kTreeBlockRows / p->block_heads;
  p->token_items = (tokens + most * blocks - 1) / (most * blocks);
  p->block_tokens = (tokens + p->token_items * blocks - 1) / (p->token_items * blocks);
  p->item_rows = blocks * p->block_tokens * p->block_heads;
  p->copies = p->item_rows <= kTreeBlockRows / 2 ? 2 : 1;
}

}  // namespace

}  // namespace tree

size_t tree_workspace_bytes(int tokens, int group, int d) {
  TreeParams one, two;
  tree::cut_rows(tokens, group, 1, &one);
  tree::cut_rows(tokens, group, 2, &two);
  return tree::rows_at(kTreeMaxBlocks, 0,
                       one.item_rows > two.item_rows ? one.item_rows : two.item_rows, d);
}

int launch_tree(const TreeParams& params, int d, bool e4m3, bool bf16, int dev, int sms,
                cudaStream_t stream) {
  tree::KernelParams kp = {};
  kp.p = params;
  TreeParams& p = kp.p;
  const CacheView& c = p.c;
  // Two blocks of rows read the cache once for both (8 sequences of 4096 to 16384, 256 rows: 88
  // us, 120 with one); an e4m3 cache's conversion leaves room for one.
  tree::cut_rows(p.tokens, p.group, 1, &p);
  const int blocks = !e4m3 && p.token_items > 1 ? 2 : 1;
  tree::cut_rows(p.tokens, p.group, blocks, &p);
  p.direct = 0;
  // Measured, of 1, 2, 3, 4, 6 and 8: 16-bit, 13 sequences of up to 1029 seen positions (9 tiles)
  // 39, 31, 30, 32, 32, 37 us; 16 of 1000 to 8192 55.7, 54.3, 53.8, 53.6, 54.3, 55.2; e4m3, whose
  // queries are converted, of 3, 4, 6, 8, 10: 32 of 4096 to 16384 215, 211, 207, 205, 205; 16 of 1000
  // to 8192 60, 59, 56, 56, 58; 32 of 100 to 1000 41.4, 40.6, 39.0, 39.5, 40.9; 64 of 20 to 300 51.4,
  // 46.1, 46.9, 48.7, 49.8.
  p.item_cost = e4m3 ? 6 : 3;
  if (!e4m3 && !tree::query_map(&kp.tm_q, p, d, &kp.q_batch)) return -4;
  if (!tree::cache_map(&kp.tm_k, c.k, c, d, e4m3, c.k_page, c.k_head, c.k_token, &kp.k_page,
                       &kp.k_head) ||
      !tree::cache_map(&kp.tm_v, c.v, c, d, e4m3, c.v_page, c.v_head, c.v_token, &kp.v_page,
                       &kp.v_head))
    return -4;
  const int type = e4m3 ? (bf16 ? tree::kE4M3Bf16 : tree::kE4M3F16)
                        : (bf16 ? tree::kBf16 : tree::kF16);
  return d == 128 ? tree::launch_d128(kp, type, blocks, dev, sms, stream)
                  : tree::launch_d64(kp, type, blocks, dev, sms, stream);
}

}  // namespace fat
