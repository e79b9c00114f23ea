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
// codes (swizzled alike where they have 128 bytes).  A dimension whose stride is 0 becomes one of size 1, and its
// coordinates are multiplied by 0.
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
                           e4m3 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows of an item: one block of 128, or two for 16-bit caches with more; the rows beyond that
// are shared out evenly, in whole warps.
int item_rows_of(int rows, int blocks) {
  const int most = blocks * kTreeBlockRows;
  const int items = (rows + most - 1) / most;
  const int each = ((rows + items - 1) / items + 31) / 32 * 32;
  return each < most ? each : most;
}

}  // namespace

}  // namespace tree

size_t tree_workspace_bytes(int tokens, int group, int d) {
  const int rows = tokens * group;
  const int one = tree::item_rows_of(rows, 1), two = tree::item_rows_of(rows, 2);
  return tree::rows_at(kTreeMaxBlocks, 0, one > two ? one : two, d);
}

int launch_tree(const TreeParams& params, int d, bool e4m3, bool bf16, int dev, int sms,
                cudaStream_t stream) {
  tree::KernelParams kp;
  kp.p = params;
  TreeParams& p = kp.p;
  const CacheView& c = p.c;
  const int rows = p.tokens * p.group;
  // Two blocks of rows read the cache once for both; an e4m3 cache's conversion leaves room
  // for one.
  const int blocks = !e4m3 && rows > kTreeBlockRows ? 2 : 1;
  p.item_rows = tree::item_rows_of(rows, blocks);
  p.row_blocks = (rows + p.item_rows - 1) / p.item_rows;
  p.direct = 0;
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
