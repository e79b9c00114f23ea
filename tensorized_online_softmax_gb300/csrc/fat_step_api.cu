// C entry points of a step of drafted tokens over the paged cache: storing them with
// their rotation, their attention, and keeping the accepted ones.  Argument
// validation and launches; nothing here allocates or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fat_attn.h"
#include "fat_cache_args.h"
#include "fat_tree.cuh"

using namespace fat;  // (the checks of fat_cache_args.h)

static_assert(FAT_TREE_TOKENS == kTreeTokens, "one bit to a drafted token");

extern "C" {

int fat_kv_append(const fat_kv_cache* cache, const fat_rotation* rotation, const void* q,
                  long long q_token_stride, long long q_head_stride, int q_heads, const void* k,
                  const void* v, int dtype, long long k_token_stride, long long k_head_stride,
                  long long v_token_stride, long long v_head_stride, const long long* slots,
                  int tokens, void* q_out, cudaStream_t stream) {
  AppendParams p = {};
  int st = cache_view(cache, true, &p.c);
  if (st != FAT_OK) return st;
  const bool e4m3 = cache->dtype == FAT_DTYPE_E4M3;
  const fat_rotation* r = rotation;
  if (!r || !wide_type(dtype) || (!e4m3 && dtype != cache->dtype) || tokens < 0 || q_heads < 0)
    return FAT_ERR_INVALID_ARG;
  if (r->dim < 16 || r->dim > cache->d || r->dim % 16 != 0 || r->rows < 1 ||
      r->row_stride < r->dim || r->axes < 1 || r->axes > FAT_ROTATION_AXES)
    return FAT_ERR_INVALID_ARG;
  long long pairs = 0;
  for (int i = 0; i < r->axes; ++i) {
    const int n = r->axes == 1 ? r->dim / 2 : r->sections[i];
    if (n < 0 || (pairs += n) > r->dim / 2) return FAT_ERR_INVALID_ARG;
    if (i < 3) p.ends[i] = static_cast<int>(pairs);
  }
  if (pairs != r->dim / 2) return FAT_ERR_INVALID_ARG;
  for (int i = r->axes; i < 3; ++i) p.ends[i] = r->dim / 2;
  if (tokens == 0) return FAT_OK;
  if (!k || !v || !slots || !r->cos_sin || !r->positions || (q_heads > 0 && (!q || !q_out)) ||
      r->token_stride < 0 || (r->axes > 1 && r->axis_stride < 0))
    return FAT_ERR_INVALID_ARG;
  if (static_cast<long long>(tokens) * (q_heads + 2ll * cache->heads) > 0x7fff0000ll)
    return FAT_ERR_INVALID_ARG;
  if (!stride_ok(k_token_stride, 2, &p.k_token) || !stride_ok(k_head_stride, 2, &p.k_head) ||
      !stride_ok(v_token_stride, 2, &p.v_token) || !stride_ok(v_head_stride, 2, &p.v_head) ||
      !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || !aligned(r->positions, 8) ||
      !aligned(r->cos_sin, 16) || r->row_stride % 4 != 0)
    return FAT_ERR_ALIGNMENT;
  if (q_heads > 0 && (!stride_ok(q_token_stride, 2, &p.q_token) ||
                      !stride_ok(q_head_stride, 2, &p.q_head) || !aligned(q, 16) ||
                      !aligned(q_out, 16)))
    return FAT_ERR_ALIGNMENT;
  int dev = 0;
  if ((st = host_device(&dev, &p.error_word)) != FAT_OK) return st;
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.q_out = static_cast<uint8_t*>(q_out);
  p.q_heads = q_heads;
  p.cos_sin = r->cos_sin;
  p.rows = r->rows;
  p.row_stride = r->row_stride;
  p.positions = r->positions;
  p.axis_stride = r->axis_stride;
  p.token_stride = r->token_stride;
  p.pairs = r->dim / 2;
  p.axes = r->axes;
  p.slots = slots;
  p.tokens = tokens;
  const int sms = sm_count(dev);
  if (sms < 1) return FAT_ERR_LAUNCH;
  return status(launch_kv_append(p, cache->d, e4m3, dtype == FAT_DTYPE_BF16, r->interleaved != 0,
                                 sms, stream));
}

int fat_kv_keep(const fat_kv_cache* cache, const fat_page_table* table, const int* path,
                long long path_stride, int width, const int* counts, cudaStream_t stream) {
  KeepParams p = {};
  int st = cache_view(cache, true, &p.c);
  if (st == FAT_OK) st = table_view(table, p.c.page_shift, &p.t);
  if (st != FAT_OK) return st;
  if (!path || !counts || width < 1 || width > (1 << 30) || path_stride < 0)
    return FAT_ERR_INVALID_ARG;
  if (!aligned(path, 4) || !aligned(counts, 4)) return FAT_ERR_ALIGNMENT;
  const bool e4m3 = cache->dtype == FAT_DTYPE_E4M3;
  p.chunks = cache->d * (e4m3 ? 1 : 2) / 16;
  p.scales = e4m3 ? 1 : 0;
  if (static_cast<long long>(table->batch) * cache->heads > (1ll << 29)) return FAT_ERR_INVALID_ARG;
  int dev = 0;
  if ((st = host_device(&dev, &p.t.error_word)) != FAT_OK) return st;
  p.path = path;
  p.path_stride = path_stride;
  p.width = width;
  p.counts = counts;
  return status(launch_kv_keep(p, stream));
}

size_t fat_attn_tree_workspace_bytes(int batch, int tokens, int q_heads, int kv_heads, int d) {
  if (batch < 1 || tokens < 1 || tokens > FAT_TREE_TOKENS || kv_heads < 1 || q_heads < 1 ||
      q_heads % kv_heads != 0 || (d != 64 && d != 128) ||
      static_cast<long long>(batch) * tokens * q_heads > (1ll << 30))
    return 0;
  return tree_workspace_bytes(tokens, q_heads / kv_heads, d);
}

int fat_attn_tree_paged(const fat_kv_cache* cache, const fat_page_table* table, const void* q,
                        int dtype, long long q_batch_stride, long long q_token_stride,
                        long long q_head_stride, int q_heads, int tokens, const long long* tree,
                        long long tree_stride, const int* draft_lens, int window, int sinks,
                        float scale, void* o, float* lse, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  return fat_attn_tree_paged_ex(cache, table, q, dtype, q_batch_stride, q_token_stride,
                                q_head_stride, q_heads, tokens, tree, tree_stride, draft_lens,
                                window, sinks, scale, o, lse, workspace, workspace_bytes, 0, stream);
}

int fat_attn_tree_paged_ex(const fat_kv_cache* cache, const fat_page_table* table, const void* q,
                           int dtype, long long q_batch_stride, long long q_token_stride,
                           long long q_head_stride, int q_heads, int tokens, const long long* tree,
                           long long tree_stride, const int* draft_lens, int window, int sinks,
                           float scale, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, unsigned long long wait_timeout_ns,
                           cudaStream_t stream) {
  TreeParams p = {};
  int st = cache_view(cache, true, &p.c);
  if (st == FAT_OK) st = table_view(table, p.c.page_shift, &p.t);
  if (st == FAT_OK)
    st = query_ok(q, dtype, q_batch_stride, q_head_stride, q_heads, cache->heads, table->batch,
                  &p.q_batch, &p.q_head);
  if (st != FAT_OK) return st;
  if (cache->dtype != FAT_DTYPE_E4M3 && cache->dtype != dtype) return FAT_ERR_INVALID_ARG;
  const size_t need =
      fat_attn_tree_workspace_bytes(table->batch, tokens, q_heads, cache->heads, cache->d);
  if (need == 0 || !tree || tree_stride < 0 || sinks < 0 || (window != 0 && window < tokens) ||
      !(scale > 0.f) || !std::isfinite(scale * kArgLog2e) || !o || !lse || !workspace ||
      workspace_bytes < need)
    return FAT_ERR_INVALID_ARG;
  if (!stride_ok(q_token_stride, 2, &p.q_token) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(tree, 8) || !aligned(draft_lens, 4) || !aligned(workspace, 16))
    return FAT_ERR_ALIGNMENT;
  // (the copies take tokens of a page, and heads and tokens of the queries, as they lie in memory)
  if (p.c.k_token == 0 || p.c.v_token == 0 || (p.q_head == 0 && q_heads > 1) ||
      (p.q_token == 0 && tokens > 1))
    return FAT_ERR_UNSUPPORTED;
  int dev = 0;
  if ((st = host_device(&dev, &p.t.error_word)) != FAT_OK) return st;
  const int sms = sm_count(dev);
  if (sms < 1) return FAT_ERR_LAUNCH;
  p.error_word = p.t.error_word;
  p.timeout_ns = wait_timeout_ns ? wait_timeout_ns : 4000000000ull;
  p.suspend_ns = p.timeout_ns < 50000 ? static_cast<uint32_t>(p.timeout_ns) : 50000u;
  p.workspace = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const uint8_t*>(q);
  p.tokens = tokens;
  p.group = q_heads / cache->heads;
  p.tree = tree;
  p.tree_stride = tree_stride;
  p.draft_lens = draft_lens;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = scale * kArgLog2e;
  p.o = static_cast<uint8_t*>(o);
  p.lse = lse;
  return status(launch_tree(p, cache->d, cache->dtype == FAT_DTYPE_E4M3, dtype == FAT_DTYPE_BF16,
                            dev, sms, stream));
}

}  // extern "C"
