// C entry points of the paged key-value cache: argument validation and
// launches.  Nothing here allocates or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fat_attn.h"
#include "fat_cache_args.h"
#include "fat_decode_plan.h"

static_assert(FAT_DECODE_DIRECT == fat::kDirectTiles * fat::kDecodeTile, "one rule");

using namespace fat;  // (the checks of fat_cache_args.h)

extern "C" {

int fat_kv_write(const fat_kv_cache* cache, const void* k, const void* v, int dtype,
                 long long k_token_stride, long long k_head_stride, long long v_token_stride,
                 long long v_head_stride, const long long* slots, int tokens,
                 cudaStream_t stream) {
  fat::WriteParams p = {};
  int st = cache_view(cache, true, &p.c);
  if (st != FAT_OK) return st;
  const bool e4m3 = cache->dtype == FAT_DTYPE_E4M3;
  if (!wide_type(dtype) || (!e4m3 && dtype != cache->dtype) || tokens < 0)
    return FAT_ERR_INVALID_ARG;
  if (tokens == 0) return FAT_OK;
  if (!k || !v || !slots) return FAT_ERR_INVALID_ARG;
  if (static_cast<long long>(tokens) * cache->heads > 0x7fff0000ll) return FAT_ERR_INVALID_ARG;
  if (!stride_ok(k_token_stride, 2, &p.k_token) || !stride_ok(k_head_stride, 2, &p.k_head) ||
      !stride_ok(v_token_stride, 2, &p.v_token) || !stride_ok(v_head_stride, 2, &p.v_head) ||
      !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return FAT_ERR_ALIGNMENT;
  int dev = 0;
  if ((st = fat::host_device(&dev, &p.error_word)) != FAT_OK) return st;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.slots = slots;
  p.tokens = tokens;
  const int sms = sm_count(dev);
  if (sms < 1) return FAT_ERR_LAUNCH;
  return status(fat::launch_kv_write(p, cache->d, e4m3, dtype == FAT_DTYPE_BF16, sms, stream));
}

int fat_kv_read(const fat_kv_cache* cache, const fat_page_table* table, void* k, void* v,
                int dtype, int max_len, cudaStream_t stream) {
  fat::ReadParams p = {};
  int st = cache_view(cache, true, &p.c);
  if (st == FAT_OK) st = table_view(table, p.c.page_shift, &p.t);
  if (st != FAT_OK) return st;
  const bool e4m3 = cache->dtype == FAT_DTYPE_E4M3;
  if (!wide_type(dtype) || (!e4m3 && dtype != cache->dtype) || max_len < 1 ||
      max_len > (1 << 30) || !k || !v)
    return FAT_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return FAT_ERR_ALIGNMENT;
  int dev = 0;
  if ((st = fat::host_device(&dev, &p.t.error_word)) != FAT_OK) return st;
  p.k = static_cast<uint8_t*>(k);
  p.v = static_cast<uint8_t*>(v);
  p.max_len = max_len;
  const int sms = sm_count(dev);
  if (sms < 1) return FAT_ERR_LAUNCH;
  return status(fat::launch_kv_read(p, cache->d, e4m3, dtype == FAT_DTYPE_BF16, sms, stream));
}

size_t fat_attn_decode_workspace_bytes(int batch, int q_heads, int kv_heads, int d) {
  if (batch < 1 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 ||
      static_cast<long long>(batch) * q_heads > (1ll << 30) || (d != 64 && d != 128))
    return 0;
  return fat::decode_workspace_bytes(d);
}

static int decode_common(const fat_kv_cache* cache, const fat_page_table* table, const void* q,
                         int dtype, long long q_batch_stride, long long q_head_stride,
                         int q_heads, float scale, void* o, float* lse, fat::DecodeParams* p) {
  int st = cache_view(cache, true, &p->c);
  if (st == FAT_OK) st = table_view(table, p->c.page_shift, &p->t);
  if (st == FAT_OK)
    st = query_ok(q, dtype, q_batch_stride, q_head_stride, q_heads, cache->heads, table->batch,
                  &p->q_batch, &p->q_head);
  if (st != FAT_OK) return st;
  if (cache->dtype != FAT_DTYPE_E4M3 && cache->dtype != dtype) return FAT_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale) || !o || !lse) return FAT_ERR_INVALID_ARG;
  if (!aligned(o, 16) || !aligned(lse, 4)) return FAT_ERR_ALIGNMENT;
  p->least_tiles = 2;
  p->q = static_cast<const uint8_t*>(q);
  p->group = q_heads / cache->heads;
  p->scale_log2 = scale * kArgLog2e;
  p->o = static_cast<uint8_t*>(o);
  p->lse = lse;
  return FAT_OK;
}

int fat_attn_decode_paged(const fat_kv_cache* cache, const fat_page_table* table, const void* q,
                          int dtype, long long q_batch_stride, long long q_head_stride,
                          int q_heads, float scale, void* o, float* lse, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
  fat::DecodeParams p = {};
  int st = decode_common(cache, table, q, dtype, q_batch_stride, q_head_stride, q_heads, scale, o,
                         lse, &p);
  if (st != FAT_OK) return st;
  const bool direct =
      (static_cast<long long>(table->width) << p.c.page_shift) <= FAT_DECODE_DIRECT;
  if (!direct && (!workspace || workspace_bytes < fat::decode_workspace_bytes(cache->d)))
    return FAT_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return FAT_ERR_ALIGNMENT;
  int dev = 0;
  if ((st = fat::host_device(&dev, &p.t.error_word)) != FAT_OK) return st;
  p.workspace = workspace;
  return status(fat::launch_decode(p, cache->d, cache->dtype == FAT_DTYPE_E4M3,
                                   dtype == FAT_DTYPE_BF16, dev, stream));
}

int fat_attn_decode_window(const fat_kv_cache* cache, const fat_page_table* table, const void* q,
                           int dtype, long long q_batch_stride, long long q_head_stride,
                           int q_heads, int window, int sinks, float scale, void* o, float* lse,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  fat::DecodeParams p = {};
  int st = decode_common(cache, table, q, dtype, q_batch_stride, q_head_stride, q_heads, scale, o,
                         lse, &p);
  if (st != FAT_OK) return st;
  if (window < 1 || sinks < 0) return FAT_ERR_INVALID_ARG;
  const bool direct =
      decode_span_most(static_cast<long long>(table->width) << p.c.page_shift, window, sinks,
                       kDecodeTile) <= kDirectTiles;
  if (!direct && (!workspace || workspace_bytes < fat::decode_workspace_bytes(cache->d)))
    return FAT_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return FAT_ERR_ALIGNMENT;
  int dev = 0;
  if ((st = fat::host_device(&dev, &p.t.error_word)) != FAT_OK) return st;
  p.window = window;
  p.sinks = sinks;
  p.workspace = workspace;
  return status(fat::launch_decode(p, cache->d, cache->dtype == FAT_DTYPE_E4M3,
                                   dtype == FAT_DTYPE_BF16, dev, stream));
}

int fat_kv_block_bounds(const fat_kv_cache* cache, const fat_page_table* table, int new_tokens,
                        void* bounds, int dtype, cudaStream_t stream) {
  fat::BoundsParams p = {};
  int st = cache_view(cache, false, &p.c);
  if (st == FAT_OK) st = table_view(table, p.c.page_shift, &p.t);
  if (st != FAT_OK) return st;
  const bool e4m3 = cache->dtype == FAT_DTYPE_E4M3;
  if (!wide_type(dtype) || (!e4m3 && dtype != cache->dtype) || new_tokens < 1 || !bounds)
    return FAT_ERR_INVALID_ARG;
  if (!aligned(bounds, 16)) return FAT_ERR_ALIGNMENT;
  int dev = 0;
  if ((st = fat::host_device(&dev, &p.t.error_word)) != FAT_OK) return st;
  p.bounds = static_cast<uint8_t*>(bounds);
  p.new_tokens = new_tokens;
  return status(fat::launch_kv_bounds(p, cache->d, e4m3, dtype == FAT_DTYPE_BF16, stream));
}

int fat_kv_block_scores(const void* q, int dtype, long long q_batch_stride,
                        long long q_head_stride, int q_heads, const void* bounds,
                        long long num_pages, int kv_heads, int page_size, int d,
                        const fat_page_table* table, float* scores, cudaStream_t stream) {
  fat::ScoreParams p = {};
  if (!bounds || !scores || kv_heads < 1 || kv_heads > (1 << 20) || num_pages < 1 ||
      num_pages > 0x7fffffffll || (d != 64 && d != 128))
    return FAT_ERR_INVALID_ARG;
  p.page_shift = page_shift_of(page_size);
  if (p.page_shift < 0) return FAT_ERR_INVALID_ARG;
  int st = table_view(table, p.page_shift, &p.t);
  if (st != FAT_OK) return st;
  st = query_ok(q, dtype, q_batch_stride, q_head_stride, q_heads, kv_heads, table->batch,
                &p.q_batch, &p.q_head);
  if (st != FAT_OK) return st;
  if (!aligned(bounds, 16) || !aligned(scores, 4)) return FAT_ERR_ALIGNMENT;
  int dev = 0;
  if ((st = fat::host_device(&dev, &p.t.error_word)) != FAT_OK) return st;
  p.q = static_cast<const uint8_t*>(q);
  p.bounds = static_cast<const uint8_t*>(bounds);
  p.num_pages = static_cast<uint32_t>(num_pages);
  p.heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.scores = scores;
  const int sms = sm_count(dev);
  if (sms < 1) return FAT_ERR_LAUNCH;
  return status(fat::launch_kv_scores(p, d, dtype == FAT_DTYPE_BF16, dev, sms, stream));
}

static size_t choice_bytes(long long bh, long long list) {
  return static_cast<size_t>((bh * (list + 1) * 4 + 15) / 16 * 16);
}

size_t fat_attn_decode_sparse_workspace_bytes(int batch, int q_heads, int kv_heads, int d,
                                              int num_blocks) {
  const size_t n = fat_attn_decode_workspace_bytes(batch, q_heads, kv_heads, d);
  if (n == 0 || num_blocks < 1 || num_blocks > (1 << 30)) return 0;
  return n + choice_bytes(static_cast<long long>(batch) * kv_heads, num_blocks);
}

int fat_attn_decode_sparse(const fat_kv_cache* cache, const fat_page_table* table, const void* q,
                           int dtype, long long q_batch_stride, long long q_head_stride,
                           int q_heads, const float* scores, int num_blocks, int first_blocks,
                           int last_blocks, float scale, void* o, float* lse, int* blocks,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  fat::DecodeParams p = {};
  int st = decode_common(cache, table, q, dtype, q_batch_stride, q_head_stride, q_heads, scale, o,
                         lse, &p);
  if (st != FAT_OK) return st;
  if (!scores || !blocks || num_blocks < 1 || num_blocks > (1 << 30) || first_blocks < 0 ||
      last_blocks < 0 ||
      static_cast<long long>(first_blocks) + last_blocks > num_blocks || !workspace ||
      workspace_bytes < fat_attn_decode_sparse_workspace_bytes(table->batch, q_heads,
                                                               cache->heads, cache->d, num_blocks))
    return FAT_ERR_INVALID_ARG;
  if (!aligned(scores, 4) || !aligned(blocks, 4) || !aligned(workspace, 16))
    return FAT_ERR_ALIGNMENT;
  int dev = 0;
  if ((st = fat::host_device(&dev, &p.t.error_word)) != FAT_OK) return st;
  const long long bh = static_cast<long long>(table->batch) * cache->heads;
  fat::SelectParams s = {};
  s.t = p.t;
  s.scores = scores;
  s.heads = cache->heads;
  s.page_shift = p.c.page_shift;
  s.num_blocks = num_blocks;
  s.first_blocks = first_blocks;
  s.last_blocks = last_blocks;
  s.blocks = blocks;
  s.list = num_blocks < table->width ? num_blocks : table->width;
  s.pages = static_cast<int*>(workspace);
  s.lens = s.pages + bh * s.list;
  if (fat::launch_select(s, stream) != 0) return FAT_ERR_LAUNCH;
  // the chosen pages are a page table of their own, one entry per (sequence, head)
  p.per_head = 1;
  p.t.pages = s.pages;
  p.t.stride = s.list;
  p.t.width = s.list;
  p.t.batch = static_cast<int>(bh);
  p.t.seq_lens = s.lens;
  p.workspace = static_cast<uint8_t*>(workspace) + choice_bytes(bh, num_blocks);
  return status(fat::launch_decode(p, cache->d, cache->dtype == FAT_DTYPE_E4M3,
                                   dtype == FAT_DTYPE_BF16, dev, stream));
}

}  // extern "C"
