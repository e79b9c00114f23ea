// C entry points of the paged key-value cache: argument validation and
// launches.  Nothing here allocates or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fat_attn.h"
#include "fat_cache.cuh"
#include "fat_decode_plan.h"

static_assert(FAT_DECODE_DIRECT == fat::kDirectTiles * fat::kDecodeTile, "one rule");

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool wide_type(int t) { return t == FAT_DTYPE_BF16 || t == FAT_DTYPE_FP16; }

int page_shift_of(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

// strides in elements of `bytes` -> bytes; false if a row would not start on 16 bytes or the
// stride is 4 GiB or more
bool stride_ok(long long elements, int bytes, uint32_t* out) {
  if (elements < 0 || elements > 0xffffffffll / bytes) return false;
  *out = static_cast<uint32_t>(elements * bytes);
  return *out % 16 == 0;
}

// the cache's description -> the kernels' view of it
int cache_view(const fat_kv_cache* c, bool need_v, fat::CacheView* out) {
  if (!c || !c->k || (need_v && !c->v)) return FAT_ERR_INVALID_ARG;
  if (c->heads < 1 || c->num_pages < 1 || (c->d != 64 && c->d != 128)) return FAT_ERR_INVALID_ARG;
  const int shift = page_shift_of(c->page_size);
  if (shift < 0 || c->num_pages > 0x7fffffffll || c->heads > (1 << 20)) return FAT_ERR_INVALID_ARG;
  const bool e4m3 = c->dtype == FAT_DTYPE_E4M3;
  if (!e4m3 && !wide_type(c->dtype)) return FAT_ERR_INVALID_ARG;
  if (e4m3 && (!c->k_scale || (need_v && !c->v_scale))) return FAT_ERR_INVALID_ARG;
  const int bytes = e4m3 ? 1 : 2;
  fat::CacheView v = {};
  if (!stride_ok(c->k_page_stride, bytes, &v.k_page) ||
      !stride_ok(c->k_head_stride, bytes, &v.k_head) ||
      !stride_ok(c->k_token_stride, bytes, &v.k_token))
    return FAT_ERR_ALIGNMENT;
  if (need_v && (!stride_ok(c->v_page_stride, bytes, &v.v_page) ||
                 !stride_ok(c->v_head_stride, bytes, &v.v_head) ||
                 !stride_ok(c->v_token_stride, bytes, &v.v_token)))
    return FAT_ERR_ALIGNMENT;
  if (!aligned(c->k, 16) || (need_v && !aligned(c->v, 16))) return FAT_ERR_ALIGNMENT;
  if (e4m3 && (!aligned(c->k_scale, 16) || (need_v && !aligned(c->v_scale, 16))))
    return FAT_ERR_ALIGNMENT;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.num_pages = static_cast<uint32_t>(c->num_pages);
  v.heads = c->heads;
  v.page_size = c->page_size;
  v.page_shift = shift;
  *out = v;
  return FAT_OK;
}

// (positions below 2^30 + 1, so that 32-bit places and a tile more never overflow)
int table_view(const fat_page_table* t, int page_shift, fat::TableView* out) {
  if (!t || !t->pages || !t->seq_lens || t->width < 1 || t->batch < 1 || t->stride < t->width ||
      (static_cast<long long>(t->width) << page_shift) > (1ll << 30))
    return FAT_ERR_INVALID_ARG;
  if (!aligned(t->pages, 4) || !aligned(t->seq_lens, 4)) return FAT_ERR_ALIGNMENT;
  out->pages = t->pages;
  out->stride = t->stride;
  out->width = t->width;
  out->batch = t->batch;
  out->seq_lens = t->seq_lens;
  return FAT_OK;
}

// query rows against a cache (or bounds) of `heads` heads and type `dtype`
int query_ok(const void* q, int q_dtype, long long batch_stride, long long head_stride,
             int q_heads, int heads, int batch, uint32_t* batch_bytes, uint32_t* head_bytes) {
  if (!q || !wide_type(q_dtype) || q_heads < 1 || q_heads % heads != 0) return FAT_ERR_INVALID_ARG;
  if (static_cast<long long>(batch) * q_heads > (1ll << 30)) return FAT_ERR_INVALID_ARG;
  if (!stride_ok(batch_stride, 2, batch_bytes) || !stride_ok(head_stride, 2, head_bytes) ||
      !aligned(q, 16))
    return FAT_ERR_ALIGNMENT;
  return FAT_OK;
}

// SMs of a device, 0 if CUDA does not say
int sm_count(int dev) {
  int n = 0;
  return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
}

int status(int launch) { return launch == 0 ? FAT_OK : FAT_ERR_LAUNCH; }

}  // namespace

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
  p->scale_log2 = scale * kLog2e;
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
