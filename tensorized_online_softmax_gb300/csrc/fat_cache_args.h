// Checks of the arguments of the C entry points over the paged cache, and the
// kernels' views of them.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/fat_attn.h"
#include "fat_cache.cuh"

namespace fat {

constexpr float kArgLog2e = 1.4426950408889634f;

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool wide_type(int t) { return t == FAT_DTYPE_BF16 || t == FAT_DTYPE_FP16; }

inline int page_shift_of(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

// strides in elements of `bytes` -> bytes; false if a row would not start on 16 bytes or the
// stride is 4 GiB or more
inline bool stride_ok(long long elements, int bytes, uint32_t* out) {
  if (elements < 0 || elements > 0xffffffffll / bytes) return false;
  *out = static_cast<uint32_t>(elements * bytes);
  return *out % 16 == 0;
}

// the cache's description -> the kernels' view of it
inline int cache_view(const fat_kv_cache* c, bool need_v, CacheView* out) {
  if (!c || !c->k || (need_v && !c->v)) return FAT_ERR_INVALID_ARG;
  if (c->heads < 1 || c->num_pages < 1 || (c->d != 64 && c->d != 128)) return FAT_ERR_INVALID_ARG;
  const int shift = page_shift_of(c->page_size);
  if (shift < 0 || c->num_pages > 0x7fffffffll || c->heads > (1 << 20)) return FAT_ERR_INVALID_ARG;
  const bool e4m3 = c->dtype == FAT_DTYPE_E4M3;
  if (!e4m3 && !wide_type(c->dtype)) return FAT_ERR_INVALID_ARG;
  if (e4m3 && (!c->k_scale || (need_v && !c->v_scale))) return FAT_ERR_INVALID_ARG;
  const int bytes = e4m3 ? 1 : 2;
  CacheView v = {};
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
inline int table_view(const fat_page_table* t, int page_shift, TableView* out) {
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
inline int query_ok(const void* q, int q_dtype, long long batch_stride, long long head_stride,
             int q_heads, int heads, int batch, uint32_t* batch_bytes, uint32_t* head_bytes) {
  if (!q || !wide_type(q_dtype) || q_heads < 1 || q_heads % heads != 0) return FAT_ERR_INVALID_ARG;
  if (static_cast<long long>(batch) * q_heads > (1ll << 30)) return FAT_ERR_INVALID_ARG;
  if (!stride_ok(batch_stride, 2, batch_bytes) || !stride_ok(head_stride, 2, head_bytes) ||
      !aligned(q, 16))
    return FAT_ERR_ALIGNMENT;
  return FAT_OK;
}

// SMs of a device, 0 if CUDA does not say
inline int sm_count(int dev) {
  int n = 0;
  return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
}

inline int status(int launch) { return launch == 0 ? FAT_OK : FAT_ERR_LAUNCH; }

}  // namespace fat
