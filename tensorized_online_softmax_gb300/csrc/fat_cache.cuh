// The paged key-value cache as the kernels see it, and the conversions between
// its row formats.
//
// An e4m3 row holds d codes and one scale byte e; its values are
// code * 2^(e - 127), e = 255 standing for a row with an inf or NaN.  A power
// of two costs e4m3 no precision (its relative step does not depend on the
// scale) and makes quantising exact up to the one rounding of the code, and
// one byte instead of an fp32 scale keeps the scales below 1 % of the row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fat_launch.cuh"

namespace fat {

// strides in bytes, in 32 bits: a row's address is then a few multiply-adds that
// widen, not 64-bit products
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scale;  // [num_pages, heads, page_size]
  uint8_t* v_scale;
  uint32_t k_page, k_head, k_token;
  uint32_t v_page, v_head, v_token;
  uint32_t num_pages;
  int heads, page_size, page_shift;
};

__device__ __forceinline__ unsigned long long wide(uint32_t a, uint32_t b) {
  return static_cast<unsigned long long>(a) * b;
}
// Row `place` of head h of a page: its byte offset, and its place among the scales.
__device__ __forceinline__ unsigned long long row_offset(uint32_t page, uint32_t h, uint32_t place,
                                                         uint32_t page_stride,
                                                         uint32_t head_stride,
                                                         uint32_t token_stride) {
  return wide(page, page_stride) + wide(h, head_stride) + wide(place, token_stride);
}
__device__ __forceinline__ unsigned long long scale_offset(const CacheView& c, uint32_t page,
                                                           uint32_t h, uint32_t place) {
  return ((wide(page, c.heads) + h) << c.page_shift) + place;
}

struct TableView {
  const int* pages;
  long long stride;  // entries between sequences
  int width;
  int batch;
  const int* seq_lens;
  unsigned int* error_word;
};

// (Lengths and pages by plain loads: the choice of blocks writes them while the
// decode kernel that waits for it has started, which read-only loads forbid.)

// Length of sequence b: at most what the table can hold, never negative.
__device__ __forceinline__ int table_length(const TableView& t, int page_shift, int b) {
  const int n = t.seq_lens[b];
  const long long most = static_cast<long long>(t.width) << page_shift;
  if (n < 0 || n > most) {
    atomicOr(t.error_word, kErrIndex);
    return n < 0 ? 0 : static_cast<int>(most);
  }
  return n;
}

// Page i of sequence b, or -1 (flagged) if it is not a page of the cache.
__device__ __forceinline__ int table_page(const TableView& t, uint32_t num_pages, int b, int i) {
  const int p = t.pages[b * t.stride + i];
  if (static_cast<uint32_t>(p) >= num_pages) {
    atomicOr(t.error_word, kErrIndex);
    return -1;
  }
  return p;
}

// 2^(e - 127) of a scale byte; NaN for 255 (e >= 1: never a subnormal)
__device__ __forceinline__ float scale_value(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7FFFFFFFu : e << 23);
}

// four e4m3 codes -> four fp16 (exact; a NaN code becomes NaN)
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

template <bool kBf16>
__device__ __forceinline__ float2 unpack16(uint32_t two) {
  if constexpr (kBf16) {
    return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xFFFF0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&two));
  }
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// X(head dim, e4m3 cache, bf16 queries or outputs) of the run-time values
#define FAT_PICK(D, E, B, ...)                                    \
  do {                                                            \
    if (D == 128)                                                 \
      E ? (B ? __VA_ARGS__(128, true, true) : __VA_ARGS__(128, true, false))     \
        : (B ? __VA_ARGS__(128, false, true) : __VA_ARGS__(128, false, false));  \
    else                                                          \
      E ? (B ? __VA_ARGS__(64, true, true) : __VA_ARGS__(64, true, false))       \
        : (B ? __VA_ARGS__(64, false, true) : __VA_ARGS__(64, false, false));    \
  } while (0)

// ---- launchers (fat_cache_kernels.cu, fat_decode_d128.cu, fat_decode_d64.cu,
// fat_block_select.cu): 0, or -4 for a CUDA error ----
struct WriteParams {
  CacheView c;
  const uint8_t* k;
  const uint8_t* v;
  uint32_t k_token, k_head, v_token, v_head;  // bytes
  const long long* slots;
  int tokens;
  unsigned int* error_word;
};
int launch_kv_write(const WriteParams& p, int d, bool e4m3, bool bf16, int sms,
                    cudaStream_t stream);

struct ReadParams {
  CacheView c;
  TableView t;
  uint8_t* k;
  uint8_t* v;
  int max_len;
};
int launch_kv_read(const ReadParams& p, int d, bool e4m3, bool bf16, int sms,
                   cudaStream_t stream);

struct BoundsParams {
  CacheView c;
  TableView t;
  uint8_t* bounds;
  int new_tokens;
};
int launch_kv_bounds(const BoundsParams& p, int d, bool e4m3, bool bf16, cudaStream_t stream);

struct ScoreParams {
  TableView t;
  const uint8_t* q;
  uint32_t q_batch, q_head;  // bytes
  const uint8_t* bounds;
  uint32_t num_pages;
  int heads, group, page_shift;
  float* scores;
};
int launch_kv_scores(const ScoreParams& p, int d, bool bf16, int dev, int sms,
                     cudaStream_t stream);

// Sequences of a decode call are its table's entries: one per sequence, whose
// cached heads share it, or (per_head) one per (sequence, cached head).
struct DecodeParams {
  CacheView c;
  TableView t;
  int per_head;
  const uint8_t* q;
  uint32_t q_batch, q_head;  // bytes
  int group;                  // query heads per cached head
  float scale_log2;           // scale * log2(e)
  uint8_t* o;
  float* lse;
  void* workspace;
  int direct;                 // each block has one item (set by the launch)
  int least_tiles;            // tiles that a thread block takes at least
};
// what launch_decode needs, whatever the batch
size_t decode_workspace_bytes(int d);
int launch_decode(const DecodeParams& p, int d, bool e4m3, bool bf16, int dev,
                  cudaStream_t stream);

struct SelectParams {
  TableView t;
  const float* scores;  // [batch, heads, width]
  int heads, page_shift;
  int num_blocks, first_blocks, last_blocks;
  int* blocks;  // [batch, heads, num_blocks]: the choice, in rising order, then -1
  int* pages;   // [batch, heads, list]: its pages
  int list;     // min(num_blocks, width)
  int* lens;    // [batch, heads]: positions in those pages
};
int launch_select(const SelectParams& p, cudaStream_t stream);

}  // namespace fat
