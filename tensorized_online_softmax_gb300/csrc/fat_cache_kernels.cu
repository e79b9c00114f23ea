// Writing tokens to the paged cache (quantising them on the way), reading
// sequences back, and the bounds of the blocks' keys.  All three move each
// byte once and do little arithmetic: they are bound by memory.  Measured on a
// GB300, back to back: 30 880 tokens of 8 heads, d = 128, bf16, quantised and read
// back (456 MB) 67 us, the measured copy rate; fp16, 3 sequences of up to 20 000,
// 12 heads, d = 64, read back after 1024 new tokens each (346 MB) 56 us, 0.92; the
// bounds of one block of 64 positions for 16 sequences and 8 heads 4 us, all of it
// latency (length, page, rows, join).
#include "fat_cache.cuh"

namespace fat {

namespace {

constexpr int kThreads = 256;

// A lane holds so many pieces of eight elements of a row, a row's lanes apart:
// for e4m3, where finding and applying the scale is most of the instructions,
// two (prompts written and read back: 67.1 us instead of 68.7).
template <bool kE4M3>
constexpr int kPieces = kE4M3 ? 2 : 1;

// ---------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------

// Two pieces of one row's lane as 16-bit values -> as codes, and the row's scale
// byte.  kLanes lanes hold the row (a power of two, adjacent).
//
// The scale: the largest magnitude is m 2^E, 1 <= m < 2, and 448 = 1.75 2^8,
// so the least power of two s with amax / s <= 448 is 2^(E - 8), or 2^(E - 7)
// if m > 1.75.  A row below 2^-118 keeps s = 2^-126 (its byte is 1).
template <int kLanes, bool kBf16>
__device__ __forceinline__ void quantise_row(const uint4 (&x)[2], uint2 (&code)[2], uint32_t& e) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  // magnitudes compare as integers, two at a time; an inf or NaN is the largest
  uint32_t two = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) two = __vmaxu2(two, w[i] & 0x7FFF7FFFu);
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1)
    two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, s));
  const uint32_t most = max(two >> 16, two & 0xFFFFu);
  if (most >= (kBf16 ? 0x7F80u : 0x7C00u)) {
    e = 255u;
    code[0] = code[1] = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    return;
  }
  const uint32_t top = __float_as_uint(unpack16<kBf16>(most).x);
  int b = static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  b = top == 0 ? 127 : max(b, 1);
  e = static_cast<uint32_t>(b);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - b) << 23);  // exact
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 f = unpack16<kBf16>(w[2 * i + j]);
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(c[j])
          : "f"(f.y * inv), "f"(f.x * inv));
    }
    h[i] = c[0] | (static_cast<uint32_t>(c[1]) << 16);
  }
  code[0] = make_uint2(h[0], h[1]);
  code[1] = make_uint2(h[2], h[3]);
}

// A thread takes one lane of kWriteRows rows (token, head) of K and V, whose
// loads are all in flight together.  (Two for large calls; one where that many
// threads would not fill the GPU.)
template <int D, bool kE4M3, bool kBf16, int kWriteRows>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const WriteParams p) {
  constexpr int kP = kPieces<kE4M3>, kLanes = D / 8 / kP, kBlockRows = kThreads / kLanes;
  const uint32_t lane = threadIdx.x % kLanes;
  const uint32_t heads = p.c.heads, rows = static_cast<uint32_t>(p.tokens) * heads;
  long long slot[kWriteRows];
  uint32_t head[kWriteRows];
  uint4 k[kWriteRows][kP], v[kWriteRows][kP];
#pragma unroll
  for (int i = 0; i < kWriteRows; ++i) {
    const uint32_t row = (blockIdx.x * kWriteRows + i) * kBlockRows + threadIdx.x / kLanes;
    const uint32_t t = row / heads;
    head[i] = row - t * heads;
    slot[i] = row < rows ? __ldg(p.slots + t) : -1;
    const uint4* kr =
        reinterpret_cast<const uint4*>(p.k + wide(t, p.k_token) + wide(head[i], p.k_head)) + lane;
    const uint4* vr =
        reinterpret_cast<const uint4*>(p.v + wide(t, p.v_token) + wide(head[i], p.v_head)) + lane;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      k[i][j] = v[i][j] = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        k[i][j] = __ldcs(kr + j * kLanes);
        v[i][j] = __ldcs(vr + j * kLanes);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kWriteRows; ++i) {
    const long long slot_page = slot[i] >> p.c.page_shift;
    bool ok = slot[i] >= 0;
    if (ok && slot_page >= p.c.num_pages) {
      atomicOr(p.error_word, kErrIndex);
      ok = false;
    }
    const uint32_t page = static_cast<uint32_t>(slot_page);
    const uint32_t place = static_cast<uint32_t>(slot[i]) & (p.c.page_size - 1);
    uint8_t* kd = p.c.k + row_offset(page, head[i], place, p.c.k_page, p.c.k_head, p.c.k_token);
    uint8_t* vd = p.c.v + row_offset(page, head[i], place, p.c.v_page, p.c.v_head, p.c.v_token);
    if constexpr (!kE4M3) {
      if (ok) {
        reinterpret_cast<uint4*>(kd)[lane] = k[i][0];
        reinterpret_cast<uint4*>(vd)[lane] = v[i][0];
      }
    } else {
      uint2 kc[2], vc[2];
      uint32_t ke, ve;
      quantise_row<kLanes, kBf16>(k[i], kc, ke);
      quantise_row<kLanes, kBf16>(v[i], vc, ve);
      if (ok) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          reinterpret_cast<uint2*>(kd)[lane + j * kLanes] = kc[j];
          reinterpret_cast<uint2*>(vd)[lane + j * kLanes] = vc[j];
        }
        if (lane == 0) {
          const unsigned long long at = scale_offset(p.c, page, head[i], place);
          p.c.k_scale[at] = static_cast<uint8_t>(ke);
          p.c.v_scale[at] = static_cast<uint8_t>(ve);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// read
// ---------------------------------------------------------------------------

template <bool kE4M3>
struct PieceOf {
  using type = uint4;
};
template <>
struct PieceOf<true> {
  using type = uint2;
};

// Eight codes of a row with scale s as 16-bit values.
template <bool kBf16>
__device__ __forceinline__ uint4 widen(uint2 c, float s) {
  uint32_t two[4], r[4];
  e4m3x4_to_f16(c.x, two[0], two[1]);
  e4m3x4_to_f16(c.y, two[2], two[3]);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack16<false>(two[j]);
    // exact in bf16 down to its subnormals; fp16 rounds outside its range
    r[j] = pack16<kBf16>(f.x * s, f.y * s);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// A thread takes one lane of kReadRows positions of one (sequence, head), their
// loads in flight together: a length, a page and then the row are three loads
// one after another, which single rows to a thread would wait for many times
// over.  blockIdx.y walks the sequences and heads.  (Four pieces in all for large
// calls; one row where that many threads would not fill the GPU.)
template <int D, bool kE4M3, bool kBf16, int kReadRows>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadParams p) {
  constexpr int kP = kPieces<kE4M3>, kLanes = D / 8 / kP, kBlockRows = kThreads / kLanes;
  using Piece = typename PieceOf<kE4M3>::type;  // eight elements as cached
  const int lane = threadIdx.x % kLanes;
  const int n0 = blockIdx.x * (kReadRows * kBlockRows) + threadIdx.x / kLanes;
  const long long bh_count = static_cast<long long>(p.t.batch) * p.c.heads;
  for (long long bh = blockIdx.y; bh < bh_count; bh += gridDim.y) {
    const int b = static_cast<int>(bh / p.c.heads);
    const int h = static_cast<int>(bh - static_cast<long long>(b) * p.c.heads);
    const int len = min(table_length(p.t, p.c.page_shift, b), p.max_len);
    const uint8_t* k0 = p.c.k + wide(h, p.c.k_head) + lane * sizeof(Piece);
    const uint8_t* v0 = p.c.v + wide(h, p.c.v_head) + lane * sizeof(Piece);
    int page[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int n = n0 + i * kBlockRows;
      page[i] = n < len ? table_page(p.t, p.c.num_pages, b, n >> p.c.page_shift) : -1;
    }
    Piece k[kReadRows][kP], v[kReadRows][kP];
    uint32_t ks[kReadRows], vs[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int place = (n0 + i * kBlockRows) & (p.c.page_size - 1);
      const uint32_t pg = max(page[i], 0);
      const Piece* kr = reinterpret_cast<const Piece*>(k0 + wide(pg, p.c.k_page) +
                                                       wide(place, p.c.k_token));
      const Piece* vr = reinterpret_cast<const Piece*>(v0 + wide(pg, p.c.v_page) +
                                                       wide(place, p.c.v_token));
      ks[i] = vs[i] = 0;
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        k[i][j] = v[i][j] = Piece{};
        if (page[i] >= 0) {
          k[i][j] = __ldg(kr + j * kLanes);
          v[i][j] = __ldg(vr + j * kLanes);
        }
      }
      if constexpr (kE4M3) {
        if (page[i] >= 0) {
          const unsigned long long at = scale_offset(p.c, pg, h, place);
          ks[i] = __ldg(p.c.k_scale + at);
          vs[i] = __ldg(p.c.v_scale + at);
        }
      }
    }
    const long long out = (bh * p.max_len + n0) * (D / 8) + lane;
    uint4* out_k = reinterpret_cast<uint4*>(p.k) + out;
    uint4* out_v = reinterpret_cast<uint4*>(p.v) + out;
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      if (n0 + i * kBlockRows >= p.max_len) break;
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        const int at = i * kBlockRows * (D / 8) + j * kLanes;
        if constexpr (kE4M3) {
          __stcs(out_k + at, widen<kBf16>(k[i][j], scale_value(ks[i])));
          __stcs(out_v + at, widen<kBf16>(v[i][j], scale_value(vs[i])));
        } else {
          __stcs(out_k + at, k[i][j]);
          __stcs(out_v + at, v[i][j]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// bounds
// ---------------------------------------------------------------------------

// One block of threads per (touched block of a sequence, head); lane -> eight
// elements, the rows shared out over the row groups and joined in shared
// memory.
template <int D, bool kE4M3, bool kBf16>
__global__ void __launch_bounds__(128) kv_bounds_kernel(const BoundsParams p) {
  constexpr int kLanes = D / 8, kGroups = 128 / kLanes;
  __shared__ float lo_s[kGroups][D], hi_s[kGroups][D];
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int h = blockIdx.x;
  for (int b = blockIdx.z; b < p.t.batch; b += gridDim.z) {
    const int len = table_length(p.t, p.c.page_shift, b);
    const int first = max(0, len - p.new_tokens) >> p.c.page_shift;
    const int blocks = (len + p.c.page_size - 1) >> p.c.page_shift;
    for (int i = first + blockIdx.y; i < blocks; i += gridDim.y) {
      const int page = table_page(p.t, p.c.num_pages, b, i);
      if (page < 0) continue;
      const int rows = min(p.c.page_size, len - (i << p.c.page_shift));
      float lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) lo[j] = INFINITY, hi[j] = -INFINITY;
      constexpr int kBatch = 4;  // rows whose loads are in flight together
      const uint8_t* base = p.c.k + wide(page, p.c.k_page) + wide(h, p.c.k_head);
      const uint8_t* scales = p.c.k_scale + scale_offset(p.c, page, h, 0);
      for (int r0 = group; r0 < rows; r0 += kBatch * kGroups) {
        uint4 c[kBatch];
        uint32_t e[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = min(r0 + i * kGroups, rows - 1);  // (the last row again changes nothing)
          const uint8_t* row = base + wide(r, p.c.k_token);
          if constexpr (kE4M3) {
            const uint2 two = __ldg(reinterpret_cast<const uint2*>(row) + lane);
            c[i].x = two.x, c[i].y = two.y;
            e[i] = __ldg(scales + r);
          } else {
            c[i] = __ldg(reinterpret_cast<const uint4*>(row) + lane);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          float x[8];
          if constexpr (kE4M3) {
            const float s = scale_value(e[i]);
            uint32_t two[4];
            e4m3x4_to_f16(c[i].x, two[0], two[1]);
            e4m3x4_to_f16(c[i].y, two[2], two[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = unpack16<false>(two[j]);
              x[2 * j] = f.x * s, x[2 * j + 1] = f.y * s;
            }
          } else {
            const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = unpack16<kBf16>(w[j]);
              x[2 * j] = f.x, x[2 * j + 1] = f.y;
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) lo[j] = min_nan(lo[j], x[j]), hi[j] = max_nan(hi[j], x[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo_s[group][lane * 8 + j] = lo[j];
        hi_s[group][lane * 8 + j] = hi[j];
      }
      __syncthreads();
      // D / 2 pairs of columns, low then high
      uint32_t* out = reinterpret_cast<uint32_t*>(p.bounds) + (wide(page, p.c.heads) + h) * D;
      for (int c = threadIdx.x; c < D; c += 128) {
        const bool high = c >= D / 2;
        const int col = 2 * (high ? c - D / 2 : c);
        float a = high ? hi_s[0][col] : lo_s[0][col];
        float z = high ? hi_s[0][col + 1] : lo_s[0][col + 1];
#pragma unroll
        for (int g = 1; g < kGroups; ++g) {
          a = high ? max_nan(a, hi_s[g][col]) : min_nan(a, lo_s[g][col]);
          z = high ? max_nan(z, hi_s[g][col + 1]) : min_nan(z, lo_s[g][col + 1]);
        }
        out[c] = pack16<kBf16>(a, z);
      }
      __syncthreads();
    }
  }
}

int launched() { return cudaGetLastError() == cudaSuccess ? 0 : -4; }

}  // namespace

// Rows to a thread: `most` if that still gives every SM two blocks, else one.
static int rows_per_thread(long long rows, int lanes, int most, int sms) {
  return rows * lanes >= 2ll * most * kThreads * sms ? most : 1;
}

int launch_kv_write(const WriteParams& p, int d, bool e4m3, bool bf16, int sms,
                    cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.tokens) * p.c.heads;
  const int lanes = d / (e4m3 ? 16 : 8), many = rows_per_thread(rows, lanes, 2, sms);
  const int each = many * kThreads / lanes;
  const unsigned grid = static_cast<unsigned>((rows + each - 1) / each);
#define FAT_RUN(D, E, B)                                              \
  (many == 2 ? kv_write_kernel<D, E, B, 2><<<grid, kThreads, 0, stream>>>(p) \
             : kv_write_kernel<D, E, B, 1><<<grid, kThreads, 0, stream>>>(p))
  FAT_PICK(d, e4m3, bf16, FAT_RUN);
#undef FAT_RUN
  return launched();
}

int launch_kv_read(const ReadParams& p, int d, bool e4m3, bool bf16, int sms,
                   cudaStream_t stream) {
  const long long bh = static_cast<long long>(p.t.batch) * p.c.heads;
  const int lanes = d / (e4m3 ? 16 : 8);
  const int many = rows_per_thread(bh * p.max_len, lanes, e4m3 ? 2 : 4, sms);
  const int rows = many * kThreads / lanes;
  const dim3 grid(p.max_len / rows + (p.max_len % rows != 0),
                  static_cast<unsigned>(bh < 65535 ? bh : 65535));
#define FAT_RUN(D, E, B)                                             \
  (many > 1 ? kv_read_kernel<D, E, B, 4 / kPieces<E>><<<grid, kThreads, 0, stream>>>(p) \
            : kv_read_kernel<D, E, B, 1><<<grid, kThreads, 0, stream>>>(p))
  FAT_PICK(d, e4m3, bf16, FAT_RUN);
#undef FAT_RUN
  return launched();
}

int launch_kv_bounds(const BoundsParams& p, int d, bool e4m3, bool bf16, cudaStream_t stream) {
  // blocks that new_tokens adjacent positions can touch
  long long most = (static_cast<long long>(p.new_tokens) + p.c.page_size - 2) / p.c.page_size + 1;
  if (most > p.t.width) most = p.t.width;
  const dim3 grid(p.c.heads, static_cast<unsigned>(most < 65535 ? most : 65535),
                  p.t.batch < 65535 ? p.t.batch : 65535);
#define FAT_RUN(D, E, B) kv_bounds_kernel<D, E, B><<<grid, 128, 0, stream>>>(p)
  FAT_PICK(d, e4m3, bf16, FAT_RUN);
#undef FAT_RUN
  return launched();
}

}  // namespace fat
