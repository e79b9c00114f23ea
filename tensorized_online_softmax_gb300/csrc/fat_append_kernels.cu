// Storing new tokens in the paged cache with the rotation of queries and keys by
// their positions on the way, and moving the rows of accepted drafted tokens.
// Both move each byte once with little arithmetic: they are bound by memory, and
// small calls by the latency of a chain of dependent loads (position, then the
// table of cosines; path, page, row).
//
// Measured on a GB300, on the device: prompts of 1000 to 8192 tokens, 48 heads of
// 128, bf16, positions of three axes (764 MB in and out): 122 us, 0.92 of the copy
// rate; the same with one axis in fp16 117 us, 0.96; into an e4m3 cache 149 (63 MB
// less to write; the conversion's instructions), three axes 168; 16 single tokens
// into an e4m3 cache and back: 4.6 us for both kernels; 64 sequences of 64 drafted
// tokens stored and up to 12 of them kept: 19.5 us, 0.80; keeping alone, 8 heads: up to
// 12 of 64 3.4 us, 32 4.9, 60 (31 MB) 7.2, in an e4m3 cache 3.5, 4.0, 4.9.
//
// Rotation: for pair i of a row, with (c, s) the table's cosine and sine at the
// token's position,  y_a = x_a c - x_b s,  y_b = x_b c + x_a s.  Products and sums
// are rounded one by one in fp32 (no FMA): the result is what the same formula
// gives in any fp32 program, so that a cache holds the same codes whoever wrote
// it.  The table is an argument: far positions' angles are the caller's to form in
// as many bits as they need.
#include "fat_cache.cuh"

namespace fat {

namespace {

constexpr int kThreads = 256;

// Sixteen elements of a row in fp32: x[0..7] of chunk a, x[8..15] of chunk b.
template <bool kBf16>
__device__ __forceinline__ void unpack_chunks(const uint4& a, const uint4& b, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack16<kBf16>(w[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}

template <bool kBf16>
__device__ __forceinline__ void pack_chunks(const float (&x)[16], uint4& a, uint4& b) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack16<kBf16>(x[2 * i], x[2 * i + 1]);
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}

// One row as codes, and its scale byte (row_scale_byte).  `group` is the mask of the
// kLanes lanes that hold the row.
template <int kLanes>
__device__ __forceinline__ void quantise(const float (&x)[16], uint32_t group, uint2& a, uint2& b,
                                         uint32_t& e) {
  uint32_t top = 0;  // magnitudes compare as integers; an inf or NaN is the largest
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(group, top, s));
  e = row_scale_byte(top);
  if (e == 255u) {
    a = b = make_uint2(kNanCodes, kNanCodes);
    return;
  }
  const float inv = row_scale_inverse(e);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = codes_of(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], inv);
  a = make_uint2(w[0], w[1]);
  b = make_uint2(w[2], w[3]);
}

// A thread takes two chunks of eight elements of kHeads heads of one token, all
// queries, all keys or all values: their loads are in flight together, and the
// cosines are loaded once for them.  The two chunks hold both members of their
// eight pairs: chunks l and l + n / 16 where the halves of the rotated n elements
// are paired, 2 l and 2 l + 1 where neighbours are (and for what is not rotated).
template <int D, bool kE4M3, bool kBf16, bool kInter, int kHeads>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 16;
  const int lane = threadIdx.x % kLanes;
  const uint32_t group = ((1u << kLanes) - 1u) << (threadIdx.x % 32 / kLanes * kLanes);
  const uint32_t q_segs = (p.q_heads + kHeads - 1) / kHeads;
  const uint32_t kv_segs = (p.c.heads + kHeads - 1) / kHeads;
  const uint32_t segs = q_segs + 2 * kv_segs;
  const uint32_t job = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const uint32_t token = job / segs;
  if (token >= static_cast<uint32_t>(p.tokens)) return;
  uint32_t seg = job - token * segs;
  const bool is_q = seg < q_segs, is_v = seg >= q_segs + kv_segs;
  if (!is_q) seg -= is_v ? q_segs + kv_segs : q_segs;
  const int head0 = static_cast<int>(seg) * kHeads;
  const int heads = is_q ? p.q_heads : p.c.heads;

  const int rotated_lanes = p.pairs / 8;
  const bool turns = !is_v && lane < rotated_lanes;
  // chunks of eight elements
  const int a = kInter ? 2 * lane : (lane < rotated_lanes ? lane : 2 * lane);
  const int b = kInter ? a + 1 : (lane < rotated_lanes ? lane + rotated_lanes : 2 * lane + 1);

  const uint8_t* from = is_q   ? p.q + wide(token, p.q_token) + wide(head0, p.q_head)
                        : is_v ? p.v + wide(token, p.v_token) + wide(head0, p.v_head)
                               : p.k + wide(token, p.k_token) + wide(head0, p.k_head);
  const uint32_t step = is_q ? p.q_head : is_v ? p.v_head : p.k_head;
  uint4 xa[kHeads], xb[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
    if (head0 + i < heads) {
      // (q may be rotated in place: no read-only loads)
      const uint4* row = reinterpret_cast<const uint4*>(from + wide(i, step));
      xa[i] = __ldcs(row + a);
      xb[i] = __ldcs(row + b);
    }
  }
  // Every axis' position is looked at by every lane, so that a token is left out as a whole.
  bool ok = true;
  float cs[8], sn[8];
  long long at[4] = {0, 0, 0, 0};
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (x < p.axes) {
      at[x] = __ldg(p.positions + x * p.axis_stride + token * p.token_stride);
      ok &= at[x] >= 0 && at[x] < p.rows;
    }
  if (turns && ok) {
    const int i0 = lane * 8;
    if (p.axes == 1) {
      const float* row = p.cos_sin + at[0] * p.row_stride + i0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(row) + j);
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + p.pairs) + j);
        cs[4 * j] = c4.x, cs[4 * j + 1] = c4.y, cs[4 * j + 2] = c4.z, cs[4 * j + 3] = c4.w;
        sn[4 * j] = s4.x, sn[4 * j + 1] = s4.y, sn[4 * j + 2] = s4.z, sn[4 * j + 3] = s4.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j;
        const long long where = i < p.ends[0]   ? at[0]
                                : i < p.ends[1] ? at[1]
                                : i < p.ends[2] ? at[2]
                                                : at[3];
        const float* row = p.cos_sin + where * p.row_stride + i;
        cs[j] = __ldg(row);
        sn[j] = __ldg(row + p.pairs);
      }
    }
  }
  if (!ok) {  // neither stored nor given out
    if (lane == 0 && seg == 0) atomicOr(p.error_word, kErrIndex);
    return;
  }
  long long slot = 0;
  if (!is_q) {
    slot = __ldg(p.slots + token);
    if (slot < 0) return;
    if ((slot >> p.c.page_shift) >= p.c.num_pages) {
      if (lane == 0 && seg == 0) atomicOr(p.error_word, kErrIndex);
      return;
    }
  }
  const uint32_t page = static_cast<uint32_t>(slot >> p.c.page_shift);
  const uint32_t place = static_cast<uint32_t>(slot) & (p.c.page_size - 1);
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = head0 + i;
    if (h >= heads) break;
    if (turns || (kE4M3 && !is_q)) {
      float x[16];
      unpack_chunks<kBf16>(xa[i], xb[i], x);
      if (turns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float& u = x[kInter ? 2 * j : j];
          float& w = x[kInter ? 2 * j + 1 : 8 + j];
          const float y = __fsub_rn(__fmul_rn(u, cs[j]), __fmul_rn(w, sn[j]));
          w = __fadd_rn(__fmul_rn(w, cs[j]), __fmul_rn(u, sn[j]));
          u = y;
        }
      }
      if constexpr (kE4M3) {
        if (!is_q) {
          uint2 ca, cb;
          uint32_t e;
          quantise<kLanes>(x, group, ca, cb, e);
          uint8_t* row =
              is_v ? p.c.v + row_offset(page, h, place, p.c.v_page, p.c.v_head, p.c.v_token)
                   : p.c.k + row_offset(page, h, place, p.c.k_page, p.c.k_head, p.c.k_token);
          reinterpret_cast<uint2*>(row)[a] = ca;
          reinterpret_cast<uint2*>(row)[b] = cb;
          if (lane == 0)
            (is_v ? p.c.v_scale : p.c.k_scale)[scale_offset(p.c, page, h, place)] =
                static_cast<uint8_t>(e);
          continue;
        }
      }
      pack_chunks<kBf16>(x, xa[i], xb[i]);
    }
    uint8_t* row =
        is_q   ? p.q_out + (wide(token, p.q_heads) + h) * (2 * D)
        : is_v ? p.c.v + row_offset(page, h, place, p.c.v_page, p.c.v_head, p.c.v_token)
               : p.c.k + row_offset(page, h, place, p.c.k_page, p.c.k_head, p.c.k_token);
    reinterpret_cast<uint4*>(row)[a] = xa[i];
    reinterpret_cast<uint4*>(row)[b] = xb[i];
  }
}

// ---------------------------------------------------------------------------
// keep
// ---------------------------------------------------------------------------

// A block takes the rows of one (sequence, head), K or V, each thread 16 bytes of a row: a wave of
// rows is in registers before any is stored.  (Waves of 1, 2, 4 and 8 rows to a thread, the 64
// sequences above with up to 12, 32 and 60 kept: 3.4, 3.4, 4.0, 5.5 us, 5.1, 4.9, 5.4, 7.2 and 7.8,
// 7.2, 7.9, 10.3; e4m3 with 60 5.3, 4.9, 5.7, 7.5.)  As the path rises, a wave's rows come from its first place on or behind it, where no earlier wave has
// written: so only a wave's own loads and stores are held apart.
__global__ void __launch_bounds__(kThreads) kv_keep_kernel(const KeepParams p) {
  constexpr int kDeep = 2;
  const int each = kThreads / p.chunks;  // rows at a time, 16 bytes to a thread
  const int row0 = threadIdx.x / p.chunks, chunk = threadIdx.x - row0 * p.chunks;
  const bool is_v = blockIdx.x & 1;
  const int b = static_cast<int>(blockIdx.x >> 1) / p.c.heads;
  const uint32_t h = (blockIdx.x >> 1) - b * p.c.heads;
  const long long most = static_cast<long long>(p.t.width) << p.c.page_shift;
  const int base = p.t.seq_lens[b];
  const int count = p.counts[b];
  if (base < 0 || base > most || count < 0 || count > p.width) {
    if (threadIdx.x == 0) atomicOr(p.t.error_word, kErrIndex);
    return;
  }
  uint8_t* data = is_v ? p.c.v : p.c.k;
  const uint32_t page_stride = is_v ? p.c.v_page : p.c.k_page;
  const uint32_t head_stride = is_v ? p.c.v_head : p.c.k_head;
  const uint32_t token_stride = is_v ? p.c.v_token : p.c.k_token;
  uint8_t* scales = is_v ? p.c.v_scale : p.c.k_scale;
  const int* path = p.path + b * p.path_stride;
  // the page of a position, or -1 (flagged)
  auto page_of = [&](long long at) {
    if (at < 0 || at >= most) {
      atomicOr(p.t.error_word, kErrIndex);
      return -1;
    }
    return table_page(p.t, p.c.num_pages, b, static_cast<int>(at >> p.c.page_shift));
  };
  auto row_of = [&](int page, uint32_t at) {
    return reinterpret_cast<uint4*>(
               data + row_offset(page, h, at, page_stride, head_stride, token_stride)) + chunk;
  };
  for (int i0 = 0; i0 < count; i0 += kDeep * each) {
    uint4 x[kDeep];
    uint8_t e[kDeep];
    int to_page[kDeep];
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const int i = i0 + j * each + row0;
      to_page[j] = -1;
      if (i >= count) continue;
      const int step = __ldg(path + i);
      if (step < 0) atomicOr(p.t.error_word, kErrIndex);
      if (step < 0 || step == i) continue;  // (it is where it belongs)
      const long long at = static_cast<long long>(base) + step;
      const int page = page_of(at);
      const int to = page_of(static_cast<long long>(base) + i);
      if (page < 0 || to < 0) continue;
      const uint32_t place = static_cast<uint32_t>(at) & (p.c.page_size - 1);
      to_page[j] = to;
      x[j] = *row_of(page, place);
      if (p.scales && chunk == 0) e[j] = scales[scale_offset(p.c, page, h, place)];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      if (to_page[j] < 0) continue;
      const uint32_t place =
          static_cast<uint32_t>(base + i0 + j * each + row0) & (p.c.page_size - 1);
      *row_of(to_page[j], place) = x[j];
      if (p.scales && chunk == 0) scales[scale_offset(p.c, to_page[j], h, place)] = e[j];
    }
  }
}

int launched() { return cudaGetLastError() == cudaSuccess ? 0 : -4; }

}  // namespace

int launch_kv_append(const AppendParams& p, int d, bool e4m3, bool bf16, bool interleaved, int sms,
                     cudaStream_t stream) {
  const int lanes = d / 16, jobs = kThreads / lanes;
  auto segments = [&](int heads) {
    return static_cast<long long>(p.tokens) *
           ((p.q_heads + heads - 1) / heads + 2 * ((p.c.heads + heads - 1) / heads));
  };
  // Four heads to a thread if that still gives every SM two blocks, else one: the prompts above
  // take 122 us with four, 212 with one, the 16 tokens (with their reading) 5.9 and 4.6.
  const bool many = segments(4) * lanes >= 2ll * kThreads * sms;
  const unsigned grid = static_cast<unsigned>((segments(many ? 4 : 1) + jobs - 1) / jobs);
#define FAT_RUN(D, E, B)                                                                   \
  (interleaved ? (many ? kv_append_kernel<D, E, B, true, 4><<<grid, kThreads, 0, stream>>>(p)   \
                       : kv_append_kernel<D, E, B, true, 1><<<grid, kThreads, 0, stream>>>(p))  \
               : (many ? kv_append_kernel<D, E, B, false, 4><<<grid, kThreads, 0, stream>>>(p)  \
                       : kv_append_kernel<D, E, B, false, 1><<<grid, kThreads, 0, stream>>>(p)))
  FAT_PICK(d, e4m3, bf16, FAT_RUN);
#undef FAT_RUN
  return launched();
}

int launch_kv_keep(const KeepParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(2ll * p.t.batch * p.c.heads);
  kv_keep_kernel<<<grid, kThreads, 0, stream>>>(p);
  return launched();
}

}  // namespace fat
