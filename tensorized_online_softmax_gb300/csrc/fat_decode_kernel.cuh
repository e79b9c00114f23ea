// Attention of one query token per sequence over the paged cache.
//
// What bounds it: every cached byte is used once, by the few query heads of its
// group, so the kernel is a stream through HBM; all else has to stay below it.
//
// Work: fat_decode_plan.h.  Each of a block's four warps takes 16 positions of
// every 64-position tile through a ring of its own in shared memory, filled by
// 16-byte asynchronous copies one to three tiles ahead, by layout (a ring per warp needs no
// barrier between warps; 16 positions never straddle two pages).  Rows behind
// the length are filled with zeros, not read.
//
// Arithmetic per 16 positions, on m16n8k16 MMAs with the positions as rows, so
// that a group of up to 8 query heads (kNT = 1; 16: kNT = 2) fills the columns:
//     S[16, heads] = K Q^T,   z = scale log2(e) S   (-inf behind the length)
//     p = 2^(z - r),  l += p,   O^T[d, heads] += V^T P^T
// r is a running reference for each head, raised to the running maximum only
// when a score exceeds it by more than 8 binades (fp16 weights: 4), so the usual
// tile needs one vote and no reduction over lanes.  P enters the MMA as a 16-bit
// value plus the 16-bit remainder (two MMAs): its rounding stays below 2^-16 and
// the only rounding that counts is that of the output.  fp16 weights are 2^11 at
// the maximum, up to 2^15 where it was let pass: a weight is off by at most 2^-25,
// 2^-36 of the largest, besides its relative rounding.
//
// e4m3 caches: the codes become fp16 exactly, the keys' scales multiply S, and
// the values' scales join the weights, w = 2^(z + log2 s - r'), with a running
// reference r' of its own, set by the rows that are not all zeros: fp16 weights
// keep their precision relative to the largest w 2^8 (a row's largest code is
// near 2^8, as written) whatever the scales are.  q is brought into fp16's range
// by a power of two for each head, without loss: a query with elements more than
// 32 binades apart takes its low parts, down to 2^-70 of the largest, by a second
// pass over the staged keys.
//
// The warps' (r, r', l, O) are joined through shared memory at an item's end;
// an item that other blocks share leaves a normalised O and its LSE in the
// workspace for the join kernel, in a fixed order: the result does not depend
// on timing.
//
// Measured on a GB300, calls back to back on the device: 32 sequences of 1000 to
// 8192 positions, 8 cached heads of 4 query heads, d = 128, bf16 (599 MB): 94 to
// 95.4 us, 0.93 of the measured copy rate (the stream itself 0.985; the rest is the
// plan, 2.5 us to the first rows, and 4 us of end and join); one sequence of 131072
// (537 MB): 85.3 us; 64 sequences of 4096 to 16384, groups of 8, e4m3 (1417 MB):
// 223 us, 0.94; 13 of 0 to 4097, 20 heads, d = 64, fp16 (148 MB): 30 us, 0.73.
// The 32 sequences with groups of 16: bf16 101 us, e4m3 91 (304 MB, 45 at the copy
// rate: 8 warps an SM do not hide the instructions' latency); of 64: 335, as every
// 16 heads are a pass of their own.
#pragma once

#include "fat_cache.cuh"
#include "fat_decode_plan.h"
#include "sm103_ptx.cuh"

namespace fat {

namespace decode {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRowsPerWarp = kDecodeTile / kWarps;  // 16
static_assert(kRowsPerWarp == 16, "one MMA tile of positions to a warp");
// Binades above the maximum at the last raise that are let pass: of scores, and of fp16 weights,
// which are 2^kShiftF16 at that maximum.  The fewer, the further down they reach, and the more
// often they are raised: with 8, 4, 3 and 2 (e4m3, d = 64, 16 heads) 61.9, 62.5, 63.5 and 64.7 us;
// d = 128, 8 heads 219.8, 220.0, 220.3, 220.8; fp16 caches alike.
constexpr float kRaise = 8.f, kRaiseF16 = 4.f, kShiftF16 = 15.f - kRaiseF16;

struct Join {  // what the join kernel needs of the item that starts, unfinished, in a block
  int entry, item;
  int last;  // the last block with a part of it; -1: nothing to join
  int part;  // where the first block keeps its part
};

// workspace: Join[kDecodeMaxBlocks], then for each block and part the LSEs
// (log2) of up to 16 rows, then the rows
constexpr int kMaxRows = 16;
constexpr size_t kJoinBytes = sizeof(Join) * kDecodeMaxBlocks;
constexpr size_t kLseBytes = sizeof(float) * kDecodeMaxBlocks * 2 * kMaxRows;

template <int D, int kNT, bool kE4M3>
struct Layout {
  static constexpr int kRow = D * (kE4M3 ? 1 : 2);  // bytes
  static constexpr int kChunks = kRow / 16;
  static constexpr int kStage = 2 * kRowsPerWarp * kRow;  // K and V of 16 positions
  static constexpr int kScales = kE4M3 ? 32 : 0;
  // blocks on an SM: what their registers allow, but three where memory is the bound already
  // (a fourth saves 7 % of the e4m3 kernel at d = 64, and costs 1 % of the 16-bit one)
  static constexpr int kBlocks = kNT > 1 ? (D == 64 ? 3 : 2) : (D == 64 && kE4M3 ? 4 : 3);
  // S is summed in so many chains: an MMA's result takes a while, but registers are scarce
  // where there are 16 heads (one chain: 2 % there)
  static constexpr int kChains = kNT > 1 ? 1 : D == 64 ? 2 : 4;
  // the rings of an SM: deeper ones gain nothing once HBM's latency is covered (e4m3, d = 128:
  // 2 stages 223 us, 3 226, 4 234 for the 64 sequences above, when they were compared; 16-bit,
  // d = 64: 3 stages 29.5 us, 2 30.1, 4 30.0 for the 13)
  static constexpr int kRoom = (kE4M3 ? 112 : 150) * 1024 / (kBlocks * kWarps);  // of one warp
  static constexpr int kFit = kRoom / (kStage + kScales);
  static constexpr int kStages = kFit < 2 ? 2 : kFit;
  static constexpr int kRing = kStages * (kStage + kScales);  // of one warp
  static_assert(8 * D * 4 <= kStage, "a stage holds a warp's O for the join");
  static constexpr int kJoinRows = 3 * kWarps * kMaxRows * 4;
  static constexpr int kSmem = kWarps * kRing + kJoinRows;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two weights rounded down to 16 bits, strictly below the weight itself, so that
// the remainder is positive: with an infinite value both products have its sign
// (a remainder of zero or of the other sign would make their sum a NaN).  In fp16
// that holds for weights from 2^-23 on, 2^-34 of the largest; below, an infinite
// value gives NaN.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack_below(float a, float b) {
  constexpr float kLess = 1.f - 0x1p-10f;  // less than a step of either type away
  uint32_t r;
  if constexpr (kBf16) {
    r = __byte_perm(__float_as_uint(a * kLess), __float_as_uint(b * kLess), 0x7632);
  } else {
    constexpr float kLeast = 0x1p-24f;  // what fp16 can still hold
    a = fmaxf(fminf(a * kLess, a - kLeast), 0.f);
    b = fmaxf(fminf(b * kLess, b - kLeast), 0.f);
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  }
  return r;
}

// The byte offset of 16-byte chunk c of row r in a stage: chunks are permuted
// within a row so that eight rows' worth of one chunk meet no bank twice.
template <int kChunks>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (kChunks >= 8)
    return static_cast<uint32_t>(r * kChunks + (c ^ (r & 7))) * 16u;
  else
    return static_cast<uint32_t>(r * kChunks + (c ^ ((r >> 1) & 3))) * 16u;
}

// bf16 queries as fp16 scaled by a power of two, `down`: the parts that are left
// behind, as fp16 times 2^39 (an element below 2^-17 there is a subnormal, off by
// 2^-25 at most; larger ones are exact).
constexpr float kLowScale = 0x1p39f;
__device__ __forceinline__ uint32_t low_part(uint32_t two, float down) {
  const float2 f = unpack16<true>(two);
  const float x = f.x * down, y = f.y * down;
  const float2 held = unpack16<false>(pack16<false>(x, y));
  return pack16<false>(fabsf(x) < 0x1p-16f ? (x - held.x) * kLowScale : 0.f,
                       fabsf(y) < 0x1p-16f ? (y - held.y) * kLowScale : 0.f);
}

// Inclusive prefix sum over the block's threads.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums,
                                                long long& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) x += warp_sums[w];
    total += warp_sums[w];
  }
  return x;
}

// What an item is: its sequence, cached head and first query head of the group.
struct Item {
  int seq, head, row0;
};
__device__ __forceinline__ Item item_of(const DecodeParams& p, const DecodePlace& at, int rows,
                                        int blocks_of_rows) {
  const int h = at.item / blocks_of_rows;
  Item r;
  r.row0 = (at.item - h * blocks_of_rows) * rows;
  r.seq = p.per_head ? at.entry / p.c.heads : at.entry;
  r.head = p.per_head ? at.entry - r.seq * p.c.heads : h;
  return r;
}

__device__ __forceinline__ int enter(const DecodeParams& p, DecodePlace& at) {
  const int len = table_length(p.t, p.c.page_shift, at.entry);
  at.tiles = decode_tiles(len);
  return len;
}

template <int D, int kNT, bool kE4M3, bool kBf16>
__global__ void __launch_bounds__(kThreads, Layout<D, kNT, kE4M3>::kBlocks)
    decode_kernel(const DecodeParams p) {
  using L = Layout<D, kNT, kE4M3>;
  constexpr bool kMmaBf16 = kBf16 && !kE4M3;
  constexpr int kR = 8 * kNT;  // query heads of a block of rows
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long warp_sums[kWarps];
  __shared__ DecodePlace start_s;
  __shared__ float down_s[kWarps][kR];  // the power of two that a head's query was scaled by
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  // [3][warp][kMaxRows]: r, r', l
  float* join_r = reinterpret_cast<float*>(smem + kWarps * L::kRing);

  grid_dep_launch();
  grid_dep_wait();

  // ---- the block's share ----
  const int blocks_of_rows = (p.group + kR - 1) / kR;
  const int heads_per_entry = p.per_head ? 1 : p.c.heads;
  const int copies = heads_per_entry * blocks_of_rows;
  long long begin, share, total;
  if (p.direct) {
    const int e = blockIdx.x / copies;
    if (threadIdx.x == 0) {
      start_s.entry = e;
      start_s.item = blockIdx.x - e * copies;
      start_s.tile = 0;
    }
    begin = 0;
    share = total = decode_tiles(table_length(p.t, p.c.page_shift, e));
    __syncthreads();
  } else {
    const int entries = p.t.batch;
    const int each = (entries + kThreads - 1) / kThreads;
    const int lo = threadIdx.x * each, hi = min(entries, lo + each);
    long long mine = 0;
    for (int e = lo; e < hi; ++e) mine += decode_tiles(table_length(p.t, p.c.page_shift, e));
    const long long upto = block_scan(mine, warp_sums, total);
    total *= copies;
    // (a 64-bit division is a few hundred cycles)
    share = total <= 0x7fffffff - kDecodeMaxBlocks
                ? decode_share(static_cast<int>(total), gridDim.x, p.least_tiles)
                : decode_share(total, static_cast<int>(gridDim.x), p.least_tiles);
    begin = blockIdx.x * share;
    long long before = (upto - mine) * copies;
    if (begin >= before && begin < upto * copies) {
      for (int e = lo; e < hi; ++e) {
        const int tiles = decode_tiles(table_length(p.t, p.c.page_shift, e));
        const long long n = static_cast<long long>(tiles) * copies;
        if (begin < before + n) {
          start_s = decode_place(e, begin - before, tiles);
          break;
        }
        before += n;
      }
    }
    __syncthreads();
  }
  Join* joins = static_cast<Join*>(p.workspace);
  if (!p.direct && threadIdx.x == 0) joins[blockIdx.x].last = -1;
  if (begin >= total) return;
  const long long end = min(total, begin + share);
  const int count = static_cast<int>(end - begin);

  // ---- the copies, ahead of the arithmetic ----
  const uint32_t ring = smem_u32(smem) + warp * L::kRing;
  DecodePlace load = start_s;
  int load_len = enter(p, load);
  const uint8_t *load_k, *load_v;  // the item's head in page 0
  const int* load_pages;           // the entry's line of the table
  int load_head;
  auto load_item = [&]() {
    load_head = item_of(p, load, kR, blocks_of_rows).head;
    load_k = p.c.k + wide(load_head, p.c.k_head);
    load_v = p.c.v + wide(load_head, p.c.v_head);
    load_pages = p.t.pages + load.entry * p.t.stride;
  };
  load_item();
  const int warp_row = warp * kRowsPerWarp;
  // The pages of the warp's rows in 32 tiles from `window`, one to a lane: loaded at an item's
  // start (and every 32 tiles) well before their use.  Checked where they are used.
  int window = 0, window_page = 0;
  auto load_window = [&]() {
    window = load.tile;
    const long long row = static_cast<long long>(load.tile + lane) * kDecodeTile + warp_row;
    window_page = row < load_len ? load_pages[row >> p.c.page_shift] : 0;
  };
  load_window();
  int loaded = 0;
  uint32_t stage_in = ring;  // of the next copy
  const int r0 = lane / L::kChunks, c0 = lane % L::kChunks;  // the lane's first chunk
  auto issue = [&]() {
    const int row = load.tile * kDecodeTile + warp_row;
    if (row < load_len) {
      const uint32_t stage = stage_in;
      const int place = row & (p.c.page_size - 1);
      int page = __shfl_sync(0xffffffffu, window_page, load.tile - window);
      int valid = min(kRowsPerWarp, load_len - row);
      if (static_cast<uint32_t>(page) >= p.c.num_pages) {
        atomicOr(p.t.error_word, kErrIndex);
        page = valid = 0;  // zeros in place of rows, and no address made of the page
      }
      const uint32_t pg = static_cast<uint32_t>(page);
      const uint8_t* k = load_k + wide(pg, p.c.k_page) + wide(place, p.c.k_token);
      const uint8_t* v = load_v + wide(pg, p.c.v_page) + wide(place, p.c.v_token);
      constexpr int kPer = kRowsPerWarp * L::kChunks / 32;  // chunks of K to a lane
      constexpr int kStep = 32 / L::kChunks;                // rows from one to the next
      if (valid == kRowsPerWarp) {
        const uint8_t* kl = k + wide(r0, p.c.k_token) + c0 * 16;
        const uint8_t* vl = v + wide(r0, p.c.v_token) + c0 * 16;
        if (p.c.k_token == L::kRow && p.c.v_token == L::kRow) {  // rows follow one another
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const uint32_t to = stage + chunk_at<L::kChunks>(r0 + i * kStep, c0);
            copy16(to, kl + i * 512);
            copy16(to + L::kStage / 2, vl + i * 512);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const uint32_t to = stage + chunk_at<L::kChunks>(r0 + i * kStep, c0);
            copy16(to, kl);
            copy16(to + L::kStage / 2, vl);
            kl += wide(kStep, p.c.k_token);
            vl += wide(kStep, p.c.v_token);
          }
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < kPer; ++i) {
          const int r = r0 + i * kStep;
          const uint32_t to = stage + chunk_at<L::kChunks>(r, c0);
          const uint32_t bytes = r < valid ? 16u : 0u;
          const int from = r < valid ? r : 0;
          copy16(to, k + wide(from, p.c.k_token) + c0 * 16, bytes);
          copy16(to + L::kStage / 2, v + wide(from, p.c.v_token) + c0 * 16, bytes);
        }
      }
      if constexpr (kE4M3) {
        if (lane < 2) {
          copy16(stage + L::kStage + lane * 16,
                 (lane == 0 ? p.c.k_scale : p.c.v_scale) +
                     scale_offset(p.c, pg, load_head, place),
                 valid ? 16u : 0u);
        }
      }
    }
    stage_in += L::kStage + L::kScales;
    if (stage_in == ring + L::kRing) stage_in = ring;
    if (++loaded < count) {
      const bool entry = decode_advance(load, copies);
      if (load.tile == 0) {
        if (entry) load_len = enter(p, load);
        load_item();
        load_window();
      } else if (load.tile == window + 32) {
        load_window();
      }
    }
  };
#pragma unroll 1
  for (int i = 0; i < L::kStages - 1; ++i) {
    if (loaded < count) issue();
    copy_commit();
  }

  // ---- the arithmetic ----
  DecodePlace cur = start_s;
  int cur_len = enter(p, cur);
  long long first_tile = begin - cur.tile;  // of the current item
  uint32_t stage_out = ring;
  uint32_t qf[D / 16][kNT][2];
  float factor[kNT][2];            // of the scores, by column
  float o[D / 16][kNT][4];
  // the references r and r' (0 while there is none), what raises them (-inf), and the sums
  float ref[kNT][2], ref_v[kNT][2], top[kNT][2], top_v[kNT][2], sum[kNT][2];
  bool fresh = true;
  bool low = false;  // the queries have a part below fp16's range
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    // With a stage to spare the next copies are issued behind the first MMAs, whose results take a
    // while (1 to 3 % of the time); two stages need them at once.
    constexpr bool kLate = L::kStages >= 3;
    if constexpr (!kLate) {
      if (loaded < count) issue();
      copy_commit();
    }
    if (fresh) {
      fresh = false;
      low = false;
      const Item it = item_of(p, cur, kR, blocks_of_rows);
      const int row0 = it.row0;
      const uint8_t* q0 = p.q + wide(it.seq, p.q_batch) + wide(it.head * p.group + row0, p.q_head);
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const bool in = row0 + n * 8 + g < p.group;
        const uint32_t* q =
            reinterpret_cast<const uint32_t*>(q0 + wide(n * 8 + (in ? g : 0), p.q_head));
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          // the columns of K that this lane's fragment multiplies: 2t, 2t + 1 and 2t + 8, 2t + 9
          // of each 16, or for e4m3 (four codes to a word) 4t .. 4t + 3
          qf[s][n][0] = in ? __ldg(q + s * 8 + (kE4M3 ? 2 * t : t)) : 0u;
          qf[s][n][1] = in ? __ldg(q + s * 8 + (kE4M3 ? 2 * t + 1 : t + 4)) : 0u;
        }
        if constexpr (kE4M3) {
          // magnitudes compare as integers, two at a time: the largest, and the least but zero, - 1
          uint32_t most = 0, least = 0xFFFFFFFFu;
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t m = qf[s][n][j] & 0x7FFF7FFFu;
              most = __vmaxu2(most, m);
              if constexpr (kBf16) least = __vminu2(least, __vsub2(m, 0x00010001u));
            }
          most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 2));
          most = __float_as_uint(unpack16<kBf16>(max(most >> 16, most & 0xFFFFu)).x);
          // The largest magnitude into [2^15, 2^16): fp16 queries stay exact, and a bf16 element
          // keeps all its bits down to 2^-32 of the largest; what is below goes by a second pass
          // over the keys (`low`).  (255: an infinity, beside which all others stay finite.)
          const uint32_t e = most > 0 ? min(max(most >> 23, 16u), 254u) : 142u;
          if constexpr (kBf16)
            low |= ((min(least >> 16, least & 0xFFFFu) + 1u) >> 7) + 32u < e;
          const float down = __uint_as_float((269u - e) << 23);
          if (t == 0) down_s[warp][n * 8 + g] = down;
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 f = unpack16<kBf16>(qf[s][n][j]);
              qf[s][n][j] = pack16<false>(f.x * down, f.y * down);
            }
          const float up = __uint_as_float((e - 15u) << 23) * p.scale_log2;
          factor[n][0] = __shfl_sync(0xffffffffu, up, 8 * t);
          factor[n][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4);
        } else {
          factor[n][0] = factor[n][1] = p.scale_log2;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          ref[n][j] = ref_v[n][j] = sum[n][j] = 0.f;
          top[n][j] = top_v[n][j] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[c][n][j] = 0.f;
      }
      if constexpr (kE4M3 && kBf16) low = __any_sync(0xffffffffu, low);
    }
    copy_wait<kLate ? L::kStages - 2 : L::kStages - 1>();
    __syncwarp();
    const int row = cur.tile * kDecodeTile + warp_row;
    const uint32_t used = stage_out - ring;  // the same in every warp
    bool issued = !kLate;
    if (row < cur_len) {
      const uint32_t stage = stage_out;
      const int mat = lane / 8, mr = lane % 8;
      // S = K Q^T
      float sc[L::kChains][kNT][4];
#pragma unroll
      for (int c = 0; c < L::kChains; ++c)
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[c][n][j] = 0.f;
      if constexpr (kE4M3 && kBf16) {
        if (low) {  // (hardly ever: the low parts of q, made again from q)
          const Item it = item_of(p, cur, kR, blocks_of_rows);
          const uint8_t* q0 =
              p.q + wide(it.seq, p.q_batch) + wide(it.head * p.group + it.row0, p.q_head);
          const int r = mr + (mat & 1) * 8;
#pragma unroll 1
          for (int s = 0; s < L::kChunks / 2; ++s) {
            uint32_t a[4];
            ldsm4(a, stage + chunk_at<L::kChunks>(r, 2 * s + (mat >> 1)));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t f[4];
              e4m3x4_to_f16(a[2 * x], f[0], f[2]);
              e4m3x4_to_f16(a[2 * x + 1], f[1], f[3]);
#pragma unroll
              for (int n = 0; n < kNT; ++n) {
                const bool in = it.row0 + n * 8 + g < p.group;
                const uint32_t* q =
                    reinterpret_cast<const uint32_t*>(q0 + wide(n * 8 + (in ? g : 0), p.q_head)) +
                    (2 * s + x) * 8 + 2 * t;
                const float down = down_s[warp][n * 8 + g];
                mma<false>(sc[0][n], f, low_part(in ? __ldg(q) : 0u, down),
                           low_part(in ? __ldg(q + 1) : 0u, down));
              }
            }
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[0][n][j] *= 1.f / kLowScale;
        }
      }
      {
        const int r = mr + (mat & 1) * 8;
#pragma unroll
        for (int s = 0; s < L::kChunks / 2; ++s) {
          uint32_t a[4];
          ldsm4(a, stage + chunk_at<L::kChunks>(r, 2 * s + (mat >> 1)));
          if constexpr (!kE4M3) {
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              mma<kMmaBf16>(sc[s % L::kChains][n], a, qf[s][n][0], qf[s][n][1]);
          } else {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t f[4];
              e4m3x4_to_f16(a[2 * x], f[0], f[2]);
              e4m3x4_to_f16(a[2 * x + 1], f[1], f[3]);
#pragma unroll
              for (int n = 0; n < kNT; ++n)
                mma<false>(sc[(2 * s + x) % L::kChains][n], f, qf[2 * s + x][n][0],
                           qf[2 * s + x][n][1]);
            }
          }
        }
      }
      if constexpr (kLate) {
        if (loaded < count) issue();
        copy_commit();
        issued = true;
      }
      float ks[2] = {1.f, 1.f}, vs[2] = {0.f, 0.f};
      if constexpr (kE4M3) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t at = stage + L::kStage + g + 8 * j;
          uint32_t ke, ve;
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(ke) : "r"(at) : "memory");
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(ve) : "r"(at + 16) : "memory");
          ks[j] = scale_value(ke);
          vs[j] = ve == 255u ? __uint_as_float(0x7FFFFFFFu) : static_cast<float>(ve) - 127.f;
        }
      }
      float z[kNT][4], zv[kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int rr = j >> 1, cc = j & 1;
          float s = sc[0][n][j];
          if constexpr (L::kChains == 2) s += sc[1][n][j];
          if constexpr (L::kChains == 4) s = (s + sc[1][n][j]) + (sc[2][n][j] + sc[3][n][j]);
          z[n][j] = s * (kE4M3 ? ks[rr] * factor[n][cc] : factor[n][cc]);
          zv[n][j] = z[n][j] + vs[rr];
        }
      if (row + kRowsPerWarp > cur_len) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row + g + 8 * (j >> 1) >= cur_len) z[n][j] = zv[n][j] = -INFINITY;
      }
      bool raise = false;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          raise |= z[n][j] > top[n][j & 1];
          if constexpr (kE4M3) raise |= zv[n][j] > top_v[n][j & 1];
        }
      if (__any_sync(0xffffffffu, raise)) {
        if constexpr (kE4M3) {
          // A row of zeros in V adds nothing whatever its scale byte says (a written one says 1,
          // far above its neighbours'): it must not set r'.  Two lanes look at a row's codes.
          uint32_t held = 0;
#pragma unroll
          for (int c = 0; c < L::kChunks / 2; ++c) {
            uint32_t x[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"(stage + L::kStage / 2 +
                               chunk_at<L::kChunks>(lane >> 1, (lane & 1) * (L::kChunks / 2) + c))
                         : "memory");
            held |= x[0] | x[1] | x[2] | x[3];
          }
          held &= 0x7F7F7F7Fu;  // (-0 is zero)
          const uint32_t rows = __ballot_sync(0xffffffffu, held != 0);
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            const bool zero = (rows >> (2 * (g + 8 * rr)) & 3u) == 0;
            if (zero && vs[rr] == vs[rr]) {  // (scale byte 255: NaN, not zeros)
#pragma unroll
              for (int n = 0; n < kNT; ++n) zv[n][2 * rr] = zv[n][2 * rr + 1] = -INFINITY;
            }
          }
        }
        // r <- the maximum so far, less the shift; what was summed shrinks by 2^(r_old - r)
        auto raise_to = [&](float a, float b, float& r, float& limit, bool f16) {
          const float shift = f16 ? kShiftF16 : 0.f, pass = f16 ? kRaiseF16 : kRaise;
          float m = fmaxf(a, b);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
          const float old = limit == -INFINITY ? -INFINITY : r;
          m = fmaxf(m - shift, old);
          if (m == -INFINITY) return 1.f;
          r = m;
          limit = m + (shift + pass);
          return ex2_approx(old - m);
        };
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            float f = raise_to(z[n][cc], z[n][2 + cc], ref[n][cc], top[n][cc],
                               !kMmaBf16 && !kE4M3);
            sum[n][cc] *= f;
            if constexpr (kE4M3)
              f = raise_to(zv[n][cc], zv[n][2 + cc], ref_v[n][cc], top_v[n][cc], true);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              o[c][n][cc] *= f;
              o[c][n][2 + cc] *= f;
            }
          }
      }
      uint32_t hi[kNT][2], lo[kNT][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = ex2_approx(z[n][j] - ref[n][j & 1]);
          sum[n][j & 1] += e;
          w[j] = kE4M3 ? ex2_approx(zv[n][j] - ref_v[n][j & 1]) : e;
        }
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          // (e4m3 has no infinities: the nearest fp16, with a remainder of either sign)
          const uint32_t h = kE4M3 ? pack16<false>(w[2 * rr], w[2 * rr + 1])
                                   : pack_below<kMmaBf16>(w[2 * rr], w[2 * rr + 1]);
          const float2 back = unpack16<kMmaBf16>(h);
          hi[n][rr] = transpose8(h);
          lo[n][rr] = transpose8(pack16<kMmaBf16>(w[2 * rr] - back.x, w[2 * rr + 1] - back.y));
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int c = 0; c < L::kChunks / 2; ++c) {
        uint32_t a[4];
        if constexpr (!kE4M3) {
          const int r = mr + (mat >> 1) * 8;
          ldsm4_t(a, stage + L::kStage / 2 + chunk_at<L::kChunks>(r, 2 * c + (mat & 1)));
#pragma unroll
          for (int n = 0; n < kNT; ++n) mma<kMmaBf16>(o[c][n], a, hi[n][0], hi[n][1]);
#pragma unroll
          for (int n = 0; n < kNT; ++n) mma<kMmaBf16>(o[c][n], a, lo[n][0], lo[n][1]);
        } else {
          const int r = mr + (mat & 1) * 8;
          ldsm4_t(a, stage + L::kStage / 2 + chunk_at<L::kChunks>(r, 2 * c + (mat >> 1)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // a word holds two adjacent columns of d at two adjacent positions: put the positions
            // of each column together; row i of the MMA tile is column 2 i, row i + 8 is 2 i + 1
            const uint32_t w0 = __byte_perm(a[2 * x], 0, 0x3120);
            const uint32_t w1 = __byte_perm(a[2 * x + 1], 0, 0x3120);
            uint32_t f[4];
            e4m3x4_to_f16(w0, f[0], f[1]);
            e4m3x4_to_f16(w1, f[2], f[3]);
#pragma unroll
            for (int n = 0; n < kNT; ++n) mma<false>(o[2 * c + x][n], f, hi[n][0], hi[n][1]);
#pragma unroll
            for (int n = 0; n < kNT; ++n) mma<false>(o[2 * c + x][n], f, lo[n][0], lo[n][1]);
          }
        }
      }
    }
    if (!issued) {
      if (loaded < count) issue();
      copy_commit();
    }
    __syncwarp();  // the stage may be filled again
    stage_out += L::kStage + L::kScales;
    if (stage_out == ring + L::kRing) stage_out = ring;

    const bool done = cur.tile == cur.tiles - 1;
    if (done || i == count - 1) {
      // ---- join the warps: each leaves O in the stage that it has just used ----
      const Item it = item_of(p, cur, kR, blocks_of_rows);
      const bool whole = done && first_tile >= begin;
      const int part = decode_part(first_tile, begin);
      float* ws_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kJoinBytes) +
                      (blockIdx.x * 2 + part) * kMaxRows;
      float* ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kJoinBytes +
                                             kLseBytes) +
                    static_cast<size_t>(blockIdx.x * 2 + part) * kMaxRows * D;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          float l = sum[n][cc];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
          const int col = 2 * t + cc;
          if (g == 0) {
            float* r = join_r + warp * kMaxRows + n * 8 + col;
            r[0] = top[n][cc] == -INFINITY ? -INFINITY : ref[n][cc];
            r[kWarps * kMaxRows] = !kE4M3                     ? r[0]
                                   : top_v[n][cc] == -INFINITY ? -INFINITY
                                                               : ref_v[n][cc];
            r[2 * kWarps * kMaxRows] = l;
          }
          float* dst = reinterpret_cast<float*>(smem + warp * L::kRing + used) + col * D;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {  // (the columns of four t go to different banks)
            dst[(16 * c + (kE4M3 ? 2 * g : g)) ^ (8 * t)] = o[c][n][cc];
            dst[(16 * c + (kE4M3 ? 2 * g + 1 : g + 8)) ^ (8 * t)] = o[c][n][2 + cc];
          }
        }
        __syncthreads();
        // two heads to a warp, D / 32 columns of both to a lane
        constexpr int kPer = D / 32;
#pragma unroll
        for (int i = 0; i < 8 / kWarps; ++i) {
          const int col = warp + i * kWarps;
          const int qr = it.row0 + n * 8 + col;  // query head within the group
          if (qr < p.group) {
            const float* r = join_r + n * 8 + col;
            float m = -INFINITY, mv = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              m = fmaxf(m, r[w * kMaxRows]);
              mv = fmaxf(mv, r[(kWarps + w) * kMaxRows]);
            }
            // (no r': all of V is zeros, and so is O)
            const float base = m == -INFINITY ? 0.f : m, base_v = mv == -INFINITY ? base : mv;
            float l = 0.f, acc[kPer] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              l += r[(2 * kWarps + w) * kMaxRows] * ex2_approx(r[w * kMaxRows] - base);
              const float f = ex2_approx(r[(kWarps + w) * kMaxRows] - base_v);
              const float* src = reinterpret_cast<const float*>(smem + w * L::kRing + used) +
                                 col * D + ((lane * kPer) ^ (8 * (col >> 1)));
              if constexpr (kPer == 4) {
                const float4 x = *reinterpret_cast<const float4*>(src);
                acc[0] = fmaf(x.x, f, acc[0]);
                acc[1] = fmaf(x.y, f, acc[1]);
                acc[2] = fmaf(x.z, f, acc[2]);
                acc[3] = fmaf(x.w, f, acc[3]);
              } else {
                const float2 x = *reinterpret_cast<const float2*>(src);
                acc[0] = fmaf(x.x, f, acc[0]);
                acc[1] = fmaf(x.y, f, acc[1]);
              }
            }
            const float scale = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int j = 0; j < kPer; ++j) acc[j] *= scale;
            if constexpr (kE4M3) {  // (2^(r' - r) / l could be a subnormal)
              const float f = exp2f(base_v - base);
#pragma unroll
              for (int j = 0; j < kPer; ++j) acc[j] *= f;
            }
            const float lse = l == 0.f ? -INFINITY : base + log2f(l);
            if (whole) {
              const long long at =
                  (static_cast<long long>(it.seq) * p.c.heads + it.head) * p.group + qr;
              uint32_t* out = reinterpret_cast<uint32_t*>(p.o) + (at * D + lane * kPer) / 2;
              if constexpr (kPer == 4)
                *reinterpret_cast<uint2*>(out) =
                    make_uint2(pack16<kBf16>(acc[0], acc[1]), pack16<kBf16>(acc[2], acc[3]));
              else
                *out = pack16<kBf16>(acc[0], acc[1]);
              if (lane == 0) p.lse[at] = lse * 0.69314718055994531f;
            } else {
              float* out = ws_o + (n * 8 + col) * D + lane * kPer;
              if constexpr (kPer == 4)
                *reinterpret_cast<float4*>(out) = make_float4(acc[0], acc[1], acc[2], acc[3]);
              else
                *reinterpret_cast<float2*>(out) = make_float2(acc[0], acc[1]);
              if (lane == 0) ws_lse[n * 8 + col] = lse;
            }
          }
        }
        __syncthreads();
      }
      if (!done && first_tile >= begin && threadIdx.x == 0) {
        Join j;
        j.entry = cur.entry;
        j.item = cur.item;
        j.last = static_cast<int>((first_tile + cur.tiles - 1) / share);
        j.part = part;
        joins[blockIdx.x] = j;
      }
      fresh = true;
      first_tile = begin + i + 1;
    }
    if (i + 1 < count && decode_advance(cur, copies)) cur_len = enter(p, cur);
  }
}

// The join of an item's parts: block (c, row) handles a row of the item that
// starts, unfinished, in block c of decode_kernel.  Groups of lanes (four
// columns each) take the parts in turn, a batch of loads at a time, with a
// running maximum: it is a chain of latencies, and each group's first part is
// loaded together with the note of what is to be joined.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads) join_kernel(const DecodeParams p, int rows_per_block) {
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes, kBatch = 8;
  __shared__ float4 acc_s[kGroups][kLanes];
  __shared__ float sum_s[kGroups], top_s[kGroups];
  const int c0 = blockIdx.x, r = blockIdx.y;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const float* ws_lse =
      reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.workspace) + kJoinBytes);
  const float4* ws_o = reinterpret_cast<const float4*>(static_cast<const uint8_t*>(p.workspace) +
                                                       kJoinBytes + kLseBytes);
  // the group's first part: of block c0 + group (for c0 itself it can be either of the two)
  const int ahead = min(c0 + group, static_cast<int>(gridDim.x) - 1) * 2 * kMaxRows + r;
  grid_dep_wait();
  const Join j = static_cast<const Join*>(p.workspace)[c0];
  float lse0 = ws_lse[ahead];
  float4 o0 = ws_o[static_cast<size_t>(ahead) * kLanes + lane];
  if (group == 0) {
    const float other = ws_lse[ahead + kMaxRows];
    const float4 other_o = ws_o[static_cast<size_t>(ahead + kMaxRows) * kLanes + lane];
    if (j.part) lse0 = other, o0 = other_o;
  }
  if (j.last < 0) return;
  const int blocks_of_rows = (p.group + rows_per_block - 1) / rows_per_block;
  const int seq = p.per_head ? j.entry / p.c.heads : j.entry;
  const int h = j.item / blocks_of_rows;
  const int head = p.per_head ? j.entry - seq * p.c.heads : h;
  const int qr = (j.item - h * blocks_of_rows) * rows_per_block + r;
  if (qr >= p.group) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float lse, const float4& x, float base) {
    const float w = ex2_approx(lse - base);
    l += w;
    acc.x = fmaf(w, x.x, acc.x);
    acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z);
    acc.w = fmaf(w, x.w, acc.w);
  };
  auto raise = [&](float to) {  // what is summed so far, relative to the maximum `to` >= m
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - to);
    const bool none = m == -INFINITY && l == 0.f;  // (a NaN stays one)
    m = to;
    if (none) return;
    l *= f;
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
  };
  if (c0 + group <= j.last) {
    m = fmaxf(lse0, m);
    add(lse0, o0, m == -INFINITY ? 0.f : m);
  }
  for (int c = c0 + group + kGroups; c <= j.last; c += kGroups * kBatch) {
    float lse[kBatch];
    float4 x[kBatch];
    float top = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int at = min(c + i * kGroups, j.last) * 2 * kMaxRows + r;
      lse[i] = ws_lse[at];
      x[i] = ws_o[static_cast<size_t>(at) * kLanes + lane];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, lse[i]);
    raise(top);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c + i * kGroups <= j.last) add(lse[i], x[i], m == -INFINITY ? 0.f : m);
  }
  acc_s[group][lane] = acc;
  if (lane == 0) sum_s[group] = l, top_s[group] = m;
  __syncthreads();
  if (group == 0) {
    float top = m;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) top = fmaxf(top, top_s[i]);
    raise(top);
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
      if (c0 + i > j.last) break;
      const float4 x = acc_s[i][lane];
      const float f = ex2_approx(top_s[i] - (top == -INFINITY ? 0.f : top));
      l = fmaf(sum_s[i], f, l);
      acc.x = fmaf(x.x, f, acc.x);
      acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(x.z, f, acc.z);
      acc.w = fmaf(x.w, f, acc.w);
    }
    const long long at = (static_cast<long long>(seq) * p.c.heads + head) * p.group + qr;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    reinterpret_cast<uint2*>(p.o)[at * kLanes + lane] =
        make_uint2(pack16<kBf16>(acc.x * inv, acc.y * inv),
                   pack16<kBf16>(acc.z * inv, acc.w * inv));
    if (lane == 0)
      p.lse[at] = l == 0.f ? -INFINITY
                           : ((top == -INFINITY ? 0.f : top) + log2f(l)) * 0.69314718055994531f;
  }
}

// ---- host ----

// `early`: the launch may begin while the kernel before it in the stream ends.
// Only where that one is a kernel of this call: it waits for its own
// predecessors, and ours waits for it (grid_dep_wait) before it reads anything.
template <typename... A>
bool launch_kernel(void (*kernel)(A...), dim3 grid, unsigned threads, size_t smem,
                   cudaStream_t stream, bool early, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <int D, int kNT, bool kE4M3, bool kBf16>
int launch(const DecodeParams& p, int dev, cudaStream_t stream) {
  using L = Layout<D, kNT, kE4M3>;
  auto kernel = decode_kernel<D, kNT, kE4M3, kBf16>;
  static std::once_flag once[kMaxDevices];
  static int sms[kMaxDevices];
  std::call_once(once[dev], [&] {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem) ==
            cudaSuccess)
      sms[dev] = n;
  });
  if (sms[dev] < 1) return -4;
  const int copies = (p.per_head ? 1 : p.c.heads) * ((p.group + 8 * kNT - 1) / (8 * kNT));
  const long long positions = static_cast<long long>(p.t.width) << p.c.page_shift;
  const long long tiles = (positions + kDecodeTile - 1) / kDecodeTile;
  if (tiles <= kDirectTiles) {  // (the items are at most the query heads: below 2^31)
    DecodeParams one = p;
    one.direct = 1;
    const unsigned items = static_cast<unsigned>(copies) * static_cast<unsigned>(p.t.batch);
    return launch_kernel(kernel, dim3(items), kThreads, L::kSmem, stream, p.per_head != 0, one)
               ? 0
               : -4;
  }
  // as many blocks as are resident; fewer if the table cannot hold that many tiles
  long long grid = static_cast<long long>(L::kBlocks) * sms[dev];
  if (grid > kDecodeMaxBlocks) grid = kDecodeMaxBlocks;
  const long long most =
      (tiles * copies * p.t.batch + p.least_tiles - 1) / p.least_tiles;
  if (grid > most) grid = most;
  const unsigned blocks = static_cast<unsigned>(grid);
  if (!launch_kernel(kernel, dim3(blocks), kThreads, L::kSmem, stream, p.per_head != 0, p))
    return -4;
  const unsigned rows = static_cast<unsigned>(p.group < 8 * kNT ? p.group : 8 * kNT);
  if (!launch_kernel(join_kernel<D, kBf16>, dim3(blocks, rows), kThreads, 0, stream, true, p,
                     8 * kNT))
    return -4;
  return 0;
}

template <int D>
int dispatch(const DecodeParams& p, bool e4m3, bool bf16, int dev, cudaStream_t stream) {
  const bool wide = p.group > 8;
  if (e4m3) {
    if (bf16)
      return wide ? launch<D, 2, true, true>(p, dev, stream)
                  : launch<D, 1, true, true>(p, dev, stream);
    return wide ? launch<D, 2, true, false>(p, dev, stream)
                : launch<D, 1, true, false>(p, dev, stream);
  }
  if (bf16)
    return wide ? launch<D, 2, false, true>(p, dev, stream)
                : launch<D, 1, false, true>(p, dev, stream);
  return wide ? launch<D, 2, false, false>(p, dev, stream)
              : launch<D, 1, false, false>(p, dev, stream);
}

}  // namespace decode

}  // namespace fat
