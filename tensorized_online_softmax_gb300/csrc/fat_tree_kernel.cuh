// Attention of drafted tokens over the paged cache.
//
// What bounds it: the rows (drafted token, query head of the group) of a cached head
// share one pass over its keys and values.  Up to about 256 rows that is a stream
// through HBM (4 rows flops to 2 bytes of a 16-bit cache); the products take the
// tensor pipe a quarter (128 rows) to a half (256) of that time, so all else has to
// hide behind the copies.
//
// Work: an item is a block of up to 128 rows of one (sequence, cached head), or two such
// blocks where a 16-bit cache has more; its positions are walked in tiles of 128
// (tree_span: with a window only those that a row may see).  The tiles of all items form
// one line, of which every thread block takes an equal share (fat_decode_plan.h); items
// that blocks share leave normalised parts in the workspace for the join kernel, in a
// fixed order.
//
//   softmax     two groups of warps.  Of two blocks of rows each group takes one, at every
//               tile; of one block both have the same rows and take alternate tiles, with
//               an O and statistics of their own that are joined at the item's end: no group
//               waits for the other inside an item.  For 16-bit caches a row has two threads,
//               64 scores each, that share its reference (they vote at every tile whether it
//               has to be raised).
//   MMA issuer  S_g = Q_g K^T (tcgen05, 128 x 128), O_g += P_g V.
//   producers   of K and V (a warp each) and of Q, ahead of the items: TMA boxes, one for each
//               page of a tile.
//   converters  (e4m3 caches) the producers bring codes and scale bytes to a ring of their own;
//               these warps make 16-bit rows of them in the rings of K and V.  The softmax
//               warps copy Q.
//
// TMEM: S_0, S_1 (P_g over S_g), O_0, O_1: 512 columns.  So the scores of a group's next tile
// wait for this one's O += P V, and a group's step is a chain: product, maximum, weights,
// product.
//
// Per score: z = scale log2(e) s - r with a running reference r for each row, raised to
// the row's maximum only where a tile exceeds it by more than kRaise binades (then O is
// rescaled in TMEM: a rare event).  The scores are read twice from TMEM, for the
// maximum and for the weights: it has the bandwidth.  P is rounded to 16 bits, the sum of
// the row is not.  (A second 16-bit term of the weights, as the single-token kernel has it,
// lengthens the chain and takes half as many MMAs again: the 16 sequences below 62 us a call
// instead of 56, the 256 rows 119 instead of 94; and as its terms have either sign, infinite
// values would become NaN.  Errors against 64 bits are 0.0023 of the results' size over bf16
// caches, of which the output's own rounding makes 0.0017, and 0.00024 of 0.00020 over fp16.)
//
// e4m3 caches: a code times its row's power of two is an fp16 wherever the scale is
// within 2^-15 .. 2^7, and a bf16 wherever the product is from 2^-133 to below 2^128 (codes
// from 2^-9 to 448 and scales from 2^-126 to 2^127 leave that at both ends: what is below
// is lost, what is above infinite).  Rows become fp16 (one conversion and one
// multiplication to two codes); the tiles of V with a scale outside that range bf16, and
// the weights of such a tile two bf16 terms.  bf16 queries become fp16 times a power of two
// for the item; where that would lose bits (elements more than 31 binades apart), they stay
// bf16 and so do the item's keys.  Keys with a scale outside the range stay codes, and the
// scale multiplies their scores.  So nothing is lost in any of them within that range.
//
// Headroom: O is summed with weights of up to 2^8 (bf16 caches) or 2^15 (2^kShift at the
// reference, kRaise binades above it) before the row's sum divides it.  So values times
// the positions that a row sees (as far as their weights come near its largest) have to
// stay below 2^120 or 2^113, else O overflows where the result would not.
//
// Measured (GB300, device time; the rate is of the bytes that have to be read, beside 6783
// GB/s of a plain copy), d = 128 and 8 cached heads but for the last:
//   16 sequences of 1000 to 8192, 64 rows a head, bf16          54 us   4.7 TB/s
//   8 of 4096 to 16384, 256 rows, bf16                          88 us   4.0 TB/s
//   32 of 4096 to 16384, 64 rows, e4m3                         208 us   3.6 TB/s
//   1 of 208, 32 rows, bf16                                    8.7 us
//   13 of 5 to 4097 under a window of 1024, 20 heads of 5 rows, d = 64, fp16   30 us  2.0 TB/s
// 64 rows over a 16-bit cache stream at the copy rate (2.8 k clocks a tile) between a start
// of 4 us (the plan, the first pages and tiles) and an end of 4; 256 rows are bound by the
// chain of a group (3.7 k clocks a tile of 2.8 k), e4m3 by it and by the issue of the
// conversions (2.6 k of 1.4 k; issue slots 57 %).  Instructions that run once in a while are
// fetched as they run, about ten clocks each: hence small loops and little code.
//
// What no row sees is zeroed in V's tile, and never fetched where it fills a page; what
// only some rows see (drafted tokens, a window's border) has its non-finite values
// zeroed and noted, and added again at the end for the rows that see it: 0 times NaN
// would be NaN in rows that do not.
#pragma once

#include <cuda.h>

#include "fat_tree.cuh"
#include "sm103_ptx.cuh"

namespace fat {

namespace tree {

// what a kernel is made for: a 16-bit cache's type, or an e4m3 cache and the queries' type
constexpr int kBf16 = 0, kF16 = 1, kE4M3Bf16 = 2, kE4M3F16 = 3;

template <int kType>
constexpr bool kIsE4M3 = kType >= kE4M3Bf16;
// softmax warps, then the MMA issuer, the producers of K, V and Q (e4m3: one for K and V, the
// softmax warps load Q), then the converters
template <int kType>
constexpr int kHalves = kIsE4M3<kType> ? 1 : 2;  // threads to a row
template <int kType>
constexpr int kSoftWarps = 8 * kHalves<kType>;
constexpr int kConvertWarps = 16;  // two teams of four for K and four for V
// Registers (e4m3): 896 threads start with 72 each; the softmax warps take what the others leave.
constexpr int kLaunchRegs = 72, kSoftRegs = 136, kControlRegs = 72, kConvertRegs = 40;
static_assert(256 * kSoftRegs + 128 * kControlRegs + 32 * kConvertWarps * kConvertRegs <=
                  (384 + 32 * kConvertWarps) * kLaunchRegs,
              "what is taken has been given");
template <int kType>
constexpr int kThreadsOf =
    32 * (kSoftWarps<kType> + 4 + (kIsE4M3<kType> ? kConvertWarps : 0));
constexpr uint32_t kTmemCols = 512;
// binades above the maximum at the last raise that are let pass; fp16 weights are
// 2^kShift at that maximum (2^15 is the most fp16 holds)
template <int kType>
constexpr float kRaise = kType == kBf16 ? 8.f : 4.f;
template <int kType>
constexpr float kShift = kType == kBf16 ? 0.f : 11.f;
// scale bytes whose rows of codes are exact in fp16: 2^-9 2^-15 is its least step, 448 2^7 < 2^16
constexpr uint32_t kScaleLow = 112, kScaleHigh = 134;

struct Join {  // what the join kernel needs of the item that starts, unfinished, in a block
  int entry, item;
  int last;  // the last block with a part of it; -1: nothing to join
  int part;  // where the first block keeps its part
};
constexpr size_t kJoinBytes = sizeof(Join) * kTreeMaxBlocks;
// then, for each block and part, `rows` LSEs (log2), and after all of those the rows: four
// columns of all rows, then the next four, as threads hold one row each
__host__ __device__ inline size_t lse_at(int block, int part, int rows) {
  return kJoinBytes + sizeof(float) * (static_cast<size_t>(block) * 2 + part) * rows;
}
__host__ __device__ inline size_t rows_at(int block, int part, int rows, int d) {
  return kJoinBytes + sizeof(float) * (static_cast<size_t>(kTreeMaxBlocks) * 2 * rows +
                                       (static_cast<size_t>(block) * 2 + part) * rows * d);
}

struct KernelParams {
  CUtensorMap tm_k, tm_v, tm_q;
  TreeParams p;
  // 0 where all heads, pages or sequences are the same memory (a stride of 0)
  int k_head, k_page, v_head, v_page, q_batch;
};

template <int D, int kType, int kNB>
struct Layout {
  static constexpr bool kE4M3 = kType >= kE4M3Bf16;
  static constexpr int kTile = kTreeTile * D * 2;
  // buffers of Q, stages of K and V, and of an e4m3 cache's codes: what the shared memory has
  // room for
  static constexpr int kQBufs = !kE4M3 && (kNB == 1 || D == 64) ? 2 : 1;
  static constexpr int kQBars = kE4M3 ? kTreeQueryBars : kQBufs;
  static constexpr int kKStages = kE4M3 || D == 128 ? 2 : kNB == 1 ? 5 : 4;
  static constexpr int kStages = kE4M3 ? 2 : D == 128 ? 3 : kNB == 1 ? 6 : 5;
  static constexpr int kRawStages = !kE4M3 ? 0 : D == 64 ? 12 : 4;
  static constexpr int kRawTile = kTreeTile * D;  // codes
  static constexpr int kAtoms = D / 64;  // slabs of 64 columns (128 bytes)
  static constexpr int kQ = 0;
  static constexpr int kK = kQBufs * kNB * kTile;
  static constexpr int kV = kK + kKStages * kTile;
  static constexpr int kRaw = kV + kStages * kTile;
  static constexpr int kScales = kRaw + kRawStages * kRawTile;  // of the codes' rows
  // u32 [kRawStages][2]: what the converters have to know of a tile: its rows that are seen, [0, a)
  // and [b, c), a byte each; and the items so far, its own counted, or 0 behind the last tile
  static constexpr int kInfo = kScales + kRawStages * kTreeTile;
  static constexpr int kBars = kInfo + kRawStages * 8;
  static constexpr int bKFull = 0;
  static constexpr int bKEmpty = bKFull + kKStages;
  static constexpr int bVFull = bKEmpty + kKStages;
  static constexpr int bVEmpty = bVFull + kStages;
  static constexpr int bRawFull = bVEmpty + kStages;
  static constexpr int bRawEmpty = bRawFull + kRawStages;
  static constexpr int bSFull = bRawEmpty + kRawStages;  // [2]
  static constexpr int bPFull = bSFull + 2;              // [2], the group's warps
  static constexpr int bPV = bPFull + 2;                 // [2]
  static constexpr int bQFull = bPV + 2;                 // [kQBars]; e4m3: the softmax warps
  static constexpr int bQFree = bQFull + kQBars;         // [kQBufs]
  static constexpr int bSync = bQFree + kQBufs;          // all softmax warps are here
  static constexpr int bVType = bSync + 1;               // [4] (e4m3) a tile's type of V is known
  static constexpr int bDrain = bVType + (kE4M3 ? 4 : 0);
  static constexpr int kNumBars = bDrain + 1;
  static __device__ __forceinline__ int arrivals(int bar) {
    if (kE4M3 && ((bar >= bKFull && bar < bKEmpty) || (bar >= bVFull && bar < bVEmpty) ||
                  (bar >= bRawEmpty && bar < bSFull)))
      return kConvertWarps / 4;
    if (bar == bPFull || bar == bPFull + 1) return kSoftWarps<kType> / 2;
    if (bar == bSync || (kE4M3 && bar >= bQFull && bar < bQFree)) return kSoftWarps<kType>;
    return 1;
  }
  static constexpr int kMisc = kBars + ((8 * kNumBars + 15) & ~15);
  // u32: 0 TMEM base, 1 abort flag; (e4m3) 2 whether the item's queries and keys are bf16, 4 of
  // the last four tiles whether their values are, 8 the exponents of the item's queries, 20 of the
  // last four tiles whether their keys are codes; u64 bad[2 parities][2] at 12
  static constexpr int kBad = kMisc + 48;
  // float: the references [2 groups][128] and the sums [2][128] of the rows; the threads of a row
  // exchange their maxima in the latter.  During the set-up the plan's sums are there.
  static constexpr int kFin = kMisc + 96;
  // where the block's share starts: every role reads it when it gets there, so nothing else is ever
  // put in its place
  static constexpr int kStart = kFin + 2 * 2 * kTreeBlockRows * 4;
  static constexpr int kBytes = kStart + static_cast<int>(sizeof(DecodePlace));
  static_assert(kRawStages % 4 == 0, "K's and V's codes of two teams in turn");
  static_assert(!kE4M3 || kNB == 1, "one block of rows where the codes need room");
  static_assert(kK % 1024 == 0 && kV % 1024 == 0 && kRaw % 1024 == 0, "tiles on 1 KB");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// A block's walk along its share: the place, and what of the sequence each role needs.
struct Walk {
  DecodePlace at;
  TreeLens n;
  DecodeSpan span;
  int lo;  // the first position that any row sees behind the sinks
  int hi;  // from here on every row sees the context
  __device__ __forceinline__ int context() const { return n.len - n.drafted; }
  __device__ __forceinline__ int row() const { return decode_span_tile(span, at.tile) * kTreeTile; }
  // Nothing was drafted for the sequence: its rows are written, and nothing else is done.
  __device__ __forceinline__ bool empty() const { return n.drafted == 0; }
};
__device__ __forceinline__ void enter(const TreeParams& p, Walk& w) {
  w.n = tree_lens(p, w.at.entry);
  w.span = tree_span(p, w.n);
  w.at.tiles = w.span.tiles;
  w.lo = w.hi = 0;
  if (p.window > 0) {  // (by a whole warp)
    const int lane = threadIdx.x % 32;
    int lo = 0x7fffffff;
    for (int t = lane; t < w.n.drafted; t += 32) lo = min(lo, tree_row(p, w.n, w.at.entry, t).lo);
    w.lo = __reduce_min_sync(0xffffffffu, lo);
    w.hi = max(0, w.n.len - p.window);
  }
}
// Whether any row sees any position of [a, b).
__device__ __forceinline__ bool some_seen(const TreeParams& p, const Walk& w, int a, int b) {
  return !w.empty() && a < w.n.len && (p.window <= 0 || a < p.sinks || b > w.lo);
}
// Whether all (live) rows see all positions of [a, b).
__device__ __forceinline__ bool all_seen(const TreeParams& p, const Walk& w, int a, int b) {
  return b <= w.context() && (p.window <= 0 || b <= p.sinks || a >= w.hi);
}

// An item's rows: the cached head, and the first token and head of the group.
struct Rows {
  int head, t0, h0;
};
__device__ __forceinline__ Rows rows_of(const TreeParams& p, int item, int blocks) {
  Rows r;
  r.head = item / (p.token_items * p.head_items);
  const int x = item - r.head * p.token_items * p.head_items;
  const int th = x / p.head_items;
  r.t0 = th * p.block_tokens * blocks;
  r.h0 = (x - th * p.head_items) * p.block_heads;
  return r;
}

// Waits for a phase of a barrier, up to p.timeout_ns; false, with the abort flag set, if it does
// not come.  Most of a block's warps wait at any time: suspended, so that their polls take no
// issue slots.  (A test for limits too short for that, and polls that do not suspend, would cost 1 %
// of the call.)
__device__ __forceinline__ bool wait_suspended(uint32_t bar, uint32_t parity, const TreeParams& p,
                                               volatile uint32_t* abort_flag) {
  if (mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_for(bar, parity, p.suspend_ns)) {
    if (*abort_flag || globaltimer_ns() - t0 > p.timeout_ns) {
      atomicOr(p.error_word, 1u);
      *abort_flag = 1u;
      return false;
    }
  }
  return true;
}

// bits 0 .. n - 1
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Bits 15 and 31 say which of two 16-bit values are not finite: their exponents overflow.
template <bool kFp16>
__device__ __forceinline__ uint32_t not_finite(uint32_t two) {
  constexpr uint32_t kExp = kFp16 ? 0x7C007C00u : 0x7F807F80u;
  return (two & kExp) + (kFp16 ? 0x04000400u : 0x00800080u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 bytes to shared memory, of which the last 16 - `bytes` are zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

// element c of the row of V at position j; what is out of range reads as 0 (the sequence's
// results are unspecified then)
template <int kType>
__device__ __forceinline__ float value_at(const TreeParams& p, int b, uint32_t head, int j, int c) {
  const int page = table_page(p.t, p.c.num_pages, b, j >> p.c.page_shift);
  if (page < 0) return 0.f;
  const uint32_t at = j & (p.c.page_size - 1);
  const uint8_t* row = p.c.v + row_offset(page, head, at, p.c.v_page, p.c.v_head, p.c.v_token);
  if constexpr (kIsE4M3<kType>) {
    uint32_t lo, hi;
    e4m3x4_to_f16(row[c], lo, hi);
    return unpack16<false>(lo).x * scale_value(p.c.v_scale[scale_offset(p.c, page, head, at)]);
  }
  return unpack16<kType == kBf16>(reinterpret_cast<const uint16_t*>(row)[c]).x;
}

// Adds the non-finite values of the positions base + (bits of `left`) to columns col0 .. of a
// row that this thread has just written: 16-bit values at `out`, or, where that is null, fp32
// in the workspace.  (Hardly ever called.)
template <int kType, bool kOutBf16>
__device__ __noinline__ void add_not_finite(const TreeParams& p, int b, uint32_t head, int base,
                                            unsigned long long left, int col0, int cols,
                                            uint16_t* out, float* part) {
  for (; left; left &= left - 1) {
    const int j = base + __ffsll(static_cast<long long>(left)) - 1;
    for (int c = col0; c < col0 + cols; ++c) {
      const float v = value_at<kType>(p, b, head, j, c);
      if (fabsf(v) < INFINITY) continue;
      if (out)
        out[c] = static_cast<uint16_t>(pack16<kOutBf16>(unpack16<kOutBf16>(out[c]).x + v, 0.f));
      else
        part[static_cast<size_t>(c / 4) * p.item_rows * 4 + c % 4] += v;
    }
  }
}

template <int D, int kType, int kNB>
__global__ void __launch_bounds__(kThreadsOf<kType>, 1)
    tree_kernel(const __grid_constant__ KernelParams kp) {
  using L = Layout<D, kType, kNB>;
  constexpr int kThreads = kThreadsOf<kType>, kWarps = kThreads / 32;
  constexpr bool kE4M3 = L::kE4M3, kFp16 = kType != kBf16;
  constexpr bool kOutBf16 = kType == kBf16 || kType == kE4M3Bf16;
  constexpr int kH = kHalves<kType>, kSoft = kSoftWarps<kType>;
  constexpr int kMmaWarp = kSoft, kKWarp = kSoft + 1, kVWarp = kSoft + 2, kQWarp = kSoft + 3,
                kConvertWarp = kSoft + 4;
  constexpr int SK = L::kKStages, SV = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const TreeParams& p = kp.p;
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc + 1;
  // what some rows see and is not finite: drafted tokens and border positions, by item parity
  unsigned long long* bad_s = reinterpret_cast<unsigned long long*>(smem + L::kBad);
  float* fin = reinterpret_cast<float*>(smem + L::kFin);
  DecodePlace* start_s = reinterpret_cast<DecodePlace*>(smem + L::kStart);
  auto bar = [&](int i) -> uint32_t { return sb + L::kBars + 8 * i; };
  auto wait = [&](int i, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_suspended(bar(i), parity, p, abort_flag));
  };

  grid_dep_launch();
  if (sb % 1024 != 0) {  // (the swizzled tiles are laid out by address; it always is)
    if (threadIdx.x == 0) atomicOr(p.error_word, 1u);
    return;
  }

  // ---- set-up, and the block's share of the line of tiles ----
  if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < L::kNumBars; ++i) mbar_init(bar(i), L::arrivals(i));
      misc[1] = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(sb + L::kMisc, kTmemCols);
    tmem_relinquish();
  } else if (warp == kKWarp && lane == 0) {
    tma_prefetch_desc(&kp.tm_k);
    tma_prefetch_desc(&kp.tm_v);
    if (!kE4M3) tma_prefetch_desc(&kp.tm_q);
  }
  const int copies = p.c.heads * p.token_items * p.head_items;
  long long begin = 0, share = 1;  // units of the line
  int count;                       // tiles of this block
  int unit = 0;                    // where its first item starts, relative to `begin`
  if (p.direct) {
    const int e = blockIdx.x / copies;
    if (threadIdx.x == 0) *start_s = {e, static_cast<int>(blockIdx.x) - e * copies, 0, 0};
    count = tree_span(p, tree_lens(p, e)).tiles;
  } else {
    long long* sums = reinterpret_cast<long long*>(fin);  // [warps][units, tiles]
    long long* ends = sums + 2 * kWarps;  // tiles up to begin, and to end
    static_assert((2 * kWarps + 3) * 8 <= L::kStart - L::kFin, "the plan's sums");
    const int each = (p.t.batch + kThreads - 1) / kThreads;
    const int lo = min(p.t.batch, static_cast<int>(threadIdx.x) * each);
    const int hi = min(p.t.batch, lo + each);
    long long units = 0, tiles = 0;
    for (int e = lo; e < hi; ++e) {
      const TreeLens n = tree_lens(p, e);
      const int t = tree_span(p, n).tiles;
      tiles += t;
      units += t + tree_cost(p, n);
    }
    long long units_upto = units, tiles_upto = tiles;  // inclusive sums over the threads
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, units_upto, s);
      const long long y = __shfl_up_sync(0xffffffffu, tiles_upto, s);
      if (lane >= s) units_upto += x, tiles_upto += y;
    }
    if (lane == 31) sums[2 * warp] = units_upto, sums[2 * warp + 1] = tiles_upto;
    __syncthreads();
    static_assert(kWarps <= 32, "a lane to a warp's sums");
    long long total = lane < kWarps ? sums[2 * lane] : 0;
    long long all_tiles = lane < kWarps ? sums[2 * lane + 1] : 0;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, total, s);
      const long long y = __shfl_up_sync(0xffffffffu, all_tiles, s);
      if (lane >= s) total += x, all_tiles += y;
    }
    const long long units_ahead = __shfl_sync(0xffffffffu, total, warp - 1);
    const long long tiles_ahead = __shfl_sync(0xffffffffu, all_tiles, warp - 1);
    if (warp > 0) units_upto += units_ahead, tiles_upto += tiles_ahead;
    total = __shfl_sync(0xffffffffu, total, 31) * copies;
    all_tiles = __shfl_sync(0xffffffffu, all_tiles, 31) * copies;
    share = total <= 0x7fffffff - kTreeMaxBlocks
                ? decode_share(static_cast<int>(total), gridDim.x, 1)
                : decode_share(total, static_cast<int>(gridDim.x), 1);
    begin = blockIdx.x * share;
    const long long end = begin + share;
    long long unit0 = (units_upto - units) * copies, tile0 = (tiles_upto - tiles) * copies;
    if (threadIdx.x == 0) {
      ends[0] = ends[1] = all_tiles;
      ends[2] = 0;
    }
    __syncthreads();
    if (begin < units_upto * copies && end >= unit0) {
      for (int e = lo; e < hi; ++e) {
        const TreeLens n = tree_lens(p, e);
        const int t = tree_span(p, n).tiles, cost = tree_cost(p, n);
        const long long u = static_cast<long long>(t + cost) * copies;
        // the tile that a place on the line, in this entry, is the first before or at
        auto place = [&](long long at, DecodePlace& d, int& off) {
          d = decode_place(e, at - unit0, t + cost);
          off = d.tile;
          d.tile = max(0, d.tile - cost);
          d.tiles = t;
          return tile0 + static_cast<long long>(d.item) * t + d.tile;
        };
        DecodePlace d;
        int off;
        if (begin >= unit0 && begin < unit0 + u) {
          ends[0] = place(begin, d, off);
          ends[2] = off;
          *start_s = d;
        }
        if (end >= unit0 && end < unit0 + u) ends[1] = place(end, d, off);
        unit0 += u;
        tile0 += static_cast<long long>(t) * copies;
      }
    }
    __syncthreads();
    count = static_cast<int>(ends[1] - ends[0]);  // (0: more blocks than tiles)
    unit = -static_cast<int>(ends[2]);
    if (threadIdx.x == 0) reinterpret_cast<Join*>(p.workspace)[blockIdx.x].last = -1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  Walk w;
  const bool works = count > 0 && (warp <= kVWarp || (warp == kQWarp && !kE4M3) ||
                                   (kE4M3 && warp >= kConvertWarp));
  if (works && warp < kConvertWarp) {
    w.at = *start_s;
    enter(p, w);
  }

  // (Each kind of warp to its very end: no code is shared between register budgets.)
  auto finish = [&]() {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  if (warp >= kSoft && warp < kConvertWarp) {
    if constexpr (kE4M3) regs_dec<kControlRegs>();
    if (!works) {
    } else if (warp == kKWarp || warp == kVWarp) {
      // =================== producers of K and V ===================
      // (e4m3: into a common ring of codes, in turn)
      const bool is_k = warp == kKWarp;
      constexpr int kStep = kE4M3 ? 2 : 1;
      const int S = kE4M3 ? L::kRawStages : is_k ? SK : SV;
      const int full = kE4M3 ? L::bRawFull : is_k ? L::bKFull : L::bVFull;
      const int empty = kE4M3 ? L::bRawEmpty : is_k ? L::bKEmpty : L::bVEmpty;
      const uint32_t ring = sb + (kE4M3 ? L::kRaw : is_k ? L::kK : L::kV);
      const CUtensorMap* tm = is_k ? &kp.tm_k : &kp.tm_v;
      const int slot0 = kE4M3 && !is_k ? 1 : 0;
      const int rows = min(p.c.page_size, kTreeTile);  // of a box
      const int boxes = kTreeTile / rows;              // to a tile, each of a page
      const uint32_t box_bytes = rows * (kE4M3 ? D : 128u);
      // Pages of 32 / boxes tiles from `window`, one box to a lane, loaded well before their use.
      const int per = 32 / boxes;
      int window = 0, window_page = 0;
      auto load_window = [&]() {
        window = w.at.tile;
        const int tile = window + lane / boxes;
        const int a = decode_span_tile(w.span, tile) * kTreeTile + lane % boxes * rows;
        window_page = tile < w.at.tiles && some_seen(p, w, a, a + rows)
                          ? p.t.pages[w.at.entry * p.t.stride + (a >> p.c.page_shift)]
                          : 0;
      };
      load_window();
      int slot = slot0;
      uint32_t phase = 0;
      bool ok = true;
      int issued = 0;
      uint32_t items = 0;
      auto next_slot = [&]() {
        ++issued;
        if ((slot += kStep) >= S) slot = slot0, phase ^= 1u;
      };
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        if (!w.empty()) {
          if (i == 0 || w.at.tile == 0) ++items;
          const int head = w.at.item / (p.token_items * p.head_items);
          const int page = __shfl_sync(0xffffffffu, window_page,
                                       (w.at.tile - window) * boxes + lane % boxes);
          const int a = w.row() + lane % boxes * rows;
          bool mine = lane < boxes && some_seen(p, w, a, a + rows);
          if (mine && static_cast<uint32_t>(page) >= p.c.num_pages) {
            atomicOr(p.t.error_word, kErrIndex);
            mine = false;  // no address is made of it
          }
          const uint32_t n = __popc(__ballot_sync(0xffffffffu, mine));
          const int place = a & (p.c.page_size - 1);
          const int c2 = head * (is_k ? kp.k_head : kp.v_head);
          const int c3 = page * (is_k ? kp.k_page : kp.v_page);
          if (!(ok = wait(empty + slot, phase ^ 1u))) break;
          if (lane == 0) {
            if constexpr (kE4M3) {
              auto byte = [&](int x) { return static_cast<uint32_t>(min(max(x, 0), kTreeTile)); };
              const int pos0 = w.row();
              const bool gap = p.window > 0 && p.sinks < w.lo;
              st_shared_u32(sb + L::kInfo + slot * 8,
                            byte(gap ? p.sinks - pos0 : w.n.len - pos0) |
                                byte(gap ? w.lo - pos0 : 0) << 8 | byte(w.n.len - pos0) << 16);
              st_shared_u32(sb + L::kInfo + slot * 8 + 4, items);
            }
            mbar_arrive_expect_tx(bar(full + slot),
                                  n * (kE4M3 ? box_bytes + rows : box_bytes * L::kAtoms));
          }
          __syncwarp();
          if (mine) {
            if constexpr (kE4M3) {
              tma_load_4d(ring + slot * L::kRawTile + lane * box_bytes, tm, bar(full + slot), 0,
                          place, c2, c3);
              bulk_load(sb + L::kScales + slot * kTreeTile + lane * rows,
                        (is_k ? p.c.k_scale : p.c.v_scale) + scale_offset(p.c, page, head, place),
                        rows, bar(full + slot));
            } else {
              const uint32_t to = ring + slot * L::kTile + lane * box_bytes;
#pragma unroll
              for (int x = 0; x < L::kAtoms; ++x)
                tma_load_4d(to + x * (kTreeTile * 128), tm, bar(full + slot), x * 64, place, c2,
                            c3);
            }
          }
          next_slot();
        }
        if (i + 1 < count) {
          if (decode_advance(w.at, copies)) enter(p, w);
          if (w.at.tile == 0 || w.at.tile == window + per) load_window();
        }
      }
      if constexpr (kE4M3) {  // to both teams' warps: there is no more
#pragma unroll 1
        for (int x = 0; ok && x < 2; ++x) {
          if (!(ok = wait(empty + slot, phase ^ 1u))) break;
          if (lane == 0) {
            st_shared_u32(sb + L::kInfo + slot * 8 + 4, 0u);
            mbar_arrive(bar(full + slot));
          }
          __syncwarp();
          next_slot();
        }
      }
      // Every copy that was issued has to land before the block may end, also where another role
      // gives up and does not wait for it.
      const int each = S / kStep;
#pragma unroll 1
      for (int x = max(0, issued - each); x < issued; ++x)
        wait_drain(bar(full + slot0 + x % each * kStep), (x / each) & 1);
      __syncwarp();
    } else if (!kE4M3 && warp == kQWarp) {
      // =================== producer of Q ===================
      const uint32_t block_bytes = p.block_tokens * p.block_heads * 128u;
      int items = 0;
#pragma unroll 1
      for (int i = 0; i < count;) {
        if (!w.empty()) {
          const Rows r = rows_of(p, w.at.item, kNB);
          const int buf = items % L::kQBufs;
          if (!wait(L::bQFree + buf, (items / L::kQBufs & 1) ^ 1u)) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(L::bQFull + buf),
                                  kNB * L::kAtoms * block_bytes);
#pragma unroll
            for (int x = 0; x < kNB; ++x)
#pragma unroll
              for (int y = 0; y < L::kAtoms; ++y)
                tma_load_4d(sb + L::kQ + (buf * kNB + x) * L::kTile + y * (kTreeTile * 128),
                            &kp.tm_q, bar(L::bQFull + buf), y * 64, r.head * p.group + r.h0,
                            r.t0 + x * p.block_tokens, w.at.entry * kp.q_batch);
          }
          __syncwarp();
          ++items;
        }
        i += w.at.tiles - w.at.tile;
        if (i < count) {
          w.at.tile = w.at.tiles - 1;
          if (decode_advance(w.at, copies)) enter(p, w);
        }
      }
#pragma unroll 1
      for (int x = max(0, items - L::kQBufs); x < items; ++x)  // (as K's and V's copies)
        wait_drain(bar(L::bQFull + x % L::kQBufs), (x / L::kQBufs) & 1);
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // =================== MMA issuer ===================
      // (A/B formats: bf16 1, fp16 0; an e4m3 cache's by the item and the tile)
      constexpr uint32_t kFmt = kFp16 ? 0u : 1u, kFmtBits = (1u << 7) | (1u << 10);
      constexpr uint32_t kIdescS = idesc_f32acc<kFmt>(kTreeBlockRows, kTreeTile, false);
      constexpr uint32_t kIdescPV = idesc_f32acc<kFmt>(kTreeBlockRows, D, true);
      const uint64_t q_desc = sdesc_sw128(sb + L::kQ, 16, 1024);
      const uint64_t k_desc = sdesc_sw128(sb + L::kK, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(sb + L::kV, kTreeTile * 128, 1024);
      int k_slot = 0, v_slot = 0, items = 0, tile_count = 0;
      uint32_t k_phase = 0, v_phase = 0, p_phase[2] = {0, 0};
      uint32_t idesc_s = kIdescS;
      bool ok = true;
      auto issue_s = [&](int g, int buf) -> bool {
        if (kNB == 1 || g == 0) {
          if (!wait(L::bKFull + k_slot, k_phase)) return false;
        }
        tc_fence_after();
        const uint64_t kd = k_desc + static_cast<uint32_t>((k_slot * L::kTile) >> 4);
        const uint64_t qd =
            q_desc + static_cast<uint32_t>(((buf * kNB + (kNB == 2 ? g : 0)) * L::kTile) >> 4);
#pragma unroll
        for (int x = 0; x < L::kAtoms; ++x)
          mma_ss_x4<false, 2>(tmem + g * kTreeTile, qd + x * 1024, kd + x * 1024, idesc_s, x > 0);
        mma_commit(bar(L::bSFull + g));
        if (kNB == 1 || g == 1) {
          mma_commit(bar(L::bKEmpty + k_slot));
          if (++k_slot == SK) k_slot = 0, k_phase ^= 1u;
        }
        return true;
      };
      auto issue_pv = [&](int g, bool acc) -> bool {
        if (kNB == 1 || g == 0) {
          if (!wait(L::bVFull + v_slot, v_phase)) return false;
        }
        if (!wait(L::bPFull + g, p_phase[g])) return false;
        p_phase[g] ^= 1u;
        tc_fence_after();
        const uint64_t vd = v_desc + static_cast<uint32_t>((v_slot * L::kTile) >> 4);
        const bool wide = kE4M3 && misc[4 + tile_count % 4];
        ++tile_count;
        // 32 positions: 32 columns of S, P in 16 of them.  (Rolled beside the converters, whose
        // code takes the nearest instruction cache: 32 sequences of 4096 to 16384 take 215 us
        // unrolled, 210 rolled; without converters it is the other way round, 88 and 90 us for
        // 256 rows.)
#pragma unroll(kE4M3 ? 1 : kTreeTile / 32)
        for (int x = 0; x < kTreeTile / 32; ++x)
          mma_ts_x2<8, 128>(tmem + 256 + g * 128, tmem + g * kTreeTile + x * 32,
                            vd + static_cast<uint32_t>(x * 256),
                            wide ? kIdescPV | kFmtBits : kIdescPV, acc || x > 0);
        if (wide) {  // the second term of the weights
#pragma unroll 1
          for (int x = 0; x < kTreeTile / 32; ++x)
            mma_ts_x2<8, 128>(tmem + 256 + g * 128, tmem + g * kTreeTile + x * 32 + 16,
                              vd + static_cast<uint32_t>(x * 256), kIdescPV | kFmtBits, 1u);
        }
        mma_commit(bar(L::bPV + g));
        if (kNB == 1 || g == 1) {
          mma_commit(bar(L::bVEmpty + v_slot));
          if (++v_slot == SV) v_slot = 0, v_phase ^= 1u;
        }
        return true;
      };
#pragma unroll 1
      for (int i = 0; ok && i < count;) {
        const int tiles = min(count - i, w.at.tiles - w.at.tile);
        if (!w.empty()) {
          const int units = tiles * kNB, buf = items % L::kQBufs;
          ok = kE4M3 ? wait(L::bQFull + tree_query_bar(items), tree_query_parity(items))
                     : wait(L::bQFull + buf, items / L::kQBufs & 1);
          if (!ok) break;
          ++items;
          if constexpr (kE4M3) idesc_s = kIdescS | (misc[2] ? kFmtBits : 0u);
          ok = issue_s(0, buf);
          if (ok && units > 1) ok = issue_s(1, buf);
          if (ok && units <= 2) mma_commit(bar(L::bQFree + buf));
#pragma unroll 1
          for (int u = 0; ok && u < units; ++u) {
            const int g = u & 1;
            if (!(ok = issue_pv(g, u > 1))) break;
            if (u + 2 < units) {
              ok = issue_s(g, buf);
              if (u + 3 == units) mma_commit(bar(L::bQFree + buf));
            }
          }
        }
        i += tiles;
        if (i < count) {
          w.at.tile = w.at.tiles - 1;
          if (decode_advance(w.at, copies)) enter(p, w);
        }
      }
      // every MMA and commit has to finish before TMEM and the barriers are given back
      mma_commit(bar(L::bDrain));
      wait_drain(bar(L::bDrain), 0);
      __syncwarp();
    }
    finish();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
  } else if (kE4M3 && warp >= kConvertWarp) {
    if constexpr (kE4M3) regs_dec<kConvertRegs>();
    if (works) {
      // =================== converters ===================
      // Two teams take tiles in turn, a stage of K and V each; half of a team's warps take K,
      // half V: 32 rows of a tile to a warp, in pieces of eight rows and 64 codes, 16 of them to
      // a lane.  128-byte rows are swizzled as they come; rows 5 apart (by xor) in neighbouring
      // groups of four lanes meet no bank twice, neither there nor in the tile that is written.
      // A piece's eight rows are eight apart from the next one's: every address is one of three
      // and a constant.
      static_assert(!kE4M3 || (SK == 2 && SV == 2), "a stage to a team");
      const int member = warp - kConvertWarp, team = member / (kConvertWarps / 2);
      const bool is_v = member % (kConvertWarps / 2) >= kConvertWarps / 4;
      const int group = lane / 4;
      const int row = member % 4 * 32 + (D == 64 ? group : (group / 2) ^ (group % 2 * 5));
      const int full = (is_v ? L::bVFull : L::bKFull) + team;
      const int empty = (is_v ? L::bVEmpty : L::bKEmpty) + team;
      const uint32_t from_at =
          sb + L::kRaw + row * D + (D == 64 ? lane % 4 : lane % 4 ^ (row & 7)) * 16;
      const uint32_t to = sb + (is_v ? L::kV : L::kK) + team * L::kTile + row * 128 +
                          (2 * (lane % 4) ^ (row & 7)) * 16;
      int raw = 2 * team + (is_v ? 1 : 0), n = team;
      uint32_t raw_phase = 0, phase = 0, items = 0;
      bool wide = false;
#pragma unroll 1
      for (;; n += 2) {
        if (!wait(L::bRawFull + raw, raw_phase)) break;
        const uint32_t rows_seen = ld_shared_u32(sb + L::kInfo + raw * 8);
        const uint32_t items_now = ld_shared_u32(sb + L::kInfo + raw * 8 + 4);
        if (items_now == 0) break;
        const uint32_t from = from_at + raw * L::kRawTile;
        const uint32_t scales = sb + L::kScales + raw * kTreeTile;
        // whether a row that is seen has a scale that fp16 has not (the byte of a NaN row, 255, is
        // NaN in either type): four bytes to a lane, compared at once
        const uint32_t four = ld_shared_u32(scales + 4 * lane);
        uint32_t off = __vcmpgtu4(__vsub4(four, kScaleLow * 0x01010101u),
                                  (kScaleHigh - kScaleLow) * 0x01010101u) &
                       ~__vcmpeq4(four, 0xFFFFFFFFu);
        if (off) {
#pragma unroll 1
          for (uint32_t y = 0; y < 4; ++y) {
            const uint32_t r = 4 * lane + y;
            if (r >= (rows_seen & 255u) && (r < (rows_seen >> 8 & 255u) || r >= rows_seen >> 16))
              off &= ~(255u << (8 * y));
          }
        }
        const bool out_of_range = __any_sync(0xffffffffu, off != 0);
        if (!is_v && items != items_now) {  // the item's keys follow its queries' type
          items = items_now;
          if (!wait(L::bQFull + tree_query_bar(items - 1), tree_query_parity(items - 1))) break;
          wide = misc[2] != 0;
        }
        // What tile n is, four deep, so once tile n - 4 has its weights.  Of V early, as the
        // weights wait for it: this team's last tile, n - 2, took the stage of n - 4, whose
        // O += P V was done.  Of K once the stage is free: the scores of n - 2 are, and were
        // issued after the O += P V of n - 4.
        const uint32_t type = out_of_range && (is_v || !wide) ? 1u : 0u;
        if (is_v && member % 4 == 0 && lane == 0) {
          misc[4 + n % 4] = type;
          mbar_arrive(bar(L::bVType + n % 4));
        }
        if (!wait(empty, phase ^ 1u)) break;
        if (!is_v && member % 4 == 0 && lane == 0) misc[20 + n % 4] = type;
        // (Little code, so that it stays in the nearest instruction cache beside the other warps'.)
        if (!(is_v ? out_of_range : wide)) {
          const bool as_codes = out_of_range && !is_v;
#pragma unroll 1
          for (int y = 0; y < 4; ++y) {
            const uint32_t e = ld_shared_u8(scales + row + 8 * y);
            // 2^(e - 127) in fp16, down to its subnormals; 1 where the rows stay codes
            uint32_t s = e == 255u  ? 0x7FFFu
                         : e < 113u ? 0x0400u >> min(113u - e, 31u)
                                    : (e - 112u) << 10;
            s = as_codes ? 0x3C003C00u : (s & 0x7FFFu) * 0x00010001u;
#pragma unroll
            for (int x = 0; x < L::kAtoms; ++x) {
              const float4 v = ld_shared_v4((from ^ (x * 64)) + y * 8 * D);
              uint32_t out[8];
              e4m3x4_to_f16(__float_as_uint(v.x), out[0], out[1]);
              e4m3x4_to_f16(__float_as_uint(v.y), out[2], out[3]);
              e4m3x4_to_f16(__float_as_uint(v.z), out[4], out[5]);
              e4m3x4_to_f16(__float_as_uint(v.w), out[6], out[7]);
#pragma unroll
              for (int k = 0; k < 8; ++k) out[k] = mul_f16x2(out[k], s);
              const uint32_t at = to + x * (kTreeTile * 128) + y * 1024;
              st_shared_v4u(at, out[0], out[1], out[2], out[3]);
              st_shared_v4u(at ^ 16u, out[4], out[5], out[6], out[7]);
            }
          }
        } else {
#pragma unroll 1
          for (int y = 0; y < 4 * L::kAtoms; ++y) {
            const int x = y / 4;
            const float f = scale_value(ld_shared_u8(scales + row + 8 * (y % 4)));
            const float4 v = ld_shared_v4((from ^ (x * 64)) + y % 4 * 8 * D);
            const uint32_t in[4] = {__float_as_uint(v.x), __float_as_uint(v.y),
                                    __float_as_uint(v.z), __float_as_uint(v.w)};
            uint32_t out[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t lo, hi;
              e4m3x4_to_f16(in[k], lo, hi);
              const float2 a = unpack16<false>(lo), b = unpack16<false>(hi);
              out[2 * k] = pack16<true>(a.x * f, a.y * f);
              out[2 * k + 1] = pack16<true>(b.x * f, b.y * f);
            }
            const uint32_t at = to + x * (kTreeTile * 128) + y % 4 * 1024;
            st_shared_v4u(at, out[0], out[1], out[2], out[3]);
            st_shared_v4u(at ^ 16u, out[4], out[5], out[6], out[7]);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(full));
          mbar_arrive(bar(L::bRawEmpty + raw));
        }
        if ((raw += 4) >= L::kRawStages) raw -= L::kRawStages, raw_phase ^= 1u;
        phase ^= 1u;
      }
      __syncwarp();
    }
    finish();
    } else {
    if constexpr (kE4M3) regs_inc<kSoftRegs>();
    if (works) {
      // =================== softmax ===================
      const int g = warp / (kSoft / 2), half = kH == 2 ? warp / 4 % 2 : 0, quarter = warp % 4;
      const int r = quarter * 32 + lane;  // TMEM lane
      const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
      // (e4m3) Where a block has up to 64 rows they stand twice among the 128 of the MMA, and each
      // copy takes half of a tile's positions (its weights for the others are 0), with statistics
      // and an O of its own: the softmax takes half as long, and the copies are joined at the
      // item's end (32 sequences of 4096 to 16384, 64 rows: 210 us; a row once: 233).  Not for
      // 16-bit caches: 0 times an infinite value would be NaN; an e4m3 cache has none below the
      // headroom's end.
      const int rows_of_copy = kE4M3 && p.copies == 2 ? kTreeBlockRows / 2 : kTreeBlockRows;
      const int copy = r / rows_of_copy, row_in = r - copy * rows_of_copy;
      const int pieces = kTreeTile / 16 / kH / (kTreeBlockRows / rows_of_copy);  // of 16 scores
      const int piece0 = (copy * kH + half) * pieces;
      const uint32_t s_at = tmem + lanes + g * kTreeTile;
      const uint32_t o_at = tmem + lanes + 256 + g * 128;
      const uint32_t pair = 1 + g * 4 + quarter;  // named barrier of the warps that share rows
      constexpr uint32_t kNan = 0x7FFFFFFFu;
      float* refs = fin;                         // [2 groups][128]
      float* sums = fin + 2 * kTreeBlockRows;    // [2 groups][128]
      float* mine_s = sums + g * kTreeBlockRows + r;
      uint32_t s_phase = 0;  // of bSFull[g] and bPV[g]: both complete once a tile of the group
      uint32_t sync_phase = 0;
      int tile_count = 0, v_slot = 0;
      int parity = 0;  // of the items so far (tree_query_bar)
      uint32_t v_phase = 0;
      auto step = [&]() {
        if (++v_slot == SV) v_slot = 0, v_phase ^= 1u;
        ++tile_count;
      };
      // All softmax warps are here (and what they wrote to shared memory before is seen); false
      // where a wait has run out.  The warps that share rows go on together or leave together: one
      // may find the flag that ends waits where the other found the barrier complete, and they meet
      // at barriers that know no limit.
      auto sync_all = [&](bool fine) -> bool {
        if (fine) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::bSync));
          fine = wait(L::bSync, sync_phase);
          sync_phase ^= 1u;
          tc_fence_after();
        }
        if constexpr (kH == 2) fine = !named_bar_or(pair, 64, !fine);
        return fine;
      };
      int i = 0;
      bool ok = true;
      if (threadIdx.x < 4) bad_s[threadIdx.x] = 0;
      if (kE4M3 && threadIdx.x < 4) misc[8 + threadIdx.x] = 0;
      if (kE4M3 && threadIdx.x == 0) misc[2] = 0;
      ok = sync_all(true);
#pragma unroll 1
      while (ok && i < count) {
        const int tiles = min(count - i, w.at.tiles - w.at.tile);
        const bool from_start = w.at.tile == 0;
        const Rows at0 = rows_of(p, w.at.item, kNB);
        const int b = w.at.entry;
        unsigned long long* bad = bad_s + 2 * parity;
        // ---- this thread's row ----
        const int block_rows = p.block_tokens * p.block_heads;
        const int t_in = row_in / p.block_heads, h_in = row_in - t_in * p.block_heads;
        const int t = at0.t0 + (kNB == 2 ? g * p.block_tokens : 0) + t_in, h = at0.h0 + h_in;
        const bool there = row_in < block_rows && t < p.tokens && h < p.group;
        const bool live = there && t < w.n.drafted;
        const bool warp_live = __any_sync(0xffffffffu, live);
        const int my_row = (kNB == 2 ? g * block_rows : 0) + row_in;  // within the item
        const int context = w.context();
        float down = 1.f;  // what makes the queries of the product out of what they became
        if constexpr (kE4M3) {
          // ---- Q: rows of 128-byte slabs, chunks of 16 bytes permuted by the row ----
          if (!w.empty()) {
            // 16 bytes of every kStep-th row to a thread, which come to their places as they are.
            // (Rolled loops: straight code that runs once an item is fetched as it runs.)
            constexpr int kChunks = D / 8, kStep = 32 * kSoft / kChunks;
            static_assert(kStep % 8 == 0, "one place in the swizzle to a thread");
            const int c = threadIdx.x % kChunks, row0 = threadIdx.x / kChunks;
            const uint32_t q_at = sb + L::kQ + (c / 8) * (kTreeTile * 128) + row0 * 128 +
                                  ((c % 8) ^ (row0 & 7)) * 16;
            const uint32_t second = (kTreeBlockRows / 2) * 128;  // the second copy's rows
            const uint8_t* q_from = p.q + wide(b, p.q_batch) + wide(at0.t0, p.q_token) +
                                    wide(at0.head * p.group + at0.h0, p.q_head) + c * 16;
#pragma unroll 1
            for (int row = row0; row < rows_of_copy; row += kStep) {
              const int qt = row / p.block_heads, qh = row - qt * p.block_heads;
              const bool is =
                  row < block_rows && at0.t0 + qt < w.n.drafted && at0.h0 + qh < p.group;
              const uint8_t* from = is ? q_from + wide(qt, p.q_token) + wide(qh, p.q_head) : p.q;
              const uint32_t to = q_at + (row - row0) * 128;
              cp_async16(to, from, is ? 16u : 0u);  // (the others are zeros)
              if (!kOutBf16 && rows_of_copy < kTreeBlockRows)
                cp_async16(to + second, from, is ? 16u : 0u);
            }
            cp_async_wait_all();
            if constexpr (kOutBf16) {
              uint32_t most = 0, least = 0xFFFFFFFFu;
#pragma unroll 1
              for (int row = row0; row < rows_of_copy; row += kStep) {
                const float4 v = ld_shared_v4(q_at + (row - row0) * 128);
                const uint32_t in[4] = {__float_as_uint(v.x), __float_as_uint(v.y),
                                        __float_as_uint(v.z), __float_as_uint(v.w)};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  // magnitudes compare as integers, two at a time: the largest, and the least but
                  // zero, less 1; infinities and NaN are what they are at any scale
                  uint32_t m = in[k] & 0x7FFF7FFFu;
                  m &= ~__vcmpgeu2(m, 0x7F807F80u);
                  most = __vmaxu2(most, m);
                  least = __vminu2(least, __vsub2(m, 0x00010001u));
                }
              }
              most = __reduce_max_sync(0xffffffffu, max(most >> 16, most & 0xFFFFu));
              least = __reduce_min_sync(0xffffffffu, min(least >> 16, least & 0xFFFFu));
              if (lane == 0) {
                atomicMax(const_cast<uint32_t*>(misc + 8 + 2 * parity), most);
                atomicMax(const_cast<uint32_t*>(misc + 9 + 2 * parity), 0xFFFFu - least);
              }
              if (!(ok = sync_all(true))) break;
              most = misc[8 + 2 * parity] >> 7;  // exponent bytes
              least = (0xFFFFu - misc[9 + 2 * parity] + 1u) >> 7;
              // The largest magnitude goes into [2^14, 2^15): an element keeps all its bits down
              // to 2^-31 of it, as bits of 2^-24 and above.  Else q stays bf16.
              const bool keep = least + 31u < most || most < 15u;
              const uint32_t up = 127u + 141u - most;  // the exponent byte of q's factor
              if (threadIdx.x == 0) misc[2] = keep ? 1u : 0u;
              if (!keep) down = __uint_as_float((254u - up) << 23);
              const float f = __uint_as_float(up << 23);
#pragma unroll 1
              for (int row = row0; row < rows_of_copy; row += kStep) {
                const uint32_t to = q_at + (row - row0) * 128;
                const float4 v = ld_shared_v4(to);
                uint32_t in[4] = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                                  __float_as_uint(v.w)};
                if (!keep) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const float2 q2 = unpack16<true>(in[k]);
                    in[k] = pack16<false>(q2.x * f, q2.y * f);
                  }
                  st_shared_v4u(to, in[0], in[1], in[2], in[3]);
                }
                if (rows_of_copy < kTreeBlockRows)
                  st_shared_v4u(to + second, in[0], in[1], in[2], in[3]);
              }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::bQFull + parity));
          }
        }
        TreeRow seen;
        seen.mask = 0;
        seen.lo = 0;
        if (live) seen = tree_row(p, w.n, b, t);
        float ref = 0.f, limit = -INFINITY, sum = 0.f;
        int mine = 0;       // tiles of this group so far in this item
        bool dead = false;  // a wait ran out; the warps of a row leave the loop together
#pragma unroll 1
        for (int local = 0; local < tiles && !w.empty(); ++local, ++w.at.tile) {
          if (kNB == 1 && (local & 1) != g) {
            step();
            continue;
          }
          const int pos0 = w.row();
          const bool whole_tile = all_seen(p, w, pos0, pos0 + kTreeTile);
          if (!wait(L::bSFull + g, s_phase)) dead = true;
          tc_fence_after();
          const bool codes = kE4M3 && misc[20 + tile_count % 4] != 0;
          // (keys that stayed codes take `down` into their scales: either factor alone may pass
          // what fp32 holds)
          const float scale = kE4M3 && !codes ? p.scale_log2 * down : p.scale_log2;
          if (kE4M3 && rows_of_copy < kTreeBlockRows) {  // the other copy's positions
            const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tmem_st8(s_at + (1 - copy) * 64 + 8 * (k + k / 2 * 2), none);
          }
          float top = -INFINITY;
          if (warp_live && !dead) {
            auto maximum = [&](const uint32_t* s) {  // of 16 scores
              float mx[2];
#pragma unroll
              for (int a = 0; a < 2; ++a) {
                mx[a] = fmax3(__uint_as_float(s[8 * a]), __uint_as_float(s[8 * a + 1]),
                              __uint_as_float(s[8 * a + 2]));
#pragma unroll
                for (int x = 3; x < 7; x += 2)
                  mx[a] = fmax3(mx[a], __uint_as_float(s[8 * a + x]),
                                __uint_as_float(s[8 * a + x + 1]));
                mx[a] = fmaxf(mx[a], __uint_as_float(s[8 * a + 7]));
              }
              top = fmax3(top, mx[0], mx[1]);
            };
            // (Little code: what does not fit the nearest instruction cache beside the other warps'
            // costs more than a loop.)
            if (whole_tile && !codes) {
#pragma unroll 1
              for (int k = piece0; k < piece0 + pieces; k += 2) {
                uint32_t s[32];
                tmem_ld32(s_at + 16 * k, s);
                tmem_wait_ld(s);
                maximum(s);
                maximum(s + 16);
              }
            } else {
              // what the row does not see becomes -inf, for the second pass too
#pragma unroll 1
              for (int k = piece0; k < piece0 + pieces; ++k) {
                uint32_t s[16];
                tmem_ld16(s_at + 16 * k, s);
                const int base = pos0 + 16 * k;
                uint32_t m = below(context - base);
                if (p.window > 0) m &= below(p.sinks - base) | ~below(seen.lo - base);
                const int shift = context - base;  // bit of the first drafted token
                m |= shift >= 32 || shift <= -64 ? 0u
                     : shift >= 0               ? static_cast<uint32_t>(seen.mask << shift)
                                                : static_cast<uint32_t>(seen.mask >> -shift);
                if (!live) m = 0;
                tmem_wait_ld(s);
                if (kE4M3 && codes) {  // (hardly ever) keys whose scales fp16 does not hold
                  const int j = base + lane % 16;
                  float f = 1.f;
                  if (some_seen(p, w, j, j + 1)) {
                    const int page = table_page(p.t, p.c.num_pages, b, j >> p.c.page_shift);
                    if (page >= 0)
                      f = down * scale_value(p.c.k_scale[scale_offset(p.c, page, at0.head,
                                                                      j & (p.c.page_size - 1))]);
                  }
#pragma unroll
                  for (int x = 0; x < 16; ++x)
                    s[x] = __float_as_uint(__uint_as_float(s[x]) * __shfl_sync(0xffffffffu, f, x));
                }
#pragma unroll
                for (int x = 0; x < 16; ++x)
                  if (!(m >> x & 1u)) s[x] = 0xFF800000u;
                tmem_st16(s_at + 16 * k, s);
                maximum(s);
              }
              tmem_wait_st();
            }
          }
          float z = top * scale;
          bool any;
          if constexpr (kH == 2) {
            any = named_bar_or(pair, 64, dead || z > limit);
            if (any) {  // the row's maximum, by way of the first of its threads
              if (half == 1) *mine_s = dead ? __uint_as_float(kNan) : z;
              named_bar_sync(pair, 64);
              if (half == 0) {
                const float other = *mine_s;
                z = dead || other != other ? __uint_as_float(kNan) : fmaxf(z, other);
                *mine_s = z;
              }
              named_bar_sync(pair, 64);
              if (half == 1) z = *mine_s;
              if (__any_sync(0xffffffffu, z != z)) dead = true;
            }
          } else {
            any = __any_sync(0xffffffffu, z > limit);
          }
          if (dead) break;
          if (any) {
            const bool raise = z > limit;
            float f = 1.f;
            if (raise) {
              const float to = z - kShift<kType>;
              if (limit != -INFINITY) f = ex2_approx(ref - to);  // (else nothing is summed yet)
              ref = to;
              limit = z + kRaise<kType>;
              sum *= f;
            }
            if (mine > 0 && warp_live) {
              // O refers to the old reference: once the last O += P V has landed
              if (!wait(L::bPV + g, s_phase ^ 1u)) {
                dead = true;  // (leaves with the row's other thread, at the next tile)
              } else {
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < D / 32 / kH; ++k) {
                  uint32_t o[32];
                  const uint32_t at = o_at + half * (D / kH) + 32 * k;
                  tmem_ld32(at, o);
                  tmem_wait_ld(o);
#pragma unroll
                  for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                  tmem_st32(at, o);
                }
              }
            }
          }
          if (warp_live) {
            bool wide = false;  // this tile's V is bf16
            if constexpr (kE4M3) {
              if (!wait(L::bVType + tile_count % 4, tile_count / 4 & 1)) dead = true;
              wide = misc[4 + tile_count % 4] != 0;
            }
            if (kE4M3 && rows_of_copy < kTreeBlockRows) {  // the other copy's positions
              const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
              for (int k = 2; k < 8; ++k)
                if (k % 4 >= 2 && wide) tmem_st8(s_at + (1 - copy) * 64 + 8 * k, none);
            }
            const uint64_t c2 = f2_pack(scale, scale), r2 = f2_pack(-ref, -ref);
            uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
            if (!kE4M3 || !wide) {
#pragma unroll 1
              for (int k = piece0; k < piece0 + pieces; k += 2) {
                uint32_t s[32], pk[16];
                tmem_ld32(s_at + 16 * k, s);
                tmem_wait_ld(s);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const uint64_t z2 = f2_fma(
                      f2_pack(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])), c2, r2);
                  float z0, z1;
                  f2_unpack(z2, z0, z1);
                  z0 = ex2_approx(z0);
                  z1 = ex2_approx(z1);
                  acc[x & 1] = f2_add(acc[x & 1], f2_pack(z0, z1));
                  pk[x] = pack16<!kFp16>(z0, z1);
                }
                tmem_st16(s_at + 16 * k, pk);  // (the first half of its 32 scores' columns)
              }
            } else {  // as two bf16 terms
#pragma unroll 1
              for (int k = piece0; k < piece0 + pieces; k += 2) {
                uint32_t s[32], hi[16], lo[16];
                tmem_ld32(s_at + 16 * k, s);
                tmem_wait_ld(s);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                  const float z0 = ex2_approx(fmaf(__uint_as_float(s[2 * x]), scale, -ref));
                  const float z1 = ex2_approx(fmaf(__uint_as_float(s[2 * x + 1]), scale, -ref));
                  acc[x & 1] = f2_add(acc[x & 1], f2_pack(z0, z1));
                  hi[x] = pack16<true>(z0, z1);
                  const float2 h = unpack16<true>(hi[x]);
                  lo[x] = pack16<true>(z0 - h.x, z1 - h.y);
                }
                tmem_st16(s_at + 16 * k, hi);
                tmem_st16(s_at + 16 * k + 16, lo);
              }
            }
            float a0, a1;
            f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
            sum += a0 + a1;
            tmem_wait_st();
          }
          if (!whole_tile && half == 0) {
            // ---- V's rows that not every row sees: thread r looks after position r ----
            if (!wait(L::bVFull + v_slot, v_phase)) dead = true;
            const int j = pos0 + r;
            if (!dead && !(j < context && (p.window <= 0 || j < p.sinks || j >= w.hi))) {
              const bool drafted = j >= context && j < w.n.len;
              const bool border = j < context && j >= w.lo;
              const bool zero = !(drafted || border);
              const bool wide = kE4M3 && misc[4 + tile_count % 4] != 0;
              const uint32_t line = sb + L::kV + v_slot * L::kTile + r * 128;
              // (chunks in the order of the swizzle: neighbouring rows meet no bank twice)
              auto at = [&](int c) {
                return line + c / 8 * (kTreeTile * 128) + ((c % 8) ^ (r & 7)) * 16;
              };
              auto odd_in = [&](uint32_t v) {
                return kFp16 && !wide ? not_finite<true>(v) : not_finite<false>(v);
              };
              uint32_t odd = 0;
              if (!zero) {
#pragma unroll 2
                for (int c = 0; c < 8 * L::kAtoms; ++c) {
                  const float4 f = ld_shared_v4(at(c));
                  odd |= odd_in(__float_as_uint(f.x)) | odd_in(__float_as_uint(f.y));
                  odd |= odd_in(__float_as_uint(f.z)) | odd_in(__float_as_uint(f.w));
                }
              }
              if (odd & 0x80008000u) {
                // noted before they are gone: the other group may look at the same row
                atomicOr(&bad[drafted ? 0 : 1], 1ull << (drafted ? j - context : j - w.lo));
                __threadfence_block();
#pragma unroll 1
                for (int c = 0; c < 32 * L::kAtoms; ++c) {
                  const uint32_t word = at(c / 4) + c % 4 * 4;
                  uint32_t v = ld_shared_u32(word);
                  const uint32_t n = odd_in(v);
                  if (n & 0x8000u) v &= 0xFFFF0000u;
                  if (n & 0x80000000u) v &= 0x0000FFFFu;
                  st_shared_u32(word, v);
                }
              }
              if (zero) {
#pragma unroll 2
                for (int c = 0; c < 8 * L::kAtoms; ++c) st_shared_v4u(at(c), 0u, 0u, 0u, 0u);
              }
            }
            fence_async_shared();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::bPFull + g));
          s_phase ^= 1u;
          ++mine;
          step();
          if (kH == 1 && dead) break;
        }
        // ---- the item's end: the block's part of O ----
        if (!dead && mine > 0 && !wait(L::bPV + g, s_phase ^ 1u)) dead = true;
        tc_fence_after();
        if (w.empty()) w.at.tile += tiles;
        const bool done = w.at.tile == w.at.tiles;
        // A block leaves at most two unfinished items: its first one (part 0) and its last.
        const bool whole = done && from_start;
        const int part = i == 0 ? 0 : 1;
        float f0 = 1.f, f1 = 0.f;  // of this group's O and of the other's
        float base = limit == -INFINITY ? -INFINITY : ref;
        if (!w.empty()) {
          // the row's sum: of its threads, and of both groups where they have the same rows
          if constexpr (kH == 2) {
            if (half == 1) *mine_s = sum;
            named_bar_sync(pair, 64);
            if (half == 0) *mine_s = sum += *mine_s;
          } else {
            *mine_s = sum;
          }
          if (half == 0) refs[g * kTreeBlockRows + r] = base;
          if (!(ok = sync_all(!dead))) break;
          sum = *mine_s;
          if constexpr (kNB == 1) {
            // both groups and copies: the largest reference, and what theirs count relative to it
            float m = -INFINITY;
#pragma unroll 1
            for (int x = row_in; x < kTreeBlockRows; x += rows_of_copy)
              m = fmaxf(m, fmaxf(refs[x], refs[kTreeBlockRows + x]));
            const float to = m == -INFINITY ? 0.f : m;
            // (a NaN in the sum of a row without a finite score stays one)
            auto factor = [&](float ref_of) {
              return ref_of == -INFINITY ? 1.f : ex2_approx(ref_of - to);
            };
            sum = 0.f;
#pragma unroll 1
            for (int x = row_in; x < kTreeBlockRows; x += rows_of_copy)
              sum += sums[x] * factor(refs[x]) +
                     sums[kTreeBlockRows + x] * factor(refs[kTreeBlockRows + x]);
            f0 = factor(base);
            f1 = factor(refs[(g ^ 1) * kTreeBlockRows + r]);
            base = m;
          }
        }
        if (!live) sum = 0.f;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float lse = sum == 0.f ? -INFINITY : (base == -INFINITY ? 0.f : base) + log2f(sum);
        const long long at =
            ((static_cast<long long>(b) * p.tokens + t) * p.c.heads + at0.head) * p.group + h;
        const bool have1 = kNB == 1 && tiles > 1;
        constexpr int kCols = (kNB == 1 ? D / 2 : D) / kH;  // of this thread
        const int col0 = kNB == 1 ? (g * kH + half) * kCols : half * kCols;
        // the O of tile 0's group and of the other one
        const uint32_t o_first = (kNB == 1 ? tmem + lanes + 256 : o_at) + col0;
        const float w0 = kNB == 1 && g == 1 ? f1 : f0, w1 = g == 1 ? f0 : f1;
        // The second copy's O goes to the first by way of Q's memory, four columns of all rows and
        // then the next four.
        const bool joined = kE4M3 && rows_of_copy < kTreeBlockRows && !w.empty();
        const uint32_t stage = sb + L::kQ + row_in * 16;
        if (joined) {
          if (copy == 1) {
#pragma unroll 1
            for (int k = 0; k < kCols; k += 16) {
              uint32_t o[16], o2[16];
              tmem_ld16(o_first + k, o);
              tmem_wait_ld(o);
              if (have1) {
                tmem_ld16(o_first + 128 + k, o2);
                tmem_wait_ld(o2);
              }
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                float x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  x[y] = __uint_as_float(o[c + y]) * w0;
                  if (have1) x[y] = fmaf(__uint_as_float(o2[c + y]), w1, x[y]);
                }
                st_shared_v4(stage + (col0 + k + c) / 4 * (kTreeBlockRows / 2 * 16), x[0], x[1],
                             x[2], x[3]);
              }
            }
          }
          if (!(ok = sync_all(true))) break;
        }
        if (copy == 0 && __any_sync(0xffffffffu, there)) {
#pragma unroll 1
          for (int k = 0; k < kCols; k += 16) {
            uint32_t o[16];
            tmem_ld16(o_first + k, o);
            tmem_wait_ld(o);
            float x[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(o[c]) * w0;
            if (have1) {
              tmem_ld16(o_first + 128 + k, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int c = 0; c < 16; ++c) x[c] = fmaf(__uint_as_float(o[c]), w1, x[c]);
            }
            if (joined) {
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                const float4 v =
                    ld_shared_v4(stage + (col0 + k + c) / 4 * (kTreeBlockRows / 2 * 16));
                x[c] += v.x, x[c + 1] += v.y, x[c + 2] += v.z, x[c + 3] += v.w;
              }
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = sum == 0.f ? 0.f : x[c] * inv;
            if (there) {
              if (whole) {
                uint4* out = reinterpret_cast<uint4*>(p.o + (at * D + col0 + k) * 2);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  out[c] = make_uint4(pack16<kOutBf16>(x[8 * c], x[8 * c + 1]),
                                      pack16<kOutBf16>(x[8 * c + 2], x[8 * c + 3]),
                                      pack16<kOutBf16>(x[8 * c + 4], x[8 * c + 5]),
                                      pack16<kOutBf16>(x[8 * c + 6], x[8 * c + 7]));
              } else {
                float4* out = reinterpret_cast<float4*>(
                                  p.workspace + rows_at(blockIdx.x, part, p.item_rows, D)) +
                              (col0 + k) / 4 * p.item_rows + my_row;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  out[c * p.item_rows] =
                      make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
              }
            }
          }
          // non-finite values that only some rows see, this one among them
          if (live && (bad[0] | bad[1])) {
            uint16_t* out = whole ? reinterpret_cast<uint16_t*>(p.o) + at * D : nullptr;
            float* ws = reinterpret_cast<float*>(p.workspace +
                                                 rows_at(blockIdx.x, part, p.item_rows, D)) +
                        4 * my_row;
            add_not_finite<kType, kOutBf16>(p, b, at0.head, context, bad[0] & seen.mask, col0,
                                            kCols, out, ws);
            const int behind = seen.lo - w.lo;  // of the border positions, those not seen
            add_not_finite<kType, kOutBf16>(p, b, at0.head, w.lo,
                                            behind >= 64 ? 0ull : bad[1] >> behind << behind, col0,
                                            kCols, out, ws);
          }
          if (there && half == 0 && (kNB == 2 || g == 0)) {
            if (whole)
              p.lse[at] = lse * 0.69314718055994531f;
            else
              reinterpret_cast<float*>(p.workspace +
                                       lse_at(blockIdx.x, part, p.item_rows))[my_row] = lse;
          }
        }
        const int units = w.at.tiles + tree_cost(p, w.n);
        if (!done && from_start && threadIdx.x == 0) {
          Join j;
          j.entry = b;
          j.item = w.at.item;
          j.last = static_cast<int>((begin + unit + units - 1) / share);
          j.part = part;
          reinterpret_cast<Join*>(p.workspace)[blockIdx.x] = j;
        }
        unit += units;
        i += tiles;
        if (i < count) {
          if (!w.empty()) {
            // (what the item before this one used; this one's may still be looked at)
            parity ^= 1;
            if (threadIdx.x < 2) bad_s[2 * parity + threadIdx.x] = 0;
            if (kE4M3 && threadIdx.x < 2) misc[8 + 2 * parity + threadIdx.x] = 0;
            if (!(ok = sync_all(true))) break;  // O is free, and nobody looks at `fin` any more
          }
          w.at.tile = w.at.tiles - 1;
          if (decode_advance(w.at, copies)) enter(p, w);
        }
      }
      tmem_wait_st();  // (a warp that leaves early may have stores on their way)
      __syncwarp();
    }
    finish();
  }
}

// The join of an item's parts: eight columns of a row of the item that starts, unfinished, in
// block blockIdx.x of tree_kernel to a thread, neighbouring rows to neighbouring threads.
// Parts are taken in order, a batch of loads at a time.
constexpr int kJoinThreads = 128;
template <int D, bool kOutBf16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const TreeParams p, int rows_most) {
  constexpr int kBatch = 4;
  const int c0 = blockIdx.x, job = blockIdx.y * kJoinThreads + threadIdx.x;
  const int cols = job / rows_most, row = job - cols * rows_most;
  grid_dep_wait();
  const Join j = reinterpret_cast<const Join*>(p.workspace)[c0];
  if (j.last < 0 || cols >= D / 8) return;
  const int block_rows = p.block_tokens * p.block_heads;
  const Rows r = rows_of(p, j.item, p.item_rows / block_rows);
  const int t = r.t0 + row / p.block_heads, h = r.h0 + row % p.block_heads;
  if (t >= p.tokens || h >= p.group) return;
  float top = -INFINITY, sum = 0.f, acc[8] = {};
#pragma unroll 1
  for (int c = c0; c <= j.last; c += kBatch) {
    float lse[kBatch];
    float4 x[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int at = min(c + i, j.last), part = at == c0 ? j.part : 0;
      lse[i] = reinterpret_cast<const float*>(p.workspace + lse_at(at, part, p.item_rows))[row];
      const float4* o =
          reinterpret_cast<const float4*>(p.workspace + rows_at(at, part, p.item_rows, D)) + row;
      x[i][0] = o[2 * cols * p.item_rows];
      x[i][1] = o[(2 * cols + 1) * p.item_rows];
    }
    float m = top;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) m = fmaxf(m, lse[i]);
    if (m > top) {
      const float f = top == -INFINITY ? 1.f : ex2_approx(top - m);
      sum *= f;
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] *= f;
      top = m;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (c + i > j.last || lse[i] == -INFINITY) continue;  // (an empty part: zeros)
      const float f = ex2_approx(lse[i] - (top == -INFINITY ? 0.f : top));
      sum += f;
      const float v[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                          x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(f, v[k], acc[k]);
    }
  }
  const long long at =
      ((static_cast<long long>(j.entry) * p.tokens + t) * p.c.heads + r.head) * p.group + h;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  reinterpret_cast<uint4*>(p.o)[at * (D / 8) + cols] =
      make_uint4(pack16<kOutBf16>(acc[0] * inv, acc[1] * inv),
                 pack16<kOutBf16>(acc[2] * inv, acc[3] * inv),
                 pack16<kOutBf16>(acc[4] * inv, acc[5] * inv),
                 pack16<kOutBf16>(acc[6] * inv, acc[7] * inv));
  if (cols == 0)
    p.lse[at] = sum == 0.f ? -INFINITY
                           : ((top == -INFINITY ? 0.f : top) + log2f(sum)) * 0.69314718055994531f;
}

// ---- host ----

template <typename K, typename... A>
bool launch_kernel(K kernel, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                   bool early, const A&... args) {
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

template <int D, int kType, int kNB>
int launch(const KernelParams& kp, int dev, int sms, cudaStream_t stream) {
  using L = Layout<D, kType, kNB>;
  constexpr int kThreads = kThreadsOf<kType>;
  auto kernel = tree_kernel<D, kType, kNB>;
  static std::once_flag once[kMaxDevices];
  static bool ready[kMaxDevices];
  std::call_once(once[dev], [&] {
    // (the split of the registers inside an e4m3 kernel assumes those that it starts with:
    // anything else could make a warp wait for more without end)
    cudaFuncAttributes fa;
    ready[dev] = cudaFuncGetAttributes(&fa, kernel) == cudaSuccess &&
                 (!L::kE4M3 || fa.numRegs == kLaunchRegs) &&
                 cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      L::kBytes) == cudaSuccess;
  });
  if (!ready[dev]) return -4;
  const TreeParams& p = kp.p;
  const long long items =
      static_cast<long long>(p.t.batch) * p.c.heads * p.token_items * p.head_items;
  const long long tiles =
      decode_span_most(static_cast<long long>(p.t.width) << p.c.page_shift,
                       p.window > 0 ? (p.window < (1 << 30) ? p.window : 1 << 30) + p.tokens : 0,
                       p.sinks, kTreeTile);
  long long grid = sms < kTreeMaxBlocks ? sms : kTreeMaxBlocks;
  if (items <= grid &&
      (tiles <= kTreeDirect || (tiles <= (p.window > 0 ? kTreeWholeWindow : kTreeWhole) &&
                                tiles * (grid - items) <= 6 * grid))) {
    KernelParams one = kp;
    one.p.direct = 1;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(items)), kThreads, L::kBytes, stream,
                         false, one)
               ? 0
               : -4;
  }
  if (grid > tiles * items) grid = tiles * items;
  if (!launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), kThreads, L::kBytes, stream, false,
                     kp))
    return -4;
  const int rows = p.item_rows;
  const dim3 join(static_cast<unsigned>(grid), (rows * (D / 8) + kJoinThreads - 1) / kJoinThreads);
  return launch_kernel(join_kernel<D, kType == kBf16 || kType == kE4M3Bf16>, join, kJoinThreads, 0,
                       stream, true, p, rows)
             ? 0
             : -4;
}

}  // namespace tree

}  // namespace fat
