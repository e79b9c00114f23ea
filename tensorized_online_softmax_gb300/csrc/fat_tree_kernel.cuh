// Attention of drafted tokens over the paged cache.
//
// What bounds it: the rows (drafted token, query head of the group) of a cached head
// share one pass over its keys and values.  Up to about 256 rows that is a stream
// through HBM (4 rows flops to 2 bytes of a 16-bit cache); the products take the
// tensor pipe a quarter (128 rows) to a half (256) of that time, so all else has to
// hide behind the copies.
//
// Work: an item is a block of 128 or 256 rows of one (sequence, cached head); its
// positions are walked in tiles of 128 (tree_span: with a window only those that a
// row may see).  The tiles of all items form one line, of which every thread block
// takes an equal share (fat_decode_plan.h); items that blocks share leave normalised
// parts in the workspace for the join kernel, in a fixed order.
//
//   warps 0-7   softmax in two groups of four, one row to a thread.  Of 256 rows each
//               group takes its half at every tile; of up to 128 both have the same rows
//               and take alternate tiles, with an O and statistics of their own that
//               are joined at the item's end: no group ever waits for the other inside
//               an item.  They load Q at an item's start, and write O at its end.
//   warp 8      MMA issuer: S_g = Q_g K^T (tcgen05, 128 x 128), O_g += P_g V.
//   warps 9,10  producers of K and V: one TMA box for each page of a tile.
//   warps 12-19 (e4m3 caches) converters: warp 9 brings the codes and scale bytes to a ring
//               of their own, and these warps make bf16 rows of them in the rings of K and
//               V.  A code times a power of two is exact in bf16.  fp16 queries go as two bf16
//               terms, which hold all their bits, and their weights as two as well.
//
// TMEM: S_0, S_1 (P_g over S_g), O_0, O_1: 512 columns.
//
// Per score: z = scale log2(e) s - r with a running reference r for each row, raised to
// the row's maximum only where a tile exceeds it by more than kRaise binades (then O is
// rescaled in TMEM: a rare event).  The scores are read twice from TMEM, for the
// maximum and for the weights: it has the bandwidth, and 128 scores to a thread would
// need the registers of two.  P is rounded to 16 bits, the sum of the row is not.
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

constexpr int kGroupThreads = 128;
constexpr int kMmaWarp = 8, kKWarp = 9, kVWarp = 10;
constexpr int kConvertWarp = 12, kConvertWarps = 8;
template <int kType>
constexpr int kThreadsOf = kType >= kE4M3Bf16 ? 640 : 384;
constexpr uint32_t kTmemCols = 512;
// binades above the maximum at the last raise that are let pass; fp16 weights are
// 2^kShift at that maximum (2^15 is the most fp16 holds)
template <bool kFp16>
constexpr float kRaise = kFp16 ? 4.f : 8.f;
template <bool kFp16>
constexpr float kShift = kFp16 ? 11.f : 0.f;

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
  CUtensorMap tm_k, tm_v;
  TreeParams p;
  // 0 where all heads, or pages, are the same memory (a stride of 0)
  int k_head, k_page, v_head, v_page;
};

template <int D, int kType, int kNB>
struct Layout {
  static constexpr bool kE4M3 = kType >= kE4M3Bf16;
  static constexpr int kParts = kType == kE4M3F16 ? 2 : 1;  // 16-bit terms of q and of a weight
  static constexpr int kTile = kTreeTile * D * 2;
  // stages of K and V, and of an e4m3 cache's codes: what the shared memory has room for
  static constexpr int kKStages = kE4M3 ? 2 : D == 64 ? (kNB == 1 ? 6 : 5) : kNB == 1 ? 3 : 2;
  static constexpr int kStages = kE4M3 ? 2 : D == 64 ? (kNB == 1 ? 6 : 5) : 3;
  static constexpr int kRawStages = !kE4M3 ? 0 : D == 64 ? 12 : kParts == 2 ? 2 : 4;
  static constexpr int kRawTile = kTreeTile * D;  // codes
  static constexpr int kAtoms = D / 64;  // slabs of 64 columns (128 bytes)
  static constexpr int kQ = 0;
  static constexpr int kK = kNB * kParts * kTile;
  static constexpr int kV = kK + kKStages * kTile;
  static constexpr int kRaw = kV + kStages * kTile;
  static constexpr int kScales = kRaw + kRawStages * kRawTile;  // of the codes' rows
  static constexpr int kBars = kScales + kRawStages * kTreeTile;
  static constexpr int bKFull = 0;
  static constexpr int bKEmpty = bKFull + kKStages;
  static constexpr int bVFull = bKEmpty + kKStages;
  static constexpr int bVEmpty = bVFull + kStages;
  static constexpr int bRawFull = bVEmpty + kStages;
  static constexpr int bRawEmpty = bRawFull + kRawStages;
  static constexpr int bSFull = bRawEmpty + kRawStages;  // [2]
  static constexpr int bPFull = bSFull + 2;              // [2], 4 arrivals
  static constexpr int bPV = bPFull + 2;                 // [2]
  static constexpr int bQFull = bPV + 2;                 // 8 arrivals
  static constexpr int bSync = bQFull + 1;               // 8 arrivals: both groups are here
  static constexpr int bDrain = bSync + 1;
  static constexpr int kNumBars = bDrain + 1;
  static __device__ __forceinline__ int arrivals(int bar) {
    if (kE4M3 && ((bar >= bKFull && bar < bKEmpty) || (bar >= bVFull && bar < bVEmpty) ||
                  (bar >= bRawEmpty && bar < bSFull)))
      return kConvertWarps / 2;
    return bar == bPFull || bar == bPFull + 1 ? 4 : bar == bQFull || bar == bSync ? 8 : 1;
  }
  static constexpr int kMisc = kBars + ((8 * kNumBars + 15) & ~15);
  // u32: TMEM base, abort flag, -, -; DecodePlace; u64 bad[2]
  static constexpr int kStart = kMisc + 16;
  static constexpr int kBad = kStart + 16;
  // float [2 groups][2][128]: reference and sum of each row; ahead of that the plan's sums
  static constexpr int kFin = kBad + 16;
  static constexpr int kBytes = kFin + 2 * 2 * kTreeBlockRows * 4;
  static_assert(kRawStages % 2 == 0, "K's and V's codes in turn");
  static_assert(!kE4M3 || kNB == 1, "one block of rows where the codes need room");
  static_assert(kK % 1024 == 0 && kV % 1024 == 0 && kRaw % 1024 == 0, "tiles on 1 KB");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// A block's walk along its share: the place, and what of the sequence each role needs.
struct Walk {
  DecodePlace at;
  TreeLens n;
  DecodeSpan span;
  int lo;     // the first position that any row sees behind the sinks
  int hi;     // from here on every row sees the context
  __device__ __forceinline__ int context() const { return n.len - n.drafted; }
  __device__ __forceinline__ int row() const { return decode_span_tile(span, at.tile) * kTreeTile; }
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
  return w.n.drafted > 0 && a < w.n.len && (p.window <= 0 || a < p.sinks || b > w.lo);
}
// Whether all (live) rows see all positions of [a, b).
__device__ __forceinline__ bool all_seen(const TreeParams& p, const Walk& w, int a, int b) {
  return b <= w.context() && (p.window <= 0 || b <= p.sinks || a >= w.hi);
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

// element c of the row of V at position j; what is out of range reads as 0 (the sequence's
// results are unspecified then)
template <int kType>
__device__ __forceinline__ float value_at(const TreeParams& p, int b, uint32_t head, int j, int c) {
  const int page = table_page(p.t, p.c.num_pages, b, j >> p.c.page_shift);
  if (page < 0) return 0.f;
  const uint32_t at = j & (p.c.page_size - 1);
  const uint8_t* row = p.c.v + row_offset(page, head, at, p.c.v_page, p.c.v_head, p.c.v_token);
  if constexpr (kType >= kE4M3Bf16) {
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
  constexpr bool kFp16 = kType == kF16;  // the products' operands
  constexpr bool kOutBf16 = kType == kBf16 || kType == kE4M3Bf16;
  constexpr int kParts = L::kParts;
  constexpr int kCh = L::kE4M3 ? 1 : 2;  // times 32 scores in registers at a time
  constexpr int SK = L::kKStages, SV = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const TreeParams& p = kp.p;
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);
  volatile uint32_t* abort_flag = misc + 1;
  DecodePlace* start_s = reinterpret_cast<DecodePlace*>(smem + L::kStart);
  unsigned long long* bad = reinterpret_cast<unsigned long long*>(smem + L::kBad);
  float* fin = reinterpret_cast<float*>(smem + L::kFin);
  auto bar = [&](int i) -> uint32_t { return sb + L::kBars + 8 * i; };
  auto wait = [&](int i, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait_bounded(bar(i), parity, p, abort_flag));
  };

  grid_dep_launch();
  if (sb % 1024 != 0) {  // (the swizzled tiles are laid out by address; it always is)
    if (threadIdx.x == 0) atomicOr(p.error_word, 1u);
    return;
  }

  // ---- the block's share of the line of tiles ----
  const int copies = p.c.heads * p.row_blocks;
  long long begin, share, total;
  if (p.direct) {
    const int e = blockIdx.x / copies;
    if (threadIdx.x == 0) *start_s = {e, static_cast<int>(blockIdx.x) - e * copies, 0, 0};
    begin = 0;
    share = total = tree_span(p, tree_lens(p, e)).tiles;
  } else {
    long long* sums = reinterpret_cast<long long*>(fin);
    const int each = (p.t.batch + kThreads - 1) / kThreads;
    const int lo = min(p.t.batch, static_cast<int>(threadIdx.x) * each);
    const int hi = min(p.t.batch, lo + each);
    long long mine = 0;
    for (int e = lo; e < hi; ++e) mine += tree_span(p, tree_lens(p, e)).tiles;
    long long upto = mine;  // inclusive sum over the threads
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, s);
      if (lane >= s) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += sums[w];
      total += sums[w];
    }
    total *= copies;
    share = total <= 0x7fffffff - kTreeMaxBlocks
                ? decode_share(static_cast<int>(total), gridDim.x, 1)
                : decode_share(total, static_cast<int>(gridDim.x), 1);
    begin = blockIdx.x * share;
    long long before = (upto - mine) * copies;
    if (begin >= before && begin < upto * copies) {
      for (int e = lo; e < hi; ++e) {
        const int tiles = tree_span(p, tree_lens(p, e)).tiles;
        const long long n = static_cast<long long>(tiles) * copies;
        if (begin < before + n) {
          *start_s = decode_place(e, begin - before, tiles);
          break;
        }
        before += n;
      }
    }
  }
  Join* joins = reinterpret_cast<Join*>(p.workspace);
  if (!p.direct && threadIdx.x == 0) joins[blockIdx.x].last = -1;
  if (begin >= total) return;
  const int count = static_cast<int>(min(total, begin + share) - begin);

  // ---- set-up ----
  if (threadIdx.x == kMmaWarp * 32) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(bar(i), L::arrivals(i));
    misc[1] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(sb + L::kMisc, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  Walk w;
  w.at = *start_s;
  enter(p, w);

  if (warp == kKWarp || (warp == kVWarp && !L::kE4M3)) {
    // =================== producers ===================
    // (e4m3: one for both, K and V of a tile in turn)
    constexpr int kTurns = L::kE4M3 ? 2 : 1;
    const bool k_warp = warp == kKWarp;
    const int S = L::kE4M3 ? L::kRawStages : k_warp ? SK : SV;
    const int full = L::kE4M3 ? L::bRawFull : k_warp ? L::bKFull : L::bVFull;
    const int empty = L::kE4M3 ? L::bRawEmpty : k_warp ? L::bKEmpty : L::bVEmpty;
    const uint32_t ring = sb + (L::kE4M3 ? L::kRaw : k_warp ? L::kK : L::kV);
    const int rows = min(p.c.page_size, kTreeTile);  // of a box
    const int boxes = kTreeTile / rows;              // to a tile, each of a page
    const uint32_t box_bytes = rows * (L::kE4M3 ? D : 128u);
    if (lane == 0 && k_warp) tma_prefetch_desc(&kp.tm_k);
    if (lane == 0 && (L::kE4M3 || !k_warp)) tma_prefetch_desc(&kp.tm_v);
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
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    int issued = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const int head = w.at.item / p.row_blocks;
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
#pragma unroll
      for (int turn = 0; turn < kTurns; ++turn) {
        const bool is_k = L::kE4M3 ? turn == 0 : k_warp;
        const CUtensorMap* tm = is_k ? &kp.tm_k : &kp.tm_v;
        const int c2 = head * (is_k ? kp.k_head : kp.v_head);
        const int c3 = page * (is_k ? kp.k_page : kp.v_page);
        if (!(ok = wait(empty + slot, phase ^ 1u))) break;
        if (lane == 0)
          mbar_arrive_expect_tx(bar(full + slot),
                                n * (L::kE4M3 ? box_bytes + rows : box_bytes * L::kAtoms));
        __syncwarp();
        if (mine) {
          if constexpr (L::kE4M3) {
            const uint32_t to = ring + slot * L::kRawTile;
            tma_load_4d(to + lane * box_bytes, tm, bar(full + slot), 0, place, c2, c3);
            bulk_load(sb + L::kScales + slot * kTreeTile + lane * rows,
                      (is_k ? p.c.k_scale : p.c.v_scale) + scale_offset(p.c, page, head, place),
                      rows, bar(full + slot));
          } else {
            const uint32_t to = ring + slot * L::kTile + lane * box_bytes;
#pragma unroll
            for (int x = 0; x < L::kAtoms; ++x)
              tma_load_4d(to + x * (kTreeTile * 128), tm, bar(full + slot), x * 64, place, c2, c3);
          }
        }
        ++issued;
        if (++slot == S) slot = 0, phase ^= 1u;
      }
      if (!ok) break;
      if (i + 1 < count) {
        if (decode_advance(w.at, copies)) enter(p, w);
        if (w.at.tile == 0 || w.at.tile == window + per) load_window();
      }
    }
    if (!ok) {  // every copy that was issued has to land before the block may end
      for (int x = max(0, issued - S); x < issued; ++x) wait_drain(bar(full + x % S), (x / S) & 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // =================== MMA issuer ===================
    constexpr uint32_t kFmt = kFp16 ? 0u : 1u;
    constexpr uint32_t idesc_s = idesc_f32acc<kFmt>(kTreeBlockRows, kTreeTile, false);
    constexpr uint32_t idesc_pv = idesc_f32acc<kFmt>(kTreeBlockRows, D, true);
    const uint64_t q_desc = sdesc_sw128(sb + L::kQ, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(sb + L::kK, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(sb + L::kV, kTreeTile * 128, 1024);
    int k_slot = 0, v_slot = 0, items = 0;
    uint32_t k_phase = 0, v_phase = 0, p_phase[2] = {0, 0};
    bool ok = true;
    auto issue_s = [&](int g) -> bool {
      if (kNB == 1 || g == 0) {
        if (!wait(L::bKFull + k_slot, k_phase)) return false;
      }
      tc_fence_after();
      const uint64_t kd = k_desc + static_cast<uint32_t>((k_slot * L::kTile) >> 4);
      const uint64_t qd = q_desc + static_cast<uint32_t>((kNB == 2 ? g * L::kTile : 0) >> 4);
#pragma unroll
      for (int part = 0; part < kParts; ++part)
#pragma unroll
        for (int x = 0; x < L::kAtoms; ++x)
          mma_ss_x4<false, 2>(tmem + g * kTreeTile,
                              qd + static_cast<uint32_t>((part * L::kTile) >> 4) + x * 1024,
                              kd + x * 1024, idesc_s, part + x > 0);
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
      if constexpr (kParts == 1) {
#pragma unroll
        for (int x = 0; x < kTreeTile / 64; ++x)  // 64 positions: 32 columns of P, 64 rows of V
          mma_ts_x4<false, 8, 128>(tmem + 256 + g * 128, tmem + g * kTreeTile + x * 32,
                                   vd + static_cast<uint32_t>(x * 512), idesc_pv, acc || x > 0);
      } else {
#pragma unroll
        for (int x = 0; x < kTreeTile / 16; ++x)  // 16 positions: both terms, 16 columns apart
#pragma unroll
          for (int part = 0; part < 2; ++part)
            mma_ts<false>(tmem + 256 + g * 128,
                          tmem + g * kTreeTile + x / 2 * 32 + x % 2 * 8 + part * 16,
                          vd + static_cast<uint32_t>(x * 128), idesc_pv, acc || x + part > 0);
      }
      mma_commit(bar(L::bPV + g));
      if (kNB == 1 || g == 1) {
        mma_commit(bar(L::bVEmpty + v_slot));
        if (++v_slot == SV) v_slot = 0, v_phase ^= 1u;
      }
      return true;
    };
    int i = 0;
#pragma unroll 1
    while (ok && i < count) {
      const int tiles = min(count - i, w.at.tiles - w.at.tile);
      const int units = tiles * kNB;
      if (!(ok = wait(L::bQFull, items & 1))) break;
      ++items;
      ok = issue_s(0);
      if (ok && units > 1) ok = issue_s(1);
#pragma unroll 1
      for (int u = 0; ok && u < units; ++u) {
        const int g = u & 1;
        if (!(ok = issue_pv(g, u > 1))) break;
        if (u + 2 < units) ok = issue_s(g);
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
  } else if (L::kE4M3 && warp >= kConvertWarp) {
    // =================== converters ===================
    // Half of the warps take K's tiles, half V's: 32 rows of a tile to a warp, 16 codes to a
    // lane at a time, four of those with their loads ahead of the arithmetic.
    constexpr int kC = D / 16, kEach = 4;
    const bool is_v = warp >= kConvertWarp + kConvertWarps / 2;
    const int row0 = (warp - kConvertWarp) % (kConvertWarps / 2) * 32;
    const int S = is_v ? SV : SK;
    const int full = is_v ? L::bVFull : L::bKFull, empty = is_v ? L::bVEmpty : L::bKEmpty;
    const uint32_t ring = sb + (is_v ? L::kV : L::kK);
    // Four lanes have 64 codes of a row, eight groups of them eight rows.  128-byte rows are
    // swizzled as they come; rows 5 apart (by xor) in neighbouring groups meet no bank twice,
    // neither here nor in the tile that is written.
    const int group = lane / 4;
    const int my_row = D == 64 ? group : (group / 2) ^ (group % 2 * 5);
    int raw = is_v ? 1 : 0, slot = 0;
    uint32_t raw_phase = 0, phase = 0;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const uint32_t from = sb + L::kRaw + raw * L::kRawTile;
      const uint32_t scales = sb + L::kScales + raw * kTreeTile;
      const uint32_t to = ring + slot * L::kTile;
      if (!(ok = wait(L::bRawFull + raw, raw_phase))) break;
      if (!(ok = wait(empty + slot, phase ^ 1u))) break;
#pragma unroll 1
      for (int x = 0; x < kC; x += kEach) {  // kC pieces of eight rows and 64 codes
        uint32_t in[kEach][4], e[kEach];
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
          const int row = row0 + (x + y) % 4 * 8 + my_row;
          const int c = (x + y) / 4 * 4 + lane % 4;
          const float4 v =
              ld_shared_v4(from + row * D + (D == 64 ? c : (c ^ (row & 7))) * 16);
          in[y][0] = __float_as_uint(v.x), in[y][1] = __float_as_uint(v.y);
          in[y][2] = __float_as_uint(v.z), in[y][3] = __float_as_uint(v.w);
          asm volatile("ld.shared.u8 %0, [%1];"
                       : "=r"(e[y])
                       : "r"(scales + row)
                       : "memory");
        }
        // A code's sign and seven other bits in the places of a bf16's sign, low exponent and
        // high mantissa are the value times 2^-120, subnormal codes included; one
        // multiplication by 2^(120 + e - 127) makes it right, and NaN of a row that is one.
        // Codes that are NaN and scales that bf16 has not take the slow way.
        uint32_t out[kEach][8];
        bool slow = false;
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
          uint32_t nan = 0;
          const uint32_t s2 = e[y] == 255u ? 0x7FFF7FFFu : ((e[y] + 120u) << 7) * 0x00010001u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            nan |= (in[y][k] & 0x7F7F7F7Fu) + 0x01010101u;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t w = __byte_perm(in[y][k], 0u, z ? 0x3424 : 0x1404);
              out[y][2 * k + z] = mul_bf16x2(((w >> 4) & 0x07F007F0u) | (w & 0x80008000u), s2);
            }
          }
          slow |= (nan & 0x80808080u) != 0 || (e[y] >= 135u && e[y] < 255u);
        }
        if (slow) {
#pragma unroll 1
          for (int y = 0; y < kEach; ++y) {
            const int row = row0 + (x + y) % 4 * 8 + my_row;
            const int c = (x + y) / 4 * 4 + lane % 4;
            const uint32_t line = to + (c / 4) * (kTreeTile * 128) + row * 128;
            const uint32_t codes = from + row * D + (D == 64 ? c : (c ^ (row & 7))) * 16;
            uint32_t eb;
            asm volatile("ld.shared.u8 %0, [%1];"
                         : "=r"(eb)
                         : "r"(scales + row)
                         : "memory");
            const float scale = scale_value(eb);
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {  // pairs
              uint32_t w, lo, hi;
              asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(codes + k / 2 * 4) : "memory");
              e4m3x4_to_f16(w, lo, hi);
              const float2 f = unpack16<false>(k % 2 ? hi : lo);
              const uint32_t at = line + ((2 * c + k / 4) % 8 ^ (row & 7)) * 16 + k % 4 * 4;
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(at),
                           "r"(pack16<true>(f.x * scale, f.y * scale))
                           : "memory");
            }
          }
        } else {
#pragma unroll
          for (int y = 0; y < kEach; ++y) {
            const int row = row0 + (x + y) % 4 * 8 + my_row;
            const int c = (x + y) / 4 * 4 + lane % 4;
            const uint32_t line = to + (c / 4) * (kTreeTile * 128) + row * 128;
#pragma unroll
            for (int z = 0; z < 2; ++z)
              st_shared_v4u(line + ((2 * c + z) % 8 ^ (row & 7)) * 16, out[y][4 * z],
                            out[y][4 * z + 1], out[y][4 * z + 2], out[y][4 * z + 3]);
          }
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(full + slot));
        mbar_arrive(bar(L::bRawEmpty + raw));
      }
      if ((raw += 2) >= L::kRawStages) raw -= L::kRawStages, raw_phase ^= 1u;
      if (++slot == S) slot = 0, phase ^= 1u;
    }
    __syncwarp();
  } else if (warp < kMmaWarp) {
    // =================== softmax ===================
    const int g = warp / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;  // TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_at = tmem + lanes + g * kTreeTile;
    const uint32_t o_at = tmem + lanes + 256 + g * 128;
    const int all_rows = p.tokens * p.group;
    uint32_t s_phase = 0;   // of bSFull[g] and bPV[g]: both complete once for each tile of the group
    uint32_t sync_phase = 0;
    int v_slot = 0;
    uint32_t v_phase = 0;
    auto step_v = [&]() {
      if (++v_slot == SV) v_slot = 0, v_phase ^= 1u;
    };
    // both groups are here (and what they wrote to shared memory before is seen)
    auto sync_groups = [&]() -> bool {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bSync));
      const bool ok = wait(L::bSync, sync_phase);
      sync_phase ^= 1u;
      tc_fence_after();
      return ok;
    };
    int i = 0;
    long long first_tile = begin - w.at.tile;  // of the current item, on the line
    bool ok = true;
#pragma unroll 1
    while (ok && i < count) {
      const int tiles = min(count - i, w.at.tiles - w.at.tile);
      const int head = w.at.item / p.row_blocks;
      const int row0 = (w.at.item - head * p.row_blocks) * p.item_rows;
      const int rows = min(p.item_rows, all_rows - row0);
      const int b = w.at.entry;
      // ---- Q of the item: rows of 128-byte slabs, chunks of 16 bytes permuted by the row ----
      {
        constexpr int kChunks = D / 8;
        for (int x = threadIdx.x; x < rows * kChunks; x += 2 * kGroupThreads) {
          const int row = x / kChunks, c = x % kChunks;
          const int t = (row0 + row) / p.group, h = (row0 + row) - t * p.group;
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(
                                    p.q + wide(b, p.q_batch) + wide(t, p.q_token) +
                                    wide(head * p.group + h, p.q_head)) +
                                c);
          const int rr = row % kTreeBlockRows;
          const uint32_t to = sb + L::kQ + (row / kTreeBlockRows) * L::kTile +
                              (c / 8) * (kTreeTile * 128) + rr * 128 + ((c % 8) ^ (rr & 7)) * 16;
          if constexpr (kParts == 1) {
            st_shared_v4u(to, v.x, v.y, v.z, v.w);
          } else {  // fp16 as a bf16 term and the rest: no bit is lost
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = unpack16<false>(in[k]);
              hi[k] = pack16<true>(f.x, f.y);
              const float2 h = unpack16<true>(hi[k]);
              lo[k] = pack16<true>(f.x - h.x, f.y - h.y);
            }
            st_shared_v4u(to, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4u(to + L::kTile, lo[0], lo[1], lo[2], lo[3]);
          }
        }
        if (threadIdx.x < 2) bad[threadIdx.x] = 0;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bQFull));
      }
      // ---- this thread's row ----
      const int my_row = (kNB == 2 ? g * kTreeBlockRows : 0) + r;  // within the item
      const int t = (row0 + my_row) / p.group;
      const bool live = my_row < rows && t < w.n.drafted;
      const bool warp_live = (kNB == 2 ? g * kTreeBlockRows : 0) + quarter * 32 < rows;
      const int context = w.context();
      TreeRow seen;
      seen.mask = 0;
      seen.lo = 0;
      if (live) seen = tree_row(p, w.n, b, t);
      float ref = 0.f, limit = -INFINITY, sum = 0.f;
      int mine = 0;  // tiles of this group so far in this item
      int local = 0;
#pragma unroll 1
      for (; local < tiles; ++local, ++w.at.tile) {
        if (kNB == 1 && (local & 1) != g) {
          step_v();
          continue;
        }
        const int pos0 = w.row();
        const bool whole_tile = all_seen(p, w, pos0, pos0 + kTreeTile);
        if (!(ok = wait(L::bSFull + g, s_phase))) break;
        tc_fence_after();
        if (warp_live) {
          float top = -INFINITY;
#pragma unroll 1  // (little code: what an item's end runs must not be fetched anew each time)
          for (int k = 0; k < 4; k += kCh) {
            uint32_t s[kCh][32];
#pragma unroll
            for (int y = 0; y < kCh; ++y) tmem_ld32(s_at + 32 * (k + y), s[y]);
#pragma unroll
            for (int y = 0; y < kCh; ++y) tmem_wait_ld(s[y]);
            if (!whole_tile) {  // what the row does not see becomes -inf, for the second pass too
#pragma unroll
              for (int y = 0; y < kCh; ++y) {
                const int base = pos0 + 32 * (k + y);
                uint32_t m = below(context - base);
                if (p.window > 0) m &= below(p.sinks - base) | ~below(seen.lo - base);
                const int shift = context - base;  // bit of the first drafted token
                m |= shift >= 32 || shift <= -64 ? 0u
                     : shift >= 0               ? static_cast<uint32_t>(seen.mask << shift)
                                                : static_cast<uint32_t>(seen.mask >> -shift);
                if (!live) m = 0;
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  if (!(m >> x & 1u)) s[y][x] = 0xFF800000u;
                tmem_st32(s_at + 32 * (k + y), s[y]);
              }
              tmem_wait_st();
            }
            float mx[2 * kCh];
#pragma unroll
            for (int a = 0; a < 2 * kCh; ++a) {
              const uint32_t* v = s[a / 2] + a % 2 * 16;
              mx[a] = fmax3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
#pragma unroll
              for (int x = 3; x < 15; x += 2)
                mx[a] = fmax3(mx[a], __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
              mx[a] = fmaxf(mx[a], __uint_as_float(v[15]));
            }
#pragma unroll
            for (int a = 0; a < kCh; ++a) top = fmax3(top, mx[2 * a], mx[2 * a + 1]);
          }
          const float z = top * p.scale_log2;
          const bool raise = z > limit;
          if (__any_sync(0xffffffffu, raise)) {
            float f = 1.f;
            if (raise) {
              const float to = z - kShift<kFp16>;
              if (limit != -INFINITY) f = ex2_approx(ref - to);  // (else nothing is summed yet)
              ref = to;
              limit = z + kRaise<kFp16>;
              sum *= f;
            }
            if (mine > 0) {
              // O refers to the old reference: once the last O += P V has landed
              if (!(ok = wait(L::bPV + g, s_phase ^ 1u))) break;
              tc_fence_after();
#pragma unroll 1
              for (int k = 0; k < D / 32; ++k) {
                uint32_t o[32];
                tmem_ld32(o_at + 32 * k, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                tmem_st32(o_at + 32 * k, o);
              }
            }
          }
          const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2), r2 = f2_pack(-ref, -ref);
          uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll 1
          for (int k = 0; k < 4; k += kCh) {
            uint32_t s[kCh][32];
#pragma unroll
            for (int y = 0; y < kCh; ++y) tmem_ld32(s_at + 32 * (k + y), s[y]);
#pragma unroll
            for (int y = 0; y < kCh; ++y) tmem_wait_ld(s[y]);
#pragma unroll
            for (int y = 0; y < kCh; ++y) {
              uint32_t pk[16 * kParts];
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const uint64_t z2 = f2_fma(f2_pack(__uint_as_float(s[y][2 * x]),
                                                   __uint_as_float(s[y][2 * x + 1])),
                                           c2, r2);
                float z0, z1;
                f2_unpack(z2, z0, z1);
                z0 = ex2_approx(z0);
                z1 = ex2_approx(z1);
                acc[x & 1] = f2_add(acc[x & 1], f2_pack(z0, z1));
                pk[x] = pack16<!kFp16>(z0, z1);
                if constexpr (kParts == 2) {
                  const float2 h = unpack16<true>(pk[x]);
                  pk[16 + x] = pack16<true>(z0 - h.x, z1 - h.y);
                }
              }
              if constexpr (kParts == 2)
                tmem_st32(s_at + 32 * (k + y), pk);
              else
                tmem_st16(s_at + 16 * (k + y), pk);
            }
          }
          float a0, a1;
          f2_unpack(f2_add(acc[0], acc[1]), a0, a1);
          sum += a0 + a1;
          tmem_wait_st();
        }
        if (!whole_tile) {
          // ---- V's rows that not every row sees: thread r looks after position r ----
          if (!(ok = wait(L::bVFull + v_slot, v_phase))) break;
          const int j = pos0 + r;
          if (!(j < context && (p.window <= 0 || j < p.sinks || j >= w.hi)) || w.n.drafted == 0) {
            const bool drafted = j >= context && j < w.n.len;
            const bool border = j < context && j >= w.lo;
            bool zero = w.n.drafted == 0 || !(drafted || border);
            const uint32_t line = sb + L::kV + v_slot * L::kTile + r * 128;
            // (chunks in the order of the swizzle: neighbouring rows meet no bank twice)
            auto at = [&](int c) {
              return line + c / 8 * (kTreeTile * 128) + ((c % 8) ^ (r & 7)) * 16;
            };
            uint32_t odd = 0;
            if (!zero) {
#pragma unroll 8
              for (int c = 0; c < 8 * L::kAtoms; ++c) {
                const float4 f = ld_shared_v4(at(c));
                odd |= not_finite<kFp16>(__float_as_uint(f.x)) |
                       not_finite<kFp16>(__float_as_uint(f.y));
                odd |= not_finite<kFp16>(__float_as_uint(f.z)) |
                       not_finite<kFp16>(__float_as_uint(f.w));
              }
            }
            if (odd & 0x80008000u) {
              // noted before they are gone: the other group may look at the same row
              atomicOr(&bad[drafted ? 0 : 1], 1ull << (drafted ? j - context : j - w.lo));
              __threadfence_block();
#pragma unroll 1
              for (int c = 0; c < 32 * L::kAtoms; ++c) {
                const uint32_t word = at(c / 4) + c % 4 * 4;
                uint32_t v;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(word) : "memory");
                const uint32_t n = not_finite<kFp16>(v);
                if (n & 0x8000u) v &= 0xFFFF0000u;
                if (n & 0x80000000u) v &= 0x0000FFFFu;
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(word), "r"(v) : "memory");
              }
            }
            if (zero) {
#pragma unroll 8
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
        step_v();
      }
      if (!ok) break;
      // ---- the item's end: the block's part of O ----
      if (mine > 0 && !(ok = wait(L::bPV + g, s_phase ^ 1u))) break;
      tc_fence_after();
      const bool done = w.at.tile == w.at.tiles;
      const bool whole = done && first_tile >= begin;
      const int part = decode_part(first_tile, begin);
      float f0 = 1.f, f1 = 0.f;  // of this group's O and of the other's
      float base = limit == -INFINITY ? -INFINITY : ref;
      if constexpr (kNB == 1) {
        fin[(g * 2 + 0) * kTreeBlockRows + r] = base;
        fin[(g * 2 + 1) * kTreeBlockRows + r] = sum;
        if (!(ok = sync_groups())) break;
        const float other = fin[((g ^ 1) * 2 + 0) * kTreeBlockRows + r];
        const float other_sum = fin[((g ^ 1) * 2 + 1) * kTreeBlockRows + r];
        const float m = fmaxf(base, other), to = m == -INFINITY ? 0.f : m;
        // (a NaN in the sum of a row without a finite score stays one)
        f0 = base == -INFINITY ? 1.f : ex2_approx(base - to);
        f1 = other == -INFINITY ? 1.f : ex2_approx(other - to);
        sum = sum * f0 + other_sum * f1;
        base = m;
      }
      if (!live) sum = 0.f;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float lse =
          sum == 0.f ? -INFINITY : (base == -INFINITY ? 0.f : base) + log2f(sum);
      const int h = (row0 + my_row) - t * p.group;
      const long long at =
          ((static_cast<long long>(b) * p.tokens + t) * p.c.heads + head) * p.group + h;
      const bool have0 = kNB == 2 || tiles > 0, have1 = kNB == 1 && tiles > 1;
      constexpr int kCols = kNB == 1 ? D / 2 : D;  // of this thread
      const int col0 = kNB == 1 ? g * kCols : 0;
      // the O of tile 0's group and of the other one
      const uint32_t o_first = kNB == 1 ? tmem + lanes + 256 : o_at;
      const float w0 = kNB == 1 && g == 1 ? f1 : f0, w1 = g == 1 ? f0 : f1;
      if (warp_live) {
#pragma unroll 1
        for (int k = 0; k < kCols / 32; ++k) {
          uint32_t o[32];
          tmem_ld32(o_first + col0 + 32 * k, o);
          tmem_wait_ld(o);
          float x[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = have0 ? __uint_as_float(o[c]) * w0 : 0.f;
          if (have1) {
            tmem_ld32(o_first + 128 + col0 + 32 * k, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = fmaf(__uint_as_float(o[c]), w1, x[c]);
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = sum == 0.f ? 0.f : x[c] * inv;
          if (my_row < rows) {
            if (whole) {
              uint4* out = reinterpret_cast<uint4*>(p.o + (at * D + col0 + 32 * k) * 2);
#pragma unroll
              for (int c = 0; c < 4; ++c)
                out[c] = make_uint4(pack16<kOutBf16>(x[8 * c], x[8 * c + 1]),
                                    pack16<kOutBf16>(x[8 * c + 2], x[8 * c + 3]),
                                    pack16<kOutBf16>(x[8 * c + 4], x[8 * c + 5]),
                                    pack16<kOutBf16>(x[8 * c + 6], x[8 * c + 7]));
            } else {
              float4* out = reinterpret_cast<float4*>(
                                p.workspace + rows_at(blockIdx.x, part, p.item_rows, D)) +
                            (col0 / 4 + 8 * k) * p.item_rows + my_row;
#pragma unroll
              for (int c = 0; c < 8; ++c)
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
          add_not_finite<kType, kOutBf16>(p, b, head, context, bad[0] & seen.mask, col0, kCols, out,
                                          ws);
          const int behind = seen.lo - w.lo;  // of the border positions: those that it does not see
          add_not_finite<kType, kOutBf16>(p, b, head, w.lo,
                                          behind >= 64 ? 0ull : bad[1] >> behind << behind, col0,
                                          kCols, out, ws);
        }
        if (my_row < rows && (kNB == 2 || g == 0)) {
          if (whole)
            p.lse[at] = lse * 0.69314718055994531f;
          else
            reinterpret_cast<float*>(p.workspace +
                                     lse_at(blockIdx.x, part, p.item_rows))[my_row] = lse;
        }
      }
      if (!done && first_tile >= begin && threadIdx.x == 0) {
        Join j;
        j.entry = b;
        j.item = w.at.item;
        j.last = static_cast<int>((first_tile + w.at.tiles - 1) / share);
        j.part = part;
        joins[blockIdx.x] = j;
      }
      i += tiles;
      first_tile = begin + i;
      if (i < count) {
        // O and Q are free, and nobody looks at `bad` or `fin` any more
        if (!(ok = sync_groups())) break;
        w.at.tile = w.at.tiles - 1;
        if (decode_advance(w.at, copies)) enter(p, w);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
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
  const int head = j.item / p.row_blocks;
  const int row0 = (j.item - head * p.row_blocks) * p.item_rows;
  if (row >= min(p.item_rows, p.tokens * p.group - row0)) return;
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
  const int t = (row0 + row) / p.group, h = (row0 + row) - t * p.group;
  const long long at =
      ((static_cast<long long>(j.entry) * p.tokens + t) * p.c.heads + head) * p.group + h;
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
    ready[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      L::kBytes) == cudaSuccess;
  });
  if (!ready[dev]) return -4;
  const TreeParams& p = kp.p;
  const long long items =
      static_cast<long long>(p.t.batch) * p.c.heads * p.row_blocks;
  const long long tiles =
      decode_span_most(static_cast<long long>(p.t.width) << p.c.page_shift,
                       p.window > 0 ? (p.window < (1 << 30) ? p.window : 1 << 30) + p.tokens : 0,
                       p.sinks, kTreeTile);
  long long grid = sms < kTreeMaxBlocks ? sms : kTreeMaxBlocks;
  if (tiles <= kTreeDirect && items <= grid) {
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
  const int rows = p.tokens * p.group < p.item_rows ? p.tokens * p.group : p.item_rows;
  const dim3 join(static_cast<unsigned>(grid), (rows * (D / 8) + kJoinThreads - 1) / kJoinThreads);
  return launch_kernel(join_kernel<D, kType == kBf16 || kType == kE4M3Bf16>, join, kJoinThreads, 0, stream, true, p, rows)
             ? 0
             : -4;
}

}  // namespace tree

}  // namespace fat
