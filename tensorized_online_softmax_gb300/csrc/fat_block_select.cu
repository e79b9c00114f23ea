// Scores of the blocks of a sequence, and the choice of the best ones.
#include "fat_cache.cuh"
#include "sm103_ptx.cuh"

namespace fat {

namespace {

int launched() { return cudaGetLastError() == cudaSuccess ? 0 : -4; }

__device__ __forceinline__ int blocks_of(const TableView& t, int page_shift, int b, int& len) {
  len = table_length(t, page_shift, b);
  return static_cast<int>((static_cast<long long>(len) + (1 << page_shift) - 1) >> page_shift);
}

// ---------------------------------------------------------------------------
// scores
//
// With q+ = max(q, 0) and q- = min(q, 0) the score of a block is one dot product
// of 2 d terms, [q-, q+] . [lo, hi], so the scores of 16 blocks for 8 query
// heads are m16n8k16 MMAs over the blocks' bounds, which lie in memory as the
// rows of that matrix.  Each byte of them is used once: the kernel is bound by
// memory, and loads straight into the MMA's fragments, 16 bytes a lane: the
// order of the columns within a row is free as long as both operands agree, so
// a lane takes the eight adjacent ones of its 16 bytes.
// ---------------------------------------------------------------------------
constexpr int kScoreWarps = 4;

template <bool kBf16>
__device__ __forceinline__ void score_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp takes `tiles` tiles of 16 blocks, all of one (sequence, cached head);
// the heads of the group go by eight.
template <int D, bool kBf16>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const ScoreParams p, int tiles) {
  constexpr int kChunks = 2 * D / 32;  // 32 columns of a row: one 16-byte load of four lanes
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const long long bh_count = static_cast<long long>(p.t.batch) * p.heads;
  for (long long bh = blockIdx.y; bh < bh_count; bh += gridDim.y) {
    const int b = static_cast<int>(bh / p.heads), h = static_cast<int>(bh - static_cast<long long>(b) * p.heads);
    int len;
    const int blocks = blocks_of(p.t, p.page_shift, b, len);
    const int first = (blockIdx.x * kScoreWarps + warp) * tiles * 16;
    const int end = min(first + tiles * 16, p.t.width);
    for (int head0 = 0; head0 < p.group; head0 += 8) {
      // q- and q+ of head g, as the other operand's fragments
      uint32_t qf[kChunks][4];
      if (first < blocks) {
        const bool in = head0 + g < p.group;
        const uint4* q = reinterpret_cast<const uint4*>(
            p.q + b * p.q_batch + (h * p.group + head0 + (in ? g : 0)) * p.q_head);
#pragma unroll
        for (int c = 0; c < kChunks / 2; ++c) {
          const uint4 x = in ? __ldg(q + c * 4 + t) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16<kBf16>(w[j]);  // (a NaN goes to both parts)
            qf[c][j] = pack16<kBf16>(min_nan(f.x, 0.f), min_nan(f.y, 0.f));
            qf[c + kChunks / 2][j] = pack16<kBf16>(max_nan(f.x, 0.f), max_nan(f.y, 0.f));
          }
        }
      }
      for (int i0 = first; i0 < end; i0 += 16) {
        float s[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (i0 < blocks) {
          const uint4* row[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int i = i0 + g + 8 * r;
            int page = i < blocks ? table_page(p.t, p.num_pages, b, i) : 0;
            page = max(page, 0);  // (a flagged page: its score is unspecified)
            row[r] = reinterpret_cast<const uint4*>(p.bounds) +
                     (static_cast<long long>(page) * p.heads + h) * (D / 4) + t;
          }
          float acc[2][4] = {};
#pragma unroll
          for (int c0 = 0; c0 < kChunks; c0 += 4) {
            uint4 x[4], y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              x[c] = __ldg(row[0] + (c0 + c) * 4);
              y[c] = __ldg(row[1] + (c0 + c) * 4);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t(&f)[4] = qf[c0 + c];
              score_mma<kBf16>(acc[0], x[c].x, y[c].x, x[c].y, y[c].y, f[0], f[1]);
              score_mma<kBf16>(acc[1], x[c].z, y[c].z, x[c].w, y[c].w, f[2], f[3]);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (head0 + 2 * t + (j & 1) < p.group && i0 + g + 8 * (j >> 1) < blocks)
              s[j] = acc[0][j] + acc[1][j];
        }
        float top[2] = {max_nan(s[0], s[1]), max_nan(s[2], s[3])};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = max_nan(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
          top[r] = max_nan(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
          const int i = i0 + g + 8 * r;
          if (t == 0 && i < end) {
            float* out = p.scores + bh * p.t.width + i;
            *out = head0 == 0 ? top[r] : max_nan(*out, top[r]);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// choice
//
// One block of threads per (sequence, cached head), whose warps hold adjacent
// runs of the scores, as unsigned integers of the same order, in registers.
// The num_blocks-th largest is found two bits at a time: three counts of the
// keys at or above a candidate, joined over the block with one barrier; 16
// such steps cost less than histograms, whose bins the alike leading bits of
// scores fill unevenly.  Then every warp writes its chosen ones at its place:
// all larger ones, and of those equal to the threshold the first.
// ---------------------------------------------------------------------------

// The order of the choice as unsigned integers: the newest blocks, the first
// ones, NaN, then the scores from +inf down to -inf (0x007FFFFF), and 0 where
// there is no block; -0 and +0 are equal.
__device__ __forceinline__ uint32_t select_key(float s, int i, int blocks, int first, int last) {
  if (i >= blocks) return 0u;
  if (i >= blocks - last) return 0xFFFFFFFFu;
  if (i < first) return 0xFFFFFFFEu;
  if (s != s) return 0xFFFFFFFDu;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// kKeys keys to a thread in registers; kKeys = 0: any number of blocks, read
// again in each step.
template <int kThreads, int kKeys>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ uint32_t counts[2][3][kWarps];
  __shared__ int warp_larger[kWarps], warp_equal[kWarps], newest;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  grid_dep_launch();
  const long long bh_count = static_cast<long long>(p.t.batch) * p.heads;
  for (long long bh = blockIdx.x; bh < bh_count; bh += gridDim.x) {
    const int b = static_cast<int>(bh / p.heads);
    int len;
    const int blocks = blocks_of(p.t, p.page_shift, b, len);
    const float* scores = p.scores + bh * p.t.width;
    const int take = min(p.num_blocks, blocks);
    // a warp's run of keys: rounds of 32
    const int rounds = kKeys ? kKeys : (blocks + kThreads - 1) / kThreads;
    const int base = warp * rounds * 32 + lane;
    uint32_t held[kKeys ? kKeys : 1];
    if constexpr (kKeys > 0) {
      float s[kKeys];
#pragma unroll
      for (int r = 0; r < kKeys; ++r)
        s[r] = base + r * 32 < blocks ? __ldg(scores + base + r * 32) : 0.f;
#pragma unroll
      for (int r = 0; r < kKeys; ++r)
        held[r] = select_key(s[r], base + r * 32, blocks, p.first_blocks, p.last_blocks);
    }
    auto key = [&](int r) {
      if constexpr (kKeys > 0) {
        return held[r];
      } else {
        const int i = base + r * 32;
        return select_key(i < blocks ? __ldg(scores + i) : 0.f, i, blocks, p.first_blocks,
                          p.last_blocks);
      }
    };
    uint32_t threshold = 0;  // the take-th largest key; all blocks are above 0
    if (take < blocks) {
      for (int shift = 30, odd = 0; shift >= 0; shift -= 2, odd ^= 1) {
        uint32_t n[3] = {0, 0, 0};
#pragma unroll
        for (int r = 0; r < (kKeys ? kKeys : rounds); ++r) {
          const uint32_t k = key(r);
#pragma unroll
          for (int j = 0; j < 3; ++j) n[j] += k >= (threshold | ((j + 1u) << shift));
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          n[j] = __reduce_add_sync(0xffffffffu, n[j]);
          if (lane == 0) counts[odd][j][warp] = n[j];
        }
        __syncthreads();  // (the other half is free: all have passed the barrier before)
        uint32_t digit = 0;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const uint32_t all =
              __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[odd][j][lane] : 0u);
          digit += all >= static_cast<uint32_t>(take);  // (the counts fall with j)
        }
        threshold |= digit << shift;
      }
    }
    // how many of each kind the warp holds
    int larger = 0, equal = 0;
#pragma unroll
    for (int r = 0; r < (kKeys ? kKeys : rounds); ++r) {
      const uint32_t k = key(r);
      larger += k > threshold;
      equal += k == threshold;
    }
    larger = __reduce_add_sync(0xffffffffu, larger);
    equal = threshold ? __reduce_add_sync(0xffffffffu, equal) : 0;
    if (lane == 0) {
      warp_larger[warp] = larger;
      warp_equal[warp] = equal;
    }
    if (threadIdx.x == 0) newest = 0;
    __syncthreads();
    // places: those of earlier warps, and of the equal ones at most `room`
    const int all_larger = __reduce_add_sync(0xffffffffu, lane < kWarps ? warp_larger[lane] : 0);
    const int before_larger = __reduce_add_sync(0xffffffffu, lane < warp ? warp_larger[lane] : 0);
    int equal_rank = __reduce_add_sync(0xffffffffu, lane < warp ? warp_equal[lane] : 0);
    const int room = take - all_larger;
    int at = before_larger + min(equal_rank, room);
    int* out = p.blocks + bh * p.num_blocks;
    int* pages = p.pages + bh * p.list;
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int r = 0; r < (kKeys ? kKeys : rounds); ++r) {
      const uint32_t k = key(r);
      const bool same = threshold != 0 && k == threshold;
      const uint32_t same_mask = __ballot_sync(0xffffffffu, same);
      const bool chosen =
          k > threshold || (same && equal_rank + __popc(same_mask & below) < room);
      const uint32_t mask = __ballot_sync(0xffffffffu, chosen);
      if (chosen) {
        const int i = base + r * 32, place = at + __popc(mask & below);
        out[place] = i;
        pages[place] = __ldg(p.t.pages + b * p.t.stride + i);
        if (i == blocks - 1) newest = 1;
      }
      equal_rank += __popc(same_mask);
      at += __popc(mask);
    }
    for (int i = take + threadIdx.x; i < p.num_blocks; i += kThreads) out[i] = -1;
    __syncthreads();
    if (threadIdx.x == 0) {
      // only the newest block can be partly filled, and it is the last chosen one if at all
      int n = len;
      if (take < blocks) {
        n = take << p.page_shift;
        if (newest) n -= (1 << p.page_shift) - (len - ((blocks - 1) << p.page_shift));
      }
      p.lens[bh] = n;
    }
    __syncthreads();
  }
}

template <int kThreads, int kKeys>
int run_select(const SelectParams& p, cudaStream_t stream) {
  const long long bh = static_cast<long long>(p.t.batch) * p.heads;
  const unsigned grid = static_cast<unsigned>(bh < (1 << 30) ? bh : (1 << 30));
  select_kernel<kThreads, kKeys><<<grid, kThreads, 0, stream>>>(p);
  return launched();
}

}  // namespace

int launch_kv_scores(const ScoreParams& p, int d, bool bf16, int sms, cudaStream_t stream) {
  const long long bh = static_cast<long long>(p.t.batch) * p.heads;
  // tiles to a warp: as many as leave 16 warps for each SM (q is loaded once for them), 8 at most
  const int row_tiles = (p.t.width + 15) / 16;
  long long tiles = bh * row_tiles / (16ll * sms);
  tiles = tiles < 1 ? 1 : tiles > 8 ? 8 : tiles;
  const long long per_block = tiles * kScoreWarps;
  const dim3 grid(static_cast<unsigned>((row_tiles + per_block - 1) / per_block),
                  static_cast<unsigned>(bh < 65535 ? bh : 65535));
  const int n = static_cast<int>(tiles);
  if (d == 128)
    bf16 ? score_kernel<128, true><<<grid, 32 * kScoreWarps, 0, stream>>>(p, n)
         : score_kernel<128, false><<<grid, 32 * kScoreWarps, 0, stream>>>(p, n);
  else
    bf16 ? score_kernel<64, true><<<grid, 32 * kScoreWarps, 0, stream>>>(p, n)
         : score_kernel<64, false><<<grid, 32 * kScoreWarps, 0, stream>>>(p, n);
  return launched();
}

int launch_select(const SelectParams& p, cudaStream_t stream) {
  if (p.t.width <= 1024) return run_select<256, 4>(p, stream);
  if (p.t.width <= 8192) return run_select<1024, 8>(p, stream);
  if (p.t.width <= 32768) return run_select<1024, 32>(p, stream);
  return run_select<1024, 0>(p, stream);
}

}  // namespace fat
