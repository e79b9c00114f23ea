// Scores of the blocks of a sequence, and the choice of the best ones.
#include "fat_cache.cuh"
#include "sm103_ptx.cuh"

namespace fat {

namespace {

int launched() { return cudaGetLastError() == cudaSuccess ? 0 : -4; }

__device__ __forceinline__ int blocks_of(const TableView& t, int page_shift, int b, int& len) {
  len = table_length(t, page_shift, b);
  return (len + (1 << page_shift) - 1) >> page_shift;
}

// ---------------------------------------------------------------------------
// scores
//
// With q+ = max(q, 0) and q- = min(q, 0) the score of a block is one dot product
// of 2 d terms, [q-, q+] . [lo, hi], so the scores of 16 blocks for 8 query
// heads are m16n8k16 MMAs over the blocks' bounds, which lie in memory as the
// rows of that matrix.  Each byte of them is used once: the kernel is bound by
// memory.  A warp keeps a ring of tiles of 16 blocks in shared memory, filled by
// asynchronous copies, and reads 16 bytes a lane from it as the MMA's fragment:
// the order of the columns within a row is free as long as both operands agree,
// so a lane takes the eight adjacent ones of its 16 bytes.
// ---------------------------------------------------------------------------
// (With two stages and twelve warps to an SM, 207 MB of bounds, 16 sequences of up to 4096
// blocks and 8 heads, take 36 us, 0.85 of the measured copy rate; with three and eight 39.)
constexpr int kScoreWarps = 4, kScoreStages = 2;

template <int D>
struct ScoreLayout {
  static constexpr int kRow = 4 * D;            // bytes of a block's bounds
  static constexpr int kCopies = kRow / 16;     // 16-byte pieces of a row: 32 or 16
  static constexpr int kStage = 16 * kRow;      // a tile
  static constexpr int kSmem = kScoreWarps * kScoreStages * kStage;
};

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

// Where 16-byte piece c of row r of a tile goes: the halves of a 128-byte line
// change places in odd rows, so that the eight lanes that are served together
// (four adjacent pieces of two rows) meet no bank twice.
__device__ __forceinline__ uint32_t score_piece(int row_bytes, int r, int c) {
  return static_cast<uint32_t>(r * row_bytes + ((c ^ ((r & 1) << 2)) << 4));
}

// A warp takes `tiles` tiles of 16 blocks, all of one (sequence, cached head);
// the heads of the group go by eight.
template <int D, bool kBf16>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const ScoreParams p, int tiles) {
  using L = ScoreLayout<D>;
  constexpr int kChunks = 2 * D / 32;  // 32 columns of a row: 16 bytes of four lanes
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const uint32_t ring = smem_u32(smem) + warp * kScoreStages * L::kStage;
  const long long bh_count = static_cast<long long>(p.t.batch) * p.heads;
  for (long long bh = blockIdx.y; bh < bh_count; bh += gridDim.y) {
    const int b = static_cast<int>(bh / p.heads);
    const int h = static_cast<int>(bh - static_cast<long long>(b) * p.heads);
    const int first = (blockIdx.x * kScoreWarps + warp) * tiles * 16;
    const int end = min(first + tiles * 16, p.t.width);
    const int* table = p.t.pages + b * p.t.stride;
    // the first pages are loaded together with the length, which says later which of them count
    const int early[2] = {first + lane < end ? table[first + lane] : -1,
                          first + 32 + lane < end ? table[first + 32 + lane] : -1};
    int len;
    const int blocks = blocks_of(p.t, p.page_shift, b, len), stop = min(end, blocks);
    for (int head0 = 0; head0 < p.group; head0 += 8) {
      // the pages of 32 blocks (two tiles), one to a lane, a step ahead; -1 where there is none
      auto usable = [&](int entry, int i) {
        if (i >= stop) return -1;
        if (static_cast<uint32_t>(entry) < p.num_pages) return entry;
        atomicOr(p.t.error_word, kErrIndex);
        return -1;
      };
      auto pages_at = [&](int i0) {
        const int i = i0 + lane;
        return i < stop ? usable(table[i], i) : -1;
      };
      int page = usable(early[0], first + lane), page_next = usable(early[1], first + 32 + lane);
      int loaded = first;
      uint32_t stage_in = ring, stage_out = ring;
      auto issue = [&]() {
        if (loaded < stop) {
          // (a row without a page, behind the end or flagged, is filled with zeros)
          constexpr int kRows = 32 / L::kCopies;  // that one copy of the warp covers
          const int mine = lane / L::kCopies, c = lane % L::kCopies;
#pragma unroll
          for (int r0 = 0; r0 < 16; r0 += kRows) {
            const int r = r0 + mine;
            const int pg = __shfl_sync(0xffffffffu, page, ((loaded - first) & 16) + r);
            const uint8_t* from =
                p.bounds + (wide(max(pg, 0), p.heads) + h) * L::kRow + c * 16;
            const uint32_t bytes = pg >= 0 ? 16u : 0u;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             stage_in + score_piece(L::kRow, r, c)),
                         "l"(from), "r"(bytes)
                         : "memory");
          }
          if ((loaded - first) & 16) {
            page = page_next;
            page_next = pages_at(loaded + 48);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        loaded += 16;
        stage_in += L::kStage;
        if (stage_in == ring + kScoreStages * L::kStage) stage_in = ring;
      };
#pragma unroll 1
      for (int i = 0; i < kScoreStages - 1; ++i) issue();
      // q- and q+ of head g, as the other operand's fragments
      uint32_t qf[kChunks][4];
      if (first < stop) {
        const bool in = head0 + g < p.group;
        const uint4* q = reinterpret_cast<const uint4*>(
            p.q + wide(b, p.q_batch) + wide(h * p.group + head0 + (in ? g : 0), p.q_head));
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
#pragma unroll 1
      for (int i0 = first; i0 < end; i0 += 16) {
        float s[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (i0 < stop) {
          issue();
          asm volatile("cp.async.wait_group %0;" ::"n"(kScoreStages - 1) : "memory");
          __syncwarp();
          float acc[2][4] = {};
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t x[4], y[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"(stage_out + score_piece(L::kRow, g, 4 * c + t))
                         : "memory");
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                         : "r"(stage_out + score_piece(L::kRow, g + 8, 4 * c + t))
                         : "memory");
            const uint32_t(&f)[4] = qf[c];
            score_mma<kBf16>(acc[0], x[0], y[0], x[1], y[1], f[0], f[1]);
            score_mma<kBf16>(acc[1], x[2], y[2], x[3], y[3], f[2], f[3]);
          }
          __syncwarp();  // the stage may be filled again
          stage_out += L::kStage;
          if (stage_out == ring + kScoreStages * L::kStage) stage_out = ring;
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
// The num_blocks-th largest of 1025 to 8192 keys is found in two steps: a
// histogram of the leading 11 bits (four copies, as scores share leading bits and
// lanes would queue for one bin) gives the bin that it is in, and a warp finds the
// other bits among the keys of that bin, two at a time, by counting.  Then every
// warp writes its chosen ones at its place: all larger ones, and of those equal to
// the threshold the first.
//
// Up to 1024 blocks, and over 8192, all keys take part in the counting, two bits
// at a time (over 32768 they are read again in each step).
//
// It is a chain of latencies, hidden behind nothing: 512 blocks of 128 (sequence,
// head) pairs 4.4 us, 8192 blocks of 8 pairs 6.2 us.
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

constexpr int kSelectBinned = 8192;

// kKeys keys to a thread in registers; kKeys = 0: any number of blocks, read
// again in each step.
template <int kThreads, int kKeys>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr bool kBins = kKeys > 0 && kThreads == 1024 && kThreads * kKeys <= kSelectBinned;
  constexpr int kBits = 11, kCopies = 4;
  // the histogram, then the keys of one bin
  constexpr int kBinWords = kCopies << kBits, kKeyWords = kThreads * kKeys;
  __shared__ __align__(16) uint32_t
      bins[!kBins ? 1 : kBinWords > kKeyWords ? kBinWords : kKeyWords];
  __shared__ uint32_t counts[2][3][kWarps];
  __shared__ uint32_t found[2], listed;  // the bin and how many of its keys are taken
  __shared__ int warp_larger[kWarps], warp_equal[kWarps], newest;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  grid_dep_launch();
  const long long bh_count = static_cast<long long>(p.t.batch) * p.heads;
  for (long long bh = blockIdx.x; bh < bh_count; bh += gridDim.x) {
    const int b = static_cast<int>(bh / p.heads);
    const float* scores = p.scores + bh * p.t.width;
    const int* table = p.t.pages + b * p.t.stride;
    // scores and pages are loaded with the length, not behind it (the pages where registers allow)
    constexpr bool kPagesEarly = kKeys > 0 && kKeys <= 8;
    float s[kKeys ? kKeys : 1];
    int page[kKeys ? kKeys : 1];
    if constexpr (kKeys > 0) {
#pragma unroll
      for (int r = 0; r < kKeys; ++r) {
        const int i = (warp * kKeys + r) * 32 + lane;
        s[r] = i < p.t.width ? __ldg(scores + i) : 0.f;
        if constexpr (kPagesEarly) page[r] = i < p.t.width ? __ldg(table + i) : 0;
      }
    }
    int len;
    const int blocks = blocks_of(p.t, p.page_shift, b, len);
    const int take = min(p.num_blocks, blocks);
    // a warp's run of keys: rounds of 32
    const int rounds = kKeys ? kKeys : (blocks + kThreads - 1) / kThreads;
    const int base = warp * rounds * 32 + lane;
    uint32_t held[kKeys ? kKeys : 1];
    if constexpr (kKeys > 0) {
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
    if constexpr (kBins) {
      if (take < blocks) {
        for (int i = threadIdx.x; i < (kCopies << kBits) / 4; i += kThreads)
          reinterpret_cast<uint4*>(bins)[i] = make_uint4(0, 0, 0, 0);
        if (threadIdx.x == 0) listed = 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kKeys; ++r)
          if (held[r]) atomicAdd(&bins[(held[r] >> (32 - kBits)) * kCopies + lane % kCopies], 1u);
        __syncthreads();
        // a thread's bins, from the top
        constexpr int kEach = (1 << kBits) / kThreads;
        uint32_t n[kEach], mine = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const int bin = (1 << kBits) - 1 - (threadIdx.x * kEach + j);
          const uint4 c = reinterpret_cast<const uint4*>(bins)[bin];
          n[j] = c.x + c.y + c.z + c.w;
          mine += n[j];
        }
        uint32_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += v;
        }
        if (lane == 31) counts[0][0][warp] = upto;
        __syncthreads();
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? counts[0][0][lane] : 0u);
        const uint32_t want = take;
        if (upto - mine < want && want <= upto) {
          uint32_t above = upto - mine;
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            if (above < want && want <= above + n[j]) {
              found[0] = (1 << kBits) - 1 - (threadIdx.x * kEach + j);
              found[1] = want - above;
            }
            above += n[j];
          }
        }
        __syncthreads();  // (also: nobody reads the histogram any more)
        const uint32_t bin = found[0];
#pragma unroll
        for (int r = 0; r < kKeys; ++r) {
          const bool in = held[r] >> (32 - kBits) == bin && held[r] != 0;
          const uint32_t mask = __ballot_sync(0xffffffffu, in);
          if (mask) {
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(&listed, __popc(mask));
            at = __shfl_sync(0xffffffffu, at, 0);
            if (in) bins[at + __popc(mask & ((1u << lane) - 1u))] = held[r];
          }
        }
        __syncthreads();
        if (warp == 0) {
          const uint32_t m = listed, rest = found[1];
          uint32_t lowest = 0xFFFFFFFFu, highest = 0;
          for (uint32_t i = lane; i < m; i += 32) {
            lowest = min(lowest, bins[i]);
            highest = max(highest, bins[i]);
          }
          lowest = __reduce_min_sync(0xffffffffu, lowest);
          highest = __reduce_max_sync(0xffffffffu, highest);
          uint32_t value = lowest;
          if (lowest != highest && m > rest) {
            // bits that all keys of the bin share need no counting
            int shift = (31 - __clz(lowest ^ highest)) & ~1;
            value = shift == 30 ? 0u : lowest >> (shift + 2) << (shift + 2);
            for (; shift >= 0; shift -= 2) {
              uint32_t c[3] = {0, 0, 0};
              for (uint32_t i = lane; i < m; i += 32) {
                const uint32_t k = bins[i];
#pragma unroll
                for (int j = 0; j < 3; ++j) c[j] += k >= (value | ((j + 1u) << shift));
              }
              uint32_t digit = 0;
              bool exact = false;
#pragma unroll
              for (int j = 0; j < 3; ++j) {
                const uint32_t all = __reduce_add_sync(0xffffffffu, c[j]);
                digit += all >= rest;
                exact |= all == rest;
              }
              value |= digit << shift;
              if (exact) break;
            }
          }
          if (lane == 0) found[0] = value;
        }
        __syncthreads();
        threshold = found[0];
      }
    } else if (take < blocks) {
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
        bool exact = false;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const uint32_t all =
              __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[odd][j][lane] : 0u);
          digit += all >= static_cast<uint32_t>(take);  // (the counts fall with j)
          exact |= all == static_cast<uint32_t>(take);
        }
        threshold |= digit << shift;
        if (exact) break;  // just the wanted number is at or above it (the same in all threads)
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
    if constexpr (kKeys > 0 && !kPagesEarly) {  // (together: one latency, not one a round)
#pragma unroll
      for (int r = 0; r < kKeys; ++r)
        page[r] = base + r * 32 < blocks ? __ldg(table + base + r * 32) : 0;
    }
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
        pages[place] = kKeys ? page[kKeys ? r : 0] : __ldg(table + i);
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

template <int D, bool kBf16>
static int run_scores(const ScoreParams& p, int dev, int sms, cudaStream_t stream) {
  using L = ScoreLayout<D>;
  static std::once_flag once[kMaxDevices];
  static bool ready[kMaxDevices];
  std::call_once(once[dev], [&] {
    ready[dev] = cudaFuncSetAttribute(score_kernel<D, kBf16>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      L::kSmem) == cudaSuccess;
  });
  if (!ready[dev]) return -4;
  const long long bh = static_cast<long long>(p.t.batch) * p.heads;
  // tiles to a warp: as many as leave twelve warps for each SM (the ring fills and q is loaded
  // once for them), 16 at most
  const int row_tiles = p.t.width / 16 + (p.t.width % 16 != 0);
  long long tiles = bh * row_tiles / (12ll * sms);
  tiles = tiles < 1 ? 1 : tiles > 16 ? 16 : tiles;
  const long long per_block = tiles * kScoreWarps;
  const dim3 grid(static_cast<unsigned>((row_tiles + per_block - 1) / per_block),
                  static_cast<unsigned>(bh < 65535 ? bh : 65535));
  score_kernel<D, kBf16><<<grid, 32 * kScoreWarps, L::kSmem, stream>>>(p, static_cast<int>(tiles));
  return launched();
}

int launch_kv_scores(const ScoreParams& p, int d, bool bf16, int dev, int sms,
                     cudaStream_t stream) {
  if (d == 128)
    return bf16 ? run_scores<128, true>(p, dev, sms, stream)
                : run_scores<128, false>(p, dev, sms, stream);
  return bf16 ? run_scores<64, true>(p, dev, sms, stream)
              : run_scores<64, false>(p, dev, sms, stream);
}

int launch_select(const SelectParams& p, cudaStream_t stream) {
  if (p.t.width <= 1024) return run_select<256, 4>(p, stream);
  if (p.t.width <= 8192) return run_select<1024, 8>(p, stream);
  if (p.t.width <= 32768) return run_select<1024, 32>(p, stream);
  return run_select<1024, 0>(p, stream);
}

}  // namespace fat
