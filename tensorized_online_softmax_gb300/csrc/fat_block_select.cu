// Scores of the blocks of a sequence, and the choice of the best ones.
#include "fat_cache.cuh"

namespace fat {

namespace {

// ---------------------------------------------------------------------------
// scores: one warp per (sequence, cached head, block)
// ---------------------------------------------------------------------------
template <int D, bool kBf16>
__global__ void __launch_bounds__(128) score_kernel(const ScoreParams p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long bh_count = static_cast<long long>(p.t.batch) * p.heads;
  for (long long bh = blockIdx.y; bh < bh_count; bh += gridDim.y) {
    const int b = static_cast<int>(bh / p.heads), h = static_cast<int>(bh % p.heads);
    const int len = table_length(p.t, p.page_shift, b);
    const int blocks = static_cast<int>((static_cast<long long>(len) + (1 << p.page_shift) - 1) >> p.page_shift);
    const int i = blockIdx.x * 4 + warp;
    if (i >= p.t.width) continue;
    float best = -INFINITY;
    const long long page = i < blocks ? table_page(p.t, p.num_pages, b, i) : -1;
    if (page >= 0) {
      const uint16_t* lo = reinterpret_cast<const uint16_t*>(p.bounds) + (page * p.heads + h) * 2 * D;
      for (int g = 0; g < p.group; ++g) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q + b * p.q_batch + (h * p.group + g) * p.q_head);
        float s = 0.f;
#pragma unroll
        for (int c = lane; c < D; c += 32) {
          const float x = unpack16<kBf16>(q[c]).x;
          s = fmaf(fmaxf(x, 0.f), unpack16<kBf16>(lo[D + c]).x, s);
          s = fmaf(fminf(x, 0.f), unpack16<kBf16>(lo[c]).x, s);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        best = g == 0 ? s : max_nan(best, s);
      }
    }
    if (lane == 0) p.scores[bh * p.t.width + i] = best;
  }
}

// ---------------------------------------------------------------------------
// choice: one block of threads per (sequence, cached head)
// ---------------------------------------------------------------------------
constexpr int kSelectThreads = 512;

// The order of the choice as unsigned integers: the newest blocks, the first
// ones, NaN, then the scores from +inf down; -0 and +0 are equal.
__device__ __forceinline__ uint32_t select_key(float s, int i, int blocks, int first, int last) {
  if (i >= blocks - last) return 0xFFFFFFFFu;
  if (i < first) return 0xFFFFFFFEu;
  if (s != s) return 0xFFFFFFFDu;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of one count per thread, and the total.
__device__ __forceinline__ int block_prefix(int x, int* warp_sums, int& total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();  // the last use of warp_sums is over
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kSelectThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return before + s - x;
}

// The k-th largest key is found byte by byte from the top (a histogram of the
// keys that agree with the bytes found so far); a last pass over the blocks in
// order takes all larger keys and, of the equal ones, the first.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p) {
  __shared__ int hist[256], warp_sums[kSelectThreads / 32], found[2], newest;
  const long long bh_count = static_cast<long long>(p.t.batch) * p.heads;
  for (long long bh = blockIdx.x; bh < bh_count; bh += gridDim.x) {
    const int b = static_cast<int>(bh / p.heads);
    const int len = table_length(p.t, p.page_shift, b);
    const int size = 1 << p.page_shift;
    const int blocks = static_cast<int>((static_cast<long long>(len) + size - 1) >> p.page_shift);
    const float* scores = p.scores + bh * p.t.width;
    const int take = min(p.num_blocks, blocks);
    uint32_t threshold = 0;
    int equal = take;  // how many keys equal to the threshold are taken
    if (take < blocks) {
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < blocks; i += kSelectThreads) {
          const uint32_t key = select_key(scores[i], i, blocks, p.first_blocks, p.last_blocks);
          if (shift == 24 || (key >> (shift + 8)) == (threshold >> (shift + 8)))
            atomicAdd(&hist[(key >> shift) & 255u], 1);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
          int left = equal, bin = 255;
          while (hist[bin] < left) left -= hist[bin--];
          found[0] = bin;
          found[1] = left;
        }
        __syncthreads();
        threshold |= static_cast<uint32_t>(found[0]) << shift;
        equal = found[1];
        __syncthreads();
      }
    }
    int done = 0, taken_equal = 0;  // over the blocks of earlier rounds
    if (threadIdx.x == 0) newest = 0;  // (the rounds' barriers order this)
    int* out = p.blocks + bh * p.num_blocks;
    int* pages = p.pages + bh * p.list;
    for (int base = 0; base < blocks; base += kSelectThreads) {
      const int i = base + threadIdx.x;
      uint32_t key = 0;
      bool larger = false, same = false;
      if (i < blocks) {
        if (take == blocks) {
          larger = true;
        } else {
          key = select_key(scores[i], i, blocks, p.first_blocks, p.last_blocks);
          larger = key > threshold;
          same = key == threshold;
        }
      }
      int total_same, total;
      const int rank = block_prefix(same, warp_sums, total_same);
      const bool chosen = larger || (same && taken_equal + rank < equal);
      const int at = done + block_prefix(chosen, warp_sums, total);
      if (chosen) {
        out[at] = i;
        pages[at] = __ldg(p.t.pages + b * p.t.stride + i);
        if (i == blocks - 1) newest = 1;
      }
      taken_equal += total_same;
      done += total;
    }
    for (int i = take + threadIdx.x; i < p.num_blocks; i += kSelectThreads) out[i] = -1;
    __syncthreads();
    if (threadIdx.x == 0) {
      // only the newest block can be partly filled, and it is the last chosen one if at all
      int n = len;
      if (take < blocks) {
        n = take << p.page_shift;
        if (newest) n -= size - (len - ((blocks - 1) << p.page_shift));
      }
      p.lens[bh] = n;
    }
    __syncthreads();
  }
}

}  // namespace

int launch_kv_scores(const ScoreParams& p, int d, bool bf16, cudaStream_t stream) {
  const long long bh = static_cast<long long>(p.t.batch) * p.heads;
  const dim3 grid((p.t.width + 3) / 4, static_cast<unsigned>(bh < 65535 ? bh : 65535));
  if (d == 128)
    bf16 ? score_kernel<128, true><<<grid, 128, 0, stream>>>(p)
         : score_kernel<128, false><<<grid, 128, 0, stream>>>(p);
  else
    bf16 ? score_kernel<64, true><<<grid, 128, 0, stream>>>(p)
         : score_kernel<64, false><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

int launch_select(const SelectParams& p, cudaStream_t stream) {
  const long long bh = static_cast<long long>(p.t.batch) * p.heads;
  const unsigned grid = static_cast<unsigned>(bh < (1 << 30) ? bh : (1 << 30));
  select_kernel<<<grid, kSelectThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace fat
