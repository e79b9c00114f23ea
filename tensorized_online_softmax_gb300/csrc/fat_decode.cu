// Attention of one query token per sequence over the paged cache.
//
// One block per query head; its four warps take positions in turn, each with
// its own running maximum m (in units of log2) and sum l:
//     m' = max(m, z_j),  l' = l 2^(m - m') + 2^(z_j - m'),
//     O' = O 2^(m - m') + 2^(z_j - m') V_j,
// and are joined at the end by their weights 2^(m_w - max m).
#include "fat_cache.cuh"

namespace fat {

namespace {

template <int D, bool kE4M3, bool kBf16>
__global__ void __launch_bounds__(128) decode_kernel(const DecodeParams p) {
  constexpr int kPer = D / 32;  // elements per lane
  __shared__ float o_s[4][D], m_s[4], l_s[4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int q_heads = p.c.heads * p.group;
  const long long rows = static_cast<long long>(p.batch) * q_heads;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const int b = static_cast<int>(row / q_heads), hq = static_cast<int>(row % q_heads);
    const int h = hq / p.group;
    const int e = p.per_head ? b * p.c.heads + h : b;
    const int len = table_length(p.t, p.c.page_shift, e);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q + b * p.q_batch + hq * p.q_head);
    float qf[kPer], o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      qf[i] = unpack16<kBf16>(q[lane + 32 * i]).x;
      o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = warp; j < len; j += 4) {
      const long long page = table_page(p.t, p.c.num_pages, e, j >> p.c.page_shift);
      if (page < 0) continue;
      const int place = j & (p.c.page_size - 1);
      const uint8_t* k = p.c.k + page * p.c.k_page + h * p.c.k_head + place * p.c.k_token;
      const uint8_t* v = p.c.v + page * p.c.v_page + h * p.c.v_head + place * p.c.v_token;
      const long long at = (page * p.c.heads + h) * p.c.page_size + place;
      auto value = [&](const uint8_t* r, const uint8_t* scale, int i) {
        if constexpr (kE4M3)
          return unpack16<false>(e4m3x2_to_f16x2(r[i])).x * scale_value(scale[at]);
        else
          return unpack16<kBf16>(reinterpret_cast<const uint16_t*>(r)[i]).x;
      };
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        s = fmaf(qf[i], value(k, p.c.k_scale, lane + 32 * i), s);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.scale_log2;
      const float m_new = fmaxf(m, s);  // (a NaN score leaves it and makes its weight NaN)
      const float base = m_new == -INFINITY ? 0.f : m_new;
      const float f = exp2f(m - base), w = exp2f(s - base);
      m = m_new;
      l = fmaf(l, f, w);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        o[i] = fmaf(o[i], f, w * value(v, p.c.v_scale, lane + 32 * i));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) o_s[warp][lane + 32 * i] = o[i];
    if (lane == 0) m_s[warp] = m, l_s[warp] = l;
    __syncthreads();
    if (threadIdx.x < D) {
      float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, m_s[w]);
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = exp2f(m_s[w] - base);
        sum = fmaf(l_s[w], f, sum);
        acc = fmaf(o_s[w][threadIdx.x], f, acc);
      }
      const float out = sum == 0.f ? 0.f : acc / sum;
      reinterpret_cast<uint16_t*>(p.o)[row * D + threadIdx.x] =
          static_cast<uint16_t>(pack16<kBf16>(out, 0.f));
      if (threadIdx.x == 0)
        p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

}  // namespace

size_t decode_workspace_bytes(int d) { return 16; }

int launch_decode(const DecodeParams& p, int d, bool e4m3, bool bf16, int dev,
                  cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.batch) * p.c.heads * p.group;
  const unsigned grid = static_cast<unsigned>(rows < (1 << 30) ? rows : (1 << 30));
#define FAT_RUN(D, E, B) decode_kernel<D, E, B><<<grid, 128, 0, stream>>>(p)
  FAT_PICK(d, e4m3, bf16, FAT_RUN);
#undef FAT_RUN
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace fat
