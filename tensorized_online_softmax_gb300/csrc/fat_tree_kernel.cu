// Attention of drafted tokens over the paged cache: a block to each (sequence,
// drafted token, query head), whose warps take every fourth position.
#include "fat_tree.cuh"

namespace fat {

namespace {

constexpr int kWarps = 4;

template <int D, bool kE4M3, bool kBf16>
__global__ void __launch_bounds__(32 * kWarps) tree_kernel(const TreeParams p) {
  constexpr int kPer = D / 32;
  __shared__ float top_s[kWarps], sum_s[kWarps], o_s[kWarps][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int q_heads = p.group * p.c.heads;
  const int qh = blockIdx.x, t = blockIdx.y;
  const uint32_t h = qh / p.group;
  for (int b = blockIdx.z; b < p.t.batch; b += gridDim.z) {
    const TreeLens n = tree_lens(p, b);
    const int context = n.len - n.drafted;
    float top = -INFINITY, sum = 0.f, o[kPer] = {};
    if (t < n.drafted) {
      const TreeRow row = tree_row(p, n, b, t);
      float q[kPer];
      const uint16_t* qp = reinterpret_cast<const uint16_t*>(
          p.q + wide(b, p.q_batch) + wide(t, p.q_token) + wide(qh, p.q_head));
#pragma unroll
      for (int i = 0; i < kPer; ++i) q[i] = unpack16<kBf16>(qp[lane + 32 * i]).x;
      for (int j = warp; j < n.len; j += kWarps) {
        const bool seen = j >= context ? (row.mask >> (j - context) & 1) != 0
                                       : p.window <= 0 || j < p.sinks || j >= row.lo;
        if (!seen) continue;
        const int page = table_page(p.t, p.c.num_pages, b, j >> p.c.page_shift);
        if (page < 0) continue;
        const uint32_t at = j & (p.c.page_size - 1);
        const uint8_t* kr = p.c.k + row_offset(page, h, at, p.c.k_page, p.c.k_head, p.c.k_token);
        const uint8_t* vr = p.c.v + row_offset(page, h, at, p.c.v_page, p.c.v_head, p.c.v_token);
        float k[kPer], v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int c = lane + 32 * i;
          if constexpr (kE4M3) {
            uint32_t lo, hi;
            e4m3x4_to_f16(kr[c] | static_cast<uint32_t>(vr[c]) << 8, lo, hi);
            const float2 f = unpack16<false>(lo);
            const unsigned long long s = scale_offset(p.c, page, h, at);
            k[i] = f.x * scale_value(p.c.k_scale[s]);
            v[i] = f.y * scale_value(p.c.v_scale[s]);
          } else {
            k[i] = unpack16<kBf16>(reinterpret_cast<const uint16_t*>(kr)[c]).x;
            v[i] = unpack16<kBf16>(reinterpret_cast<const uint16_t*>(vr)[c]).x;
          }
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float z = s * p.scale_log2;
        const float m = fmaxf(top, z);
        const float f = top == -INFINITY ? 0.f : exp2f(top - m);
        const float w = m == -INFINITY ? (z == z ? 0.f : z) : exp2f(z - m);
        sum = sum * f + w;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + w * v[i];
        top = m;
      }
    }
    if (lane == 0) top_s[warp] = top, sum_s[warp] = sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o_s[warp][lane + 32 * i] = o[i];
    __syncthreads();
    if (warp == 0) {
      float m = -INFINITY;
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, top_s[w]);
      float l = 0.f, acc[kPer] = {};
      for (int w = 0; w < kWarps; ++w) {
        const float f = top_s[w] == -INFINITY ? (sum_s[w] == 0.f ? 0.f : 1.f) : exp2f(top_s[w] - m);
        l += sum_s[w] * f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (f != 0.f) acc[i] += o_s[w][lane + 32 * i] * f;
      }
      const long long at = (static_cast<long long>(b) * p.tokens + t) * q_heads + qh;
      uint16_t* out = reinterpret_cast<uint16_t*>(p.o) + at * D;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        out[lane + 32 * i] =
            static_cast<uint16_t>(pack16<kBf16>(l == 0.f ? 0.f : acc[i] / l, 0.f));
      if (lane == 0)
        p.lse[at] = l == 0.f ? -INFINITY
                             : ((m == -INFINITY ? 0.f : m) + log2f(l)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

}  // namespace

size_t tree_workspace_bytes(int, int, int) { return 16; }

int launch_tree(const TreeParams& p, int d, bool e4m3, bool bf16, int, cudaStream_t stream) {
  const dim3 grid(p.group * p.c.heads, p.tokens, p.t.batch < 65535 ? p.t.batch : 65535);
#define FAT_RUN(D, E, B) tree_kernel<D, E, B><<<grid, 32 * kWarps, 0, stream>>>(p)
  FAT_PICK(d, e4m3, bf16, FAT_RUN);
#undef FAT_RUN
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace fat
