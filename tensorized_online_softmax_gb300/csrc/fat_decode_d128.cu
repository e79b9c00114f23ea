// Decode kernels, head dim 128, and the choice by head dim.
#include "fat_decode_kernel.cuh"

namespace fat {

int launch_decode_d64(const DecodeParams& p, bool e4m3, bool bf16, int dev, cudaStream_t stream);

size_t decode_workspace_bytes(int d) {
  return decode::kJoinBytes + decode::kLseBytes +
         sizeof(float) * kDecodeMaxBlocks * 2 * decode::kMaxRows * d;
}

int launch_decode(const DecodeParams& p, int d, bool e4m3, bool bf16, int dev,
                  cudaStream_t stream) {
  return d == 128 ? decode::dispatch<128>(p, e4m3, bf16, dev, stream)
                  : launch_decode_d64(p, e4m3, bf16, dev, stream);
}

}  // namespace fat
