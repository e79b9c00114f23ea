// Decode kernels, head dim 64.
#include "fat_decode_kernel.cuh"

namespace fat {

int launch_decode_d64(const DecodeParams& p, bool e4m3, bool bf16, int dev, cudaStream_t stream) {
  return decode::dispatch<64>(p, e4m3, bf16, dev, stream);
}

}  // namespace fat
