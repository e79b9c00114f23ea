// Kernels of the attention of drafted tokens, head dim 64.
#include "fat_tree_kernel.cuh"

namespace fat {

namespace tree {

int launch_d64(const KernelParams& kp, int type, int blocks, int dev, int sms,
               cudaStream_t stream) {
  switch (type) {
    case kBf16:
      return blocks == 1 ? launch<64, kBf16, 1>(kp, dev, sms, stream)
                         : launch<64, kBf16, 2>(kp, dev, sms, stream);
    case kF16:
      return blocks == 1 ? launch<64, kF16, 1>(kp, dev, sms, stream)
                         : launch<64, kF16, 2>(kp, dev, sms, stream);
    case kE4M3Bf16: return launch<64, kE4M3Bf16, 1>(kp, dev, sms, stream);
    default: return launch<64, kE4M3F16, 1>(kp, dev, sms, stream);
  }
}

}  // namespace tree

}  // namespace fat
