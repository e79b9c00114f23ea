// Kernels of the attention of drafted tokens, head dim 128.
#include "fat_tree_kernel.cuh"

namespace fat {

namespace tree {

int launch_d128(const KernelParams& kp, int type, int blocks, int dev, int sms,
               cudaStream_t stream) {
  switch (type) {
    case kBf16:
      return blocks == 1 ? launch<128, kBf16, 1>(kp, dev, sms, stream)
                         : launch<128, kBf16, 2>(kp, dev, sms, stream);
    case kF16:
      return blocks == 1 ? launch<128, kF16, 1>(kp, dev, sms, stream)
                         : launch<128, kF16, 2>(kp, dev, sms, stream);
    case kE4M3Bf16: return launch<128, kE4M3Bf16, 1>(kp, dev, sms, stream);
    default: return launch<128, kE4M3F16, 1>(kp, dev, sms, stream);
  }
}

}  // namespace tree

}  // namespace fat
