// pi_kv_split_d256.cu -- split attention kernels, head dim 256 (template in pi_kv_split.cuh).
#include "pi_kv_split.cuh"

namespace pi {
PI_KV_SPLIT(, 256)
}  // namespace pi
