// pi_kv_split_d64.cu -- split attention kernels, head dim 64 (template in pi_kv_split.cuh).
#include "pi_kv_split.cuh"

namespace pi {
PI_KV_SPLIT(, 64)
}  // namespace pi
