// pi_kv_split_d128.cu -- split attention kernels, head dim 128 (template in pi_kv_split.cuh).
#include "pi_kv_split.cuh"

namespace pi {
PI_KV_SPLIT(, 128)
}  // namespace pi
