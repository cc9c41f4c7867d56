// pi_kv_split_shared_d256.cu -- split attention kernels, for a pass over or behind shared prefixes, head dim 256 (template in
// pi_kv_split.cuh).
#include "pi_kv_split.cuh"

namespace pi {
PI_KV_SPLIT_SHARED()
}  // namespace pi
