// pi_kv_split_d256.cu -- split attention kernels for head dim 256 (template in pi_kv_split.cuh).
#include "pi_kv_split.cuh"

namespace pi {
template cudaError_t split_setup<256, true>();
template cudaError_t split_setup<256, false>();
template cudaError_t split_launch<256, true>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
template cudaError_t split_launch<256, false>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                             cudaStream_t);
}  // namespace pi
