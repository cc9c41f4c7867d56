// pi_kv_split_d64.cu -- split attention kernels for head dim 64 (template in pi_kv_split.cuh).
#include "pi_kv_split.cuh"

namespace pi {
template cudaError_t split_setup<64, true>();
template cudaError_t split_setup<64, false>();
template cudaError_t split_launch<64, true>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
template cudaError_t split_launch<64, false>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                             cudaStream_t);
}  // namespace pi
