// pi_kv_split_d256.cu -- split attention kernels for head dim 256 (template in pi_kv_split.cuh).
#include "pi_kv_split.cuh"

namespace pi {
template cudaError_t split_setup<256, 1, 1>();
template cudaError_t split_launch<256, 1, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
template cudaError_t split_setup<256, 1, 2>();
template cudaError_t split_launch<256, 1, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
template cudaError_t split_setup<256, 2, 1>();
template cudaError_t split_launch<256, 2, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
template cudaError_t split_setup<256, 2, 2>();
template cudaError_t split_launch<256, 2, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
}  // namespace pi
