// pi_kv_split_d64.cu -- split attention kernels for head dim 64 (template in pi_kv_split.cuh).
#include "pi_kv_split.cuh"

namespace pi {
template cudaError_t split_setup<64, 1, 1>();
template cudaError_t split_launch<64, 1, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
template cudaError_t split_setup<64, 1, 2>();
template cudaError_t split_launch<64, 1, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
template cudaError_t split_setup<64, 2, 1>();
template cudaError_t split_launch<64, 2, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
template cudaError_t split_setup<64, 2, 2>();
template cudaError_t split_launch<64, 2, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int,
                                            cudaStream_t);
}  // namespace pi
