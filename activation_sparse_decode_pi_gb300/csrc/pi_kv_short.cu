// pi_kv_short.cu -- attention behind a shared prefix (template in pi_kv_short.cuh).
#include "pi_kv_short.cuh"

namespace pi {
template cudaError_t short_setup<64, 1>();
template cudaError_t short_setup<64, 2>();
template cudaError_t short_setup<128, 1>();
template cudaError_t short_setup<128, 2>();
template cudaError_t short_launch<64, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t);
template cudaError_t short_launch<64, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t);
template cudaError_t short_launch<128, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t);
template cudaError_t short_launch<128, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t);
}  // namespace pi
