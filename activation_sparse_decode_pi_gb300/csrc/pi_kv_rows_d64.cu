// pi_kv_rows_d64.cu -- attention kernels for many query rows, head dim 64 (template in pi_kv_rows.cuh).
#include "pi_kv_rows.cuh"

namespace pi {
template cudaError_t rows_setup<64, 1>();
template cudaError_t rows_setup<64, 2>();
template cudaError_t rows_launch<64, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, unsigned, unsigned, cudaStream_t);
template cudaError_t rows_launch<64, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, unsigned, unsigned, cudaStream_t);
}  // namespace pi
