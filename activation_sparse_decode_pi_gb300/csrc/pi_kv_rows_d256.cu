// pi_kv_rows_d256.cu -- attention kernels for many query rows, head dim 256 (template in pi_kv_rows.cuh).
#include "pi_kv_rows.cuh"

namespace pi {
template cudaError_t rows_setup<256, 1>();
template cudaError_t rows_setup<256, 2>();
template cudaError_t rows_launch<256, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, unsigned, unsigned, cudaStream_t);
template cudaError_t rows_launch<256, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, unsigned, unsigned, cudaStream_t);
}  // namespace pi
