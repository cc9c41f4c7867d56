// pi_kv_rows_d128.cu -- attention kernels for many query rows, head dim 128 (template in pi_kv_rows.cuh).
#include "pi_kv_rows.cuh"

namespace pi {
template cudaError_t rows_setup<128, 1>();
template cudaError_t rows_setup<128, 2>();
template cudaError_t rows_launch<128, 1>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, unsigned, unsigned, cudaStream_t);
template cudaError_t rows_launch<128, 2>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, unsigned, unsigned, cudaStream_t);
}  // namespace pi
