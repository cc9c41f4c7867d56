// pi_kv_rows_d64.cu -- attention kernels for many query rows, head dim 64 (template in pi_kv_rows.cuh).
#include "pi_kv_rows.cuh"

namespace pi {
PI_KV_ROWS(, 64, false)
}  // namespace pi
