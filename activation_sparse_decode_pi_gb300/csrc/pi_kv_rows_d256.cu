// pi_kv_rows_d256.cu -- attention kernels for many query rows, head dim 256 (template in pi_kv_rows.cuh).
#include "pi_kv_rows.cuh"

namespace pi {
PI_KV_ROWS(, 256, false)
}  // namespace pi
