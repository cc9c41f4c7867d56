// pi_kv_rows_d128.cu -- attention kernels for many query rows, head dim 128 (template in pi_kv_rows.cuh).
#include "pi_kv_rows.cuh"

namespace pi {
PI_KV_ROWS(, 128, false)
}  // namespace pi
