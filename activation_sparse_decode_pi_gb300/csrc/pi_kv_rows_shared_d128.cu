// pi_kv_rows_shared_d128.cu -- attention kernels for many query rows, for a pass over or behind shared prefixes, head dim 128 (template in
// pi_kv_rows.cuh).
#include "pi_kv_rows.cuh"

namespace pi {
PI_KV_ROWS(, 128, true)
PI_KV_ROWS_FEW(, 128)
}  // namespace pi
