// pi_kv_rows_shared_d256.cu -- attention kernels for many query rows, for a pass over or behind shared prefixes, head dim 256 (template in
// pi_kv_rows.cuh).
#include "pi_kv_rows.cuh"

namespace pi {
PI_KV_ROWS(, 256, true)
}  // namespace pi
