// pi_kv_share.cu -- what groups of sequences share, found in their table rows (sm_103a).
//
// A CTA to a group compares its sequences' rows with the first one's, a warp to a row, and stops at the first column that
// differs from it in any row. A few microseconds once for the steps of a batch; bound by the latency of the loads.
#include "pi_kv_device.cuh"

namespace pi {

constexpr int SH_NT = 1024, SH_NW = SH_NT / 32;

__global__ void __launch_bounds__(SH_NT) k_kv_share(const KvView c, const KvBatch b, const int32_t *groups, int ng, int32_t *plan)
{
    __shared__ int s_room, s_first, s_count, s_cols;
    int32_t *const lead = plan, *const start = lead + ng, *const len = start + ng + 1, *const skip = len + ng;
    int32_t *const was = skip + b.n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    int bad = 0;   // groups out of order or out of range: nothing is shared
    for (int x = tid; x <= ng; x += SH_NT) {
        const int v = groups[x];
        bad |= v < 0 || v > b.n || (x > 0 && groups[x - 1] > v);
    }
    bad = __syncthreads_or(bad);
    if (g == ng) {   // the rest of the plan: sequences of no group, and the batch that it is for
        if (bad && tid == 0) set_status(c.status, ST_DEVICE_CHECK);
        for (int x = tid; x < b.n; x += SH_NT) {
            if (bad || x < groups[0] || x >= groups[ng]) skip[x] = 0;
            was[x] = b.seqs[x];
        }
        for (int x = tid; x <= b.n; x += SH_NT) was[b.n + x] = b.start[x];
        if (tid == 0) start[ng] = bad ? 0 : b.start[groups[ng]];
        return;
    }
    const int lo = bad ? 0 : groups[g], hi = bad ? 0 : groups[g + 1];
    if (tid == 0) {
        s_room = INT32_MAX;
        s_first = INT32_MAX;
        s_count = 0;
    }
    __syncthreads();
    // sequences with new tokens: how many, the first, and the positions that all of them had before
    for (int i = lo + tid; i < hi; i += SH_NT) {
        const KvSeq q = kv_sequence(c, b, i, true);
        if (q.n == 0) continue;
        atomicAdd(&s_count, 1);
        atomicMin(&s_first, i);
        atomicMin(&s_room, max(q.len - q.n, 0));
    }
    __syncthreads();
    const int room = s_room;
    const bool any = s_count > 1;
    if (tid == 0) s_cols = any ? room / c.page : 0;
    __syncthreads();
    const int first = any ? s_first : 0;
    const int32_t *const row = c.table + (size_t)(any ? b.seqs[first] : 0) * c.max_pages;
    for (int i = first + warp; any && i < hi; i += SH_NW) {
        const KvSeq q = kv_sequence(c, b, i, false);
        if (q.n == 0) continue;
        const int32_t *const mine = c.table + (size_t)q.row * c.max_pages;
        for (int x = 0; x < __shfl_sync(0xffffffffu, *(volatile int *)&s_cols, 0); x += 32) {   // (one answer to a warp)
            const int at = x + lane;
            bool differs = false;
            if (at * (int64_t)c.page < room) {
                const int id = row[at];
                differs = id < 0 || id >= c.n_pages || mine[at] != id;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, differs);
            if (m) {
                if (lane == 0) atomicMin(&s_cols, x + __ffs(m) - 1);
                break;
            }
        }
    }
    __syncthreads();
    const int shared = any ? min(room, s_cols * c.page) / KV_SHARE * KV_SHARE : 0;
    for (int i = lo + tid; i < hi; i += SH_NT) skip[i] = kv_sequence(c, b, i, false).n ? shared : 0;
    if (tid == 0) {
        lead[g] = any ? b.seqs[first] : 0;
        start[g] = bad ? 0 : b.start[lo];
        len[g] = shared;
    }
}

cudaError_t launch_kv_share(const KvView &c, const KvBatch &b, const int32_t *groups, int n_groups, int32_t *plan, cudaStream_t s)
{
    Launch L;
    L.grid = dim3((unsigned)n_groups + 1);
    L.block = dim3(SH_NT);
    L.smem = 0;
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    return launch_ex(L, k_kv_share, c, b, groups, n_groups, plan);
}

}  // namespace pi
