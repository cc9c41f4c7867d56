// pi_kv_pages.cu -- bookkeeping and copies of the paged cache's pages (sm_103a).
//
// A page is free when its reference count is 0, and pages are handed out lowest id first: there is no
// free list to keep, the pool stays dense at its bottom, and every result is a function of the state.
// The bookkeeping of reserve, fork and compact needs the counts in order (a prefix sum), so one CTA
// does it; the copies of the listed pages run on the whole GPU right behind it. Measured: 8 to 64 sequences
// forked over 8 layers 48 us (7 us of it bookkeeping), 16 of 32 sequences' pages moved down 205 us = 5.6 TB/s.
#include <algorithm>

#include "pi_kv_device.cuh"

namespace pi {

constexpr int PG_NT = 1024, PG_NW = PG_NT / 32;
constexpr uint32_t ST_OOM = 4;

// Exclusive prefix sum over the CTA's PG_NT threads; total: the sum. ws: PG_NW + 1 words.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *ws, T &total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) ws[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        T w = ws[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        ws[lane] = w;
    }
    __syncthreads();
    const T base = warp ? ws[warp - 1] : 0;
    total = ws[PG_NW - 1];
    __syncthreads();
    return base + inc - v;
}

// The lowest `need` free pages, ascending, into list; their number (less than need when the pool is short).
__device__ int find_free(const KvView &c, long long need, int32_t *list, int *ws)
{
    constexpr int PER = 8;
    int found = 0;
    for (int base = 0; base < c.n_pages && found < need; base += PG_NT * PER) {
        const int id0 = base + threadIdx.x * PER;
        uint32_t bits = 0;
#pragma unroll
        for (int x = 0; x < PER; ++x)
            if (id0 + x < c.n_pages && __ldcg(c.ref + id0 + x) <= 0) bits |= 1u << x;
        int total;
        int at = found + block_scan(__popc(bits), ws, total);
        for (; bits; bits &= bits - 1, ++at)
            if (at < need) list[at] = id0 + __ffs(bits) - 1;
        found += total;
    }
    __syncthreads();
    return (int)min((long long)found, need);
}

__device__ __forceinline__ int pages_of(const KvView &c, int len) { return (int)(((long long)len + c.page - 1) / c.page); }

// Give back columns [c0, c1) of table row `row` by the calling warp (the entries stay).
__device__ __forceinline__ void warp_release(const KvView &c, int row, int c0, int c1)
{
    const int32_t *r = c.table + (size_t)row * c.max_pages;
    for (int x = c0 + (threadIdx.x & 31); x < c1; x += 32) {
        const int id = r[x];
        if (id >= 0 && id < c.n_pages) atomicSub(c.ref + id, 1);
        else if (id != -1) set_status(c.status, ST_DEVICE_CHECK);
    }
}

// Length of table row `row`, 0 (and flagged) when it is not one the row can have.
__device__ __forceinline__ int row_length(const KvView &c, int row)
{
    const int len = c.length[row];
    if (len >= 0 && len <= c.max_pages * c.page) return len;
    set_status(c.status, ST_DEVICE_CHECK);
    return 0;
}

__global__ void __launch_bounds__(PG_NT) k_kv_reserve(const KvView c, const KvBatch b, int32_t *list)
{
    __shared__ long long ws[PG_NW + 1];
    __shared__ int wi[PG_NW + 1];
    __shared__ int s_row[PI_KV_MAX_CALL_SEQS], s_c0[PI_KV_MAX_CALL_SEQS], s_need[PI_KV_MAX_CALL_SEQS];
    __shared__ long long s_off[PI_KV_MAX_CALL_SEQS];
    pdl_wait();
    pdl_launch_dependents();
    const int i = threadIdx.x;
    KvSeq q{0, 0, 0, 0};
    int need = 0;
    if (i < b.n) {
        q = kv_sequence(c, b, i, true);
        if ((long long)q.len + q.n > (long long)c.max_pages * c.page) {
            set_status(c.status, ST_OOM);
            q.n = 0;
        }
        need = pages_of(c, q.len + q.n) - pages_of(c, q.len);
    }
    long long total;
    const long long off = block_scan((long long)need, ws, total);
    const int have = find_free(c, min(total, (long long)c.n_pages), list, wi);
    if (i < b.n) {
        const bool ok = need == 0 || off + need <= have;
        if (!ok) set_status(c.status, ST_OOM);
        s_row[i] = q.row;
        s_c0[i] = pages_of(c, q.len);
        s_need[i] = ok ? need : 0;
        s_off[i] = off;
        if (ok && q.n > 0) c.length[q.row] = q.len + q.n;
    }
    __syncthreads();
    for (int k = threadIdx.x >> 5; k < b.n; k += PG_NW)
        for (int x = threadIdx.x & 31; x < s_need[k]; x += 32) {
            const int id = list[s_off[k] + x];
            c.table[(size_t)s_row[k] * c.max_pages + s_c0[k] + x] = id;
            c.ref[id] = 1;
        }
}

__global__ void __launch_bounds__(PG_NT) k_kv_fork(const KvView c, const int32_t *src, const int32_t *dst, int n,
                                                   const KvCopyList l)
{
    __shared__ int wi[PG_NW + 1];
    __shared__ int s_src[PI_KV_MAX_CALL_SEQS], s_dst[PI_KV_MAX_CALL_SEQS], s_rank[PI_KV_MAX_CALL_SEQS];
    __shared__ int s_len[PI_KV_MAX_CALL_SEQS], s_old[PI_KV_MAX_CALL_SEQS];
    pdl_wait();
    pdl_launch_dependents();
    const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
    int need = 0;
    if (i < n) {
        const int a = src[i], d = dst[i];
        const bool bad = a < 0 || a >= c.max_seqs || d < 0 || d >= c.max_seqs || a == d;
        if (bad) set_status(c.status, ST_DEVICE_CHECK);
        s_src[i] = bad ? -1 : a;
        s_dst[i] = d;
        s_len[i] = bad ? 0 : row_length(c, a);
        s_old[i] = bad ? 0 : pages_of(c, row_length(c, d));
        need = s_len[i] % c.page != 0;
    }
    int total;
    const int rank = block_scan(need, wi, total);
    if (i < n) s_rank[i] = rank;
    __syncthreads();
    for (int k = warp; k < n; k += PG_NW)
        if (s_src[k] >= 0) warp_release(c, s_dst[k], 0, s_old[k]);
    __syncthreads();
    const int have = find_free(c, total, l.dst, wi);
    for (int k = warp; k < n; k += PG_NW) {
        if (s_src[k] < 0) continue;
        const int32_t *from = c.table + (size_t)s_src[k] * c.max_pages;
        int32_t *to = c.table + (size_t)s_dst[k] * c.max_pages;
        int full = s_len[k] / c.page, len = s_len[k];
        const bool part = len % c.page != 0;
        if (part && s_rank[k] >= have) {
            if (lane == 0) set_status(c.status, ST_OOM);
            full = len = 0;
        }
        for (int x = lane; x < full; x += 32) {
            const int id = from[x];
            to[x] = id;
            if (id >= 0 && id < c.n_pages) atomicAdd(c.ref + id, 1);
        }
        const int used = full + (part && len > 0);
        if (used > full && lane == 0) {
            const int id = l.dst[s_rank[k]];
            to[full] = id;
            c.ref[id] = 1;
            l.src[s_rank[k]] = from[full];
        }
        for (int x = used + lane; x < s_old[k]; x += 32) to[x] = -1;
        if (lane == 0) c.length[s_dst[k]] = len;
    }
    if (i == 0) *l.count = have;
}

__global__ void __launch_bounds__(256) k_kv_free(const KvView c, const int32_t *seqs)
{
    pdl_wait();
    pdl_launch_dependents();
    const int row = seqs[blockIdx.x];
    if (row < 0 || row >= c.max_seqs) {
        if (threadIdx.x == 0) set_status(c.status, ST_DEVICE_CHECK);
        return;
    }
    const int used = pages_of(c, row_length(c, row));
    __syncthreads();
    for (int x = threadIdx.x; x < used; x += 256) {
        int32_t *e = c.table + (size_t)row * c.max_pages + x;
        const int id = *e;
        if (id >= 0 && id < c.n_pages) atomicSub(c.ref + id, 1);
        else if (id != -1) set_status(c.status, ST_DEVICE_CHECK);
        *e = -1;
    }
    if (threadIdx.x == 0) c.length[row] = 0;
}

__global__ void __launch_bounds__(256) k_kv_trim(const KvView c, const int32_t *seqs, int window, int sinks)
{
    pdl_wait();
    pdl_launch_dependents();
    const int row = seqs[blockIdx.x];
    if (row < 0 || row >= c.max_seqs) {
        if (threadIdx.x == 0) set_status(c.status, ST_DEVICE_CHECK);
        return;
    }
    const long long last = (long long)row_length(c, row) - window;   // last position out of view
    const int c0 = (int)(((long long)sinks + c.page - 1) / c.page);
    const long long c1 = (last + 1) / c.page;                        // pages that end at or before it
    for (long long x = c0 + (int)threadIdx.x; x < c1; x += 256) {
        int32_t *e = c.table + (size_t)row * c.max_pages + x;
        const int id = *e;
        if (id >= 0 && id < c.n_pages) atomicSub(c.ref + id, 1);
        else if (id != -1) set_status(c.status, ST_DEVICE_CHECK);
        *e = -1;
    }
}

__global__ void __launch_bounds__(PG_NT) k_kv_compact(const KvView c, const KvCopyList l, int32_t *map, int32_t *n_live)
{
    constexpr int PER = 8;
    __shared__ int wi[PG_NW + 1];
    pdl_wait();
    pdl_launch_dependents();
    int mine = 0, m;
    for (int id = threadIdx.x; id < c.n_pages; id += PG_NT) mine += c.ref[id] > 0;
    block_scan(mine, wi, m);
    int holes = 0, movers = 0;
    for (int base = 0; base < c.n_pages; base += PG_NT * PER) {
        const int id0 = base + threadIdx.x * PER;
        uint32_t hole = 0, move = 0;
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            const int id = id0 + x;
            if (id >= c.n_pages) break;
            const bool live = c.ref[id] > 0;
            hole |= (uint32_t)(!live && id < m) << x;
            move |= (uint32_t)(live && id >= m) << x;
            map[id] = id;
        }
        int nh, nm;
        int at = holes + block_scan(__popc(hole), wi, nh);
        for (; hole; hole &= hole - 1) l.dst[at++] = id0 + __ffs(hole) - 1;
        at = movers + block_scan(__popc(move), wi, nm);
        for (; move; move &= move - 1) l.src[at++] = id0 + __ffs(move) - 1;
        holes += nh;
        movers += nm;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < holes; x += PG_NT) {
        const int s = l.src[x], d = l.dst[x];
        map[s] = d;
        c.ref[d] = c.ref[s];
        c.ref[s] = 0;
    }
    if (threadIdx.x == 0) {
        *l.count = holes;
        if (n_live) *n_live = m;
    }
}

// ---------------------------------------------------------------- copies --------------------

constexpr int CP_NT = 256, CP_CHUNK = CP_NT * 16 * 4;   // bytes of one unit: four 16-byte vectors a thread

__global__ void __launch_bounds__(CP_NT) k_kv_copy(const KvView c, const KvLayerDev *__restrict__ layers,
                                                   const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                                                   const int32_t *count, int max_count, const int32_t *map)
{
    pdl_wait();
    pdl_launch_dependents();
    const int n = count ? min(*count, max_count) : max_count;
    const size_t bytes = (size_t)c.hkv * c.page * c.dim;   // of a page in one array
    const int chunks = (int)((bytes + CP_CHUNK - 1) / CP_CHUNK);
    const long long units = (long long)n * c.n_layers * 2 * chunks;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int ch = (int)(u % chunks);
        const long long v = u / chunks;
        const int kv = (int)(v & 1), layer = (int)((v >> 1) % c.n_layers), x = (int)((v >> 1) / c.n_layers);
        const int a = src[x], b = dst[x];
        if (a < 0 || a >= c.n_pages || b < 0 || b >= c.n_pages) {
            if (threadIdx.x == 0) set_status(c.status, ST_DEVICE_CHECK);
            continue;
        }
        const KvLayerDev &l = layers[layer];
        uint8_t *base = kv ? l.v : l.k;
        const uint4 *s = (const uint4 *)(base + (size_t)a * bytes + (size_t)ch * CP_CHUNK);
        uint4 *d = (uint4 *)(base + (size_t)b * bytes + (size_t)ch * CP_CHUNK);
        const int left = (int)(min(bytes - (size_t)ch * CP_CHUNK, (size_t)CP_CHUNK) / 16);
        uint4 r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e * CP_NT + (int)threadIdx.x < left) r[e] = __ldcs(s + e * CP_NT + threadIdx.x);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e * CP_NT + (int)threadIdx.x < left) d[e * CP_NT + threadIdx.x] = r[e];
        if (ch == 0) {
            float *sc = kv ? l.vs : l.ks;
            for (int h = threadIdx.x; h < c.hkv; h += CP_NT) sc[(size_t)b * c.hkv + h] = sc[(size_t)a * c.hkv + h];
        }
    }
    if (map)   // rename the table's entries, a warp to a row
        for (int row = blockIdx.x * (CP_NT / 32) + (threadIdx.x >> 5); row < c.max_seqs;
             row += gridDim.x * (CP_NT / 32)) {
            const int used = pages_of(c, row_length(c, row));
            for (int x = threadIdx.x & 31; x < used; x += 32) {
                int32_t *e = c.table + (size_t)row * c.max_pages + x;
                const int id = *e;
                if (id >= 0 && id < c.n_pages) {
                    const int to = map[id];
                    if (to != id) *e = to;
                }
            }
        }
}

// ---------------------------------------------------------------- launches ------------------

static Launch at(dim3 grid, int threads, cudaStream_t s)
{
    Launch L;
    L.grid = grid;
    L.block = dim3(threads);
    L.smem = 0;
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    return L;
}

cudaError_t launch_kv_reserve(const KvView &c, const KvBatch &b, int32_t *list, cudaStream_t s)
{
    return launch_ex(at(dim3(1), PG_NT, s), k_kv_reserve, c, b, list);
}

cudaError_t launch_kv_fork(const KvView &c, const int32_t *src, const int32_t *dst, int n, const KvCopyList &l,
                           cudaStream_t s)
{
    return launch_ex(at(dim3(1), PG_NT, s), k_kv_fork, c, src, dst, n, l);
}

cudaError_t launch_kv_free(const KvView &c, const int32_t *seqs, int n, cudaStream_t s)
{
    return launch_ex(at(dim3(n), 256, s), k_kv_free, c, seqs);
}

cudaError_t launch_kv_trim(const KvView &c, const int32_t *seqs, int n, int window, int sinks, cudaStream_t s)
{
    return launch_ex(at(dim3(n), 256, s), k_kv_trim, c, seqs, window, sinks);
}

cudaError_t launch_kv_compact(const KvView &c, const KvCopyList &l, int32_t *map, int32_t *n_live, cudaStream_t s)
{
    return launch_ex(at(dim3(1), PG_NT, s), k_kv_compact, c, l, map, n_live);
}

cudaError_t launch_kv_copy(const KvView &c, const KvLayerDev *layers, const int32_t *src, const int32_t *dst,
                           const int32_t *count, int max_count, const int32_t *map, int nsm, cudaStream_t s)
{
    const size_t bytes = (size_t)c.hkv * c.page * c.dim;
    const long long units = (long long)max_count * c.n_layers * 2 * ((bytes + CP_CHUNK - 1) / CP_CHUNK);
    const long long rows = map ? (c.max_seqs + CP_NT / 32 - 1) / (CP_NT / 32) : 0;
    const unsigned grid = (unsigned)std::max(1ll, std::min((long long)nsm * 8, std::max(units, rows)));
    return launch_ex(at(dim3(grid), CP_NT, s), k_kv_copy, c, layers, src, dst, count, max_count, map);
}

}  // namespace pi
