// pi_kv_api.cu -- host side of the paged-cache C ABI declared in include/pi_kv.h.
//
// Validates every argument before launching anything, owns the workspace (partials of sequences
// whose cache is split over CTAs, page lists, status word) and the tensor maps of the pools.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "pi_internal.h"
#include "pi_kv_internal.h"

using namespace pi;

struct pi_kv {
    pi_kv_desc_t desc;
    std::vector<KvLayerDev> layers;
    std::vector<CUtensorMap> map_k, map_v;
    KvView view;
    int dev = 0, nsm = 0;
    void *ws = nullptr;
    float *part = nullptr, *part_ml = nullptr;
    float *rows_part = nullptr, *rows_ml = nullptr;
    uint32_t *tickets = nullptr, *rows_tickets = nullptr, *status = nullptr;
    KvLayerDev *layers_dev = nullptr;
    int32_t *list_src = nullptr, *list_dst = nullptr, *list_count = nullptr, *page_map = nullptr;
};

namespace {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        return (EncodeFn)p;
    cudaGetLastError();
    return nullptr;
}

pi_status_t cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return PI_OK;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? PI_ERR_OOM : PI_ERR_CUDA;
}

pi_status_t validate(const pi_kv_desc_t *d)
{
    if (!d || injected_fault() == FAULT_BADARG) return PI_ERR_INVALID_ARG;
    if (d->n_layers < 1 || d->n_kv_heads < 1 || d->n_heads < d->n_kv_heads || d->n_heads % d->n_kv_heads ||
        d->head_dim < 1 || d->page_tokens < 1 || d->n_pages < 1 || d->max_seqs < 1 || d->max_pages < 1)
        return PI_ERR_INVALID_ARG;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return PI_ERR_UNSUPPORTED;
    if (d->page_tokens != 16 && d->page_tokens != 32 && d->page_tokens != 64 && d->page_tokens != 128)
        return PI_ERR_UNSUPPORTED;
    if (d->n_heads > (1 << 16)) return PI_ERR_UNSUPPORTED;
    const int64_t lim = (int64_t)1 << 31;
    // tensor-map rows and positions are 32-bit
    if ((int64_t)d->n_pages * d->n_kv_heads >= lim / d->page_tokens || (int64_t)d->max_pages * d->page_tokens > KV_MAX_LEN)
        return PI_ERR_UNSUPPORTED;
    return PI_OK;
}

// Pool of one layer as rows of head_dim bytes; boxes of one 64-position tile's share of a page and
// 128 bytes (64 for head_dim 64), swizzled so that the kernels' reads spread over the banks.
bool encode_pool(EncodeFn fn, CUtensorMap *m, const pi_kv_desc_t &d, void *base)
{
    const cuuint64_t dims[2] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.n_pages * d.n_kv_heads * d.page_tokens};
    const cuuint64_t strides[1] = {(cuuint64_t)d.head_dim};
    const cuuint32_t box[2] = {(cuuint32_t)(d.head_dim < 128 ? d.head_dim : 128),
                               (cuuint32_t)(d.page_tokens < KV_TILE ? d.page_tokens : KV_TILE)};
    const cuuint32_t one[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              d.head_dim < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t setup_of()
{
    for (cudaError_t e : {split_setup<D, 1, 1>(), split_setup<D, 1, 2>(), split_setup<D, 2, 1>(), split_setup<D, 2, 2>(),
                          rows_setup<D, 1>(), rows_setup<D, 2>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

// Sequences with at least this many rows (new tokens x heads of a group) are worth a 128-row tile. Measured, 16 sequences
// of 4096, 64 query heads on 8, split / rows kernel: 16 rows 45 / 79 us, 32 rows 71 / 83 us, 48 rows 95 / 72 us, 64 rows
// 120 / 73 us; fp32: 32 rows 99 / 118 us, 64 rows 173 / 109 us.
constexpr int ROWS_FROM = 33;

// The kernels of one call: the split kernel for sequences with few rows, the rows kernel for the others.
template <int D>
cudaError_t attend_of(const pi_kv *h, int layer, KvAttendArgs a, cudaStream_t s)
{
    const int64_t n = a.b.n, group = a.c.hq / a.c.hkv, rows = (int64_t)a.b.n_tokens * group;
    // the host knows the rows' total only: one sequence has them all, and a token each is a decode step
    const bool many = rows >= ROWS_FROM && (n == 1 || a.b.n_tokens > n), few = n > 1 || !many;
    a.rows_from = many ? (few ? ROWS_FROM : 0) : INT32_MAX;
    cudaError_t e = cudaSuccess;
    if (few) {
        // 16 rows to a tile where the rows of a sequence (on average: all that the host knows) fill more than 8: the cache
        // is then read once instead of twice (64 sequences, 16 heads to a group: 229 / 323 us with 16 / 8; 8 heads, 128
        // sequences: 381 / 330 us, since 16 leave room for fewer warps)
        const bool wide = many || rows > 8 * n, one = a.dtype == PI_BF16;
        const auto run = wide ? (one ? split_launch<D, 2, 1> : split_launch<D, 2, 2>)
                              : (one ? split_launch<D, 1, 1> : split_launch<D, 1, 2>);
        e = run(a, h->map_k[layer], h->map_v[layer], h->nsm, s);
    }
    if (many && e == cudaSuccess) {
        const int64_t items = (rows / rows_per_item(D) + n) * a.c.hkv;   // at most one partly filled per sequence
        const int64_t splits = items < h->nsm ? std::min<int64_t>(16, 2 * h->nsm / items) : 1;
        const CUtensorMap &mk = h->map_k[layer], &mv = h->map_v[layer];
        e = a.dtype == PI_F32 ? rows_launch<D, 2>(a, mk, mv, (unsigned)items, (unsigned)splits, s)
                              : rows_launch<D, 1>(a, mk, mv, (unsigned)items, (unsigned)splits, s);
    }
    return e;
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

pi_status_t kv_create(pi_kv_t **out, const pi_kv_desc_t *desc, const pi_kv_layer_t *layers,
                      const pi_kv_state_t *state)
{
    pi_status_t s;
    if ((s = validate(desc))) return s;
    if (!layers || !state) return PI_ERR_INVALID_ARG;
    const pi_kv_desc_t &d = *desc;
    int dev = 0, nsm = 0;
    if ((s = cuda_status(cudaGetDevice(&dev)))) return s;
    if ((s = cuda_status(cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))) return s;
    const size_t rows = (size_t)d.n_pages * d.n_kv_heads, pool = rows * d.page_tokens * d.head_dim;
    for (int l = 0; l < d.n_layers; ++l) {
        if ((s = check_ptr(layers[l].k, pool, 128, dev))) return s;
        if ((s = check_ptr(layers[l].v, pool, 128, dev))) return s;
        if ((s = check_ptr(layers[l].k_scale, rows * 4, 4, dev))) return s;
        if ((s = check_ptr(layers[l].v_scale, rows * 4, 4, dev))) return s;
    }
    if ((s = check_ptr(state->table, (size_t)d.max_seqs * d.max_pages * 4, 4, dev))) return s;
    if ((s = check_ptr(state->length, (size_t)d.max_seqs * 4, 4, dev))) return s;
    if ((s = check_ptr(state->ref, (size_t)d.n_pages * 4, 4, dev))) return s;
    EncodeFn enc = encode_fn();
    if (!enc) return PI_ERR_CUDA;

    struct Holder {   // frees what exists when a later step fails
        pi_kv_t *h;
        ~Holder()
        {
            if (!h) return;
            if (h->ws) cudaFree(h->ws);
            delete h;
        }
    } hold{new pi_kv};
    pi_kv_t *h = hold.h;
    h->desc = d;
    h->dev = dev;
    h->nsm = nsm;
    h->map_k.resize(d.n_layers);
    h->map_v.resize(d.n_layers);
    for (int l = 0; l < d.n_layers; ++l) {
        h->layers.push_back({(uint8_t *)layers[l].k, (uint8_t *)layers[l].v, layers[l].k_scale, layers[l].v_scale});
        if (!encode_pool(enc, &h->map_k[l], d, layers[l].k) || !encode_pool(enc, &h->map_v[l], d, layers[l].v))
            return PI_ERR_CUDA;
    }
    if ((s = cuda_status(d.head_dim == 64    ? setup_of<64>()
                         : d.head_dim == 128 ? setup_of<128>()
                                             : setup_of<256>())))
        return s;
    const size_t list = up(sizeof(int32_t) * (size_t)std::max(d.n_pages, PI_KV_MAX_CALL_SEQS));
    const size_t part = up((size_t)2 * nsm * 16 * d.head_dim * 4), ml = up((size_t)2 * nsm * 16 * 2 * 4);
    const size_t tick = up((size_t)nsm * 4), lay = up(sizeof(KvLayerDev) * (size_t)d.n_layers);
    const size_t rpart = up((size_t)2 * nsm * rows_per_item(d.head_dim) * d.head_dim * 4),
                 rml = up((size_t)2 * nsm * rows_per_item(d.head_dim) * 2 * 4);
    const size_t total = 3 * list + part + ml + rpart + rml + 3 * tick + lay + 2 * 256;
    if (injected_fault() == FAULT_ALLOC) return PI_ERR_OOM;
    if ((s = cuda_status(cudaMalloc(&h->ws, total)))) return s;
    if (injected_fault() == FAULT_UPLOAD) return PI_ERR_CUDA;
    if ((s = cuda_status(cudaMemset(h->ws, 0, total)))) return s;
    uint8_t *p = (uint8_t *)h->ws;
    auto take = [&](size_t n) {
        uint8_t *r = p;
        p += n;
        return r;
    };
    h->part = (float *)take(part);
    h->part_ml = (float *)take(ml);
    h->rows_part = (float *)take(rpart);
    h->rows_ml = (float *)take(rml);
    h->tickets = (uint32_t *)take(tick);
    h->rows_tickets = (uint32_t *)take(2 * tick);
    h->layers_dev = (KvLayerDev *)take(lay);
    h->list_src = (int32_t *)take(list);
    h->list_dst = (int32_t *)take(list);
    h->page_map = (int32_t *)take(list);
    h->list_count = (int32_t *)take(256);
    h->status = (uint32_t *)take(256);
    if ((s = cuda_status(cudaMemcpy(h->layers_dev, h->layers.data(), sizeof(KvLayerDev) * (size_t)d.n_layers,
                                    cudaMemcpyHostToDevice))))
        return s;
    if ((s = cuda_status(cudaDeviceSynchronize()))) return s;
    h->view = {d.n_layers, d.n_heads,  d.n_kv_heads, d.head_dim,    d.page_tokens, d.n_pages,
               d.max_seqs, d.max_pages, state->table, state->length, state->ref,    h->status};
    *out = h;
    hold.h = nullptr;
    return PI_OK;
}

// The handle is used on the device it was made on, with a list of at most PI_KV_MAX_CALL_SEQS sequences.
pi_status_t check_call(const pi_kv_t *h, int32_t n)
{
    if (!h || n < 0 || n > PI_KV_MAX_CALL_SEQS) return PI_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cuda_status(cudaGetLastError());
    return dev == h->dev ? PI_OK : PI_ERR_INVALID_ARG;
}

pi_status_t check_batch(const pi_kv_t *h, const int32_t *seqs, const int32_t *start, int32_t n)
{
    pi_status_t s;
    if ((s = check_ptr(seqs, (size_t)n * 4, 4, h->dev))) return s;
    return check_ptr(start, ((size_t)n + 1) * 4, 4, h->dev);
}

// [n_tokens x width] elements of es bytes, rows ld elements apart, all on 16-byte boundaries.
pi_status_t check_rows(const pi_kv_t *h, const void *p, int64_t n_tokens, int64_t width, int64_t ld, int es)
{
    // (rows beyond any memory first: (n_tokens - 1) * ld * es has to stay a 64-bit number)
    if (ld < width || ld > ((int64_t)1 << 60) / n_tokens || (ld * es) % 16) return PI_ERR_INVALID_ARG;
    return check_ptr(p, (size_t)(((n_tokens - 1) * ld + width) * es), 16, h->dev);
}

int elt_size(int32_t dtype) { return dtype == PI_F32 ? 4 : dtype == PI_BF16 || dtype == PI_F16 ? 2 : 0; }

}  // namespace

extern "C" {

pi_status_t pi_kv_create(pi_kv_t **out, const pi_kv_desc_t *desc, const pi_kv_layer_t *layers,
                         const pi_kv_state_t *state)
{
    if (!out) return PI_ERR_INVALID_ARG;
    *out = nullptr;
    try {
        return kv_create(out, desc, layers, state);
    } catch (const std::bad_alloc &) {
        return PI_ERR_OOM;
    } catch (...) {
        return PI_ERR_CUDA;
    }
}

void pi_kv_destroy(pi_kv_t *h)
{
    if (!h) return;
    cudaDeviceSynchronize();
    cudaFree(h->ws);
    cudaGetLastError();
    delete h;
}

pi_status_t pi_kv_get_status(pi_kv_t *h)
{
    if (!h) return PI_ERR_INVALID_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return cuda_status(cudaGetLastError());
    uint32_t v = 0;
    pi_status_t s;
    if ((s = cuda_status(cudaMemcpy(&v, h->status, 4, cudaMemcpyDeviceToHost)))) return s;
    if (v && (s = cuda_status(cudaMemset(h->status, 0, 4)))) return s;
    // a kernel that gave up between its tickets leaves them: start the next call clean
    if (v == PI_ERR_TIMEOUT && (s = cuda_status(cudaMemset(h->tickets, 0, 3 * up((size_t)h->nsm * 4))))) return s;
    return (pi_status_t)v;
}

pi_status_t pi_kv_reserve(pi_kv_t *h, const int32_t *seqs, const int32_t *tok_start, int32_t n, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    if (n == 0) return PI_OK;
    if ((s = check_batch(h, seqs, tok_start, n))) return s;
    return cuda_status(launch_kv_reserve(h->view, {seqs, tok_start, n, INT32_MAX}, h->list_dst, (cudaStream_t)stream));
}

pi_status_t pi_kv_append(pi_kv_t *h, int32_t layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
                         int32_t n_tokens, const void *k_new, const void *v_new, int64_t ld, int32_t dtype,
                         void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    const int es = elt_size(dtype);
    if (layer < 0 || layer >= h->desc.n_layers || n_tokens < 0 || n_tokens > KV_MAX_LEN || !es) return PI_ERR_INVALID_ARG;
    if (n == 0 || n_tokens == 0) return PI_OK;
    if ((s = check_batch(h, seqs, tok_start, n))) return s;
    const int64_t width = (int64_t)h->desc.n_kv_heads * h->desc.head_dim;
    if ((s = check_rows(h, k_new, n_tokens, width, ld, es))) return s;
    if ((s = check_rows(h, v_new, n_tokens, width, ld, es))) return s;
    return cuda_status(launch_kv_append(h->view, {seqs, tok_start, n, n_tokens}, h->layers[layer], k_new, v_new, ld,
                                        dtype, h->nsm, (cudaStream_t)stream));
}

pi_status_t pi_kv_attend(pi_kv_t *h, int32_t layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
                         int32_t n_tokens, const void *q, int64_t ld_q, void *out, int64_t ld_out, float *lse,
                         int32_t dtype, float scale, int32_t window, int32_t sinks, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    const int es = elt_size(dtype);
    const double scale_log2 = (double)scale * 1.4426950408889634;
    if (layer < 0 || layer >= h->desc.n_layers || n_tokens < 0 || n_tokens > KV_MAX_LEN || !es || sinks < 0 ||
        !(std::fabs(scale_log2) <= (double)FLT_MAX))   // (a NaN scale fails too)
        return PI_ERR_INVALID_ARG;
    if (n == 0 || n_tokens == 0) return PI_OK;
    if ((s = check_batch(h, seqs, tok_start, n))) return s;
    const int64_t width = (int64_t)h->desc.n_heads * h->desc.head_dim;
    if ((s = check_rows(h, q, n_tokens, width, ld_q, es))) return s;
    if ((s = check_rows(h, out, n_tokens, width, ld_out, es))) return s;
    if (lse && (s = check_ptr(lse, (size_t)n_tokens * h->desc.n_heads * 4, 4, h->dev))) return s;
    KvAttendArgs a;
    a.c = h->view;
    a.b = {seqs, tok_start, n, n_tokens};
    a.l = h->layers[layer];
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.ldq = ld_q;
    a.ldo = ld_out;
    a.dtype = dtype;
    a.scale_log2 = (float)scale_log2;
    // no window: one that is never shorter than the distance of two positions (all below 2^30)
    a.window = window > 0 ? std::min(window, KV_MAX_LEN) : KV_MAX_LEN;
    a.sinks = std::min(sinks, KV_MAX_LEN);
    a.part = h->part;
    a.part_ml = h->part_ml;
    a.tickets = h->tickets;
    a.rows_part = h->rows_part;
    a.rows_ml = h->rows_ml;
    a.rows_tickets = h->rows_tickets;
    const auto run = h->desc.head_dim == 64 ? attend_of<64> : h->desc.head_dim == 128 ? attend_of<128> : attend_of<256>;
    return cuda_status(run(h, layer, a, (cudaStream_t)stream));
}

pi_status_t pi_kv_fork(pi_kv_t *h, const int32_t *src, const int32_t *dst, int32_t n, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    if (n == 0) return PI_OK;
    if ((s = check_ptr(src, (size_t)n * 4, 4, h->dev))) return s;
    if ((s = check_ptr(dst, (size_t)n * 4, 4, h->dev))) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const KvCopyList l{h->list_src, h->list_dst, h->list_count};
    if ((s = cuda_status(launch_kv_fork(h->view, src, dst, n, l, st)))) return s;
    return cuda_status(launch_kv_copy(h->view, h->layers_dev, l.src, l.dst, l.count, n, nullptr, h->nsm, st));
}

pi_status_t pi_kv_free(pi_kv_t *h, const int32_t *seqs, int32_t n, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    if (n == 0) return PI_OK;
    if ((s = check_ptr(seqs, (size_t)n * 4, 4, h->dev))) return s;
    return cuda_status(launch_kv_free(h->view, seqs, n, (cudaStream_t)stream));
}

pi_status_t pi_kv_trim(pi_kv_t *h, const int32_t *seqs, int32_t n, int32_t window, int32_t sinks, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    if (window < 1 || sinks < 0) return PI_ERR_INVALID_ARG;
    if (n == 0) return PI_OK;
    if ((s = check_ptr(seqs, (size_t)n * 4, 4, h->dev))) return s;
    return cuda_status(launch_kv_trim(h->view, seqs, n, window, sinks, (cudaStream_t)stream));
}

pi_status_t pi_kv_copy_pages(pi_kv_t *h, const int32_t *src, const int32_t *dst, int32_t n, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, 0))) return s;
    if (n < 0 || n > h->desc.n_pages) return PI_ERR_INVALID_ARG;
    if (n == 0) return PI_OK;
    if ((s = check_ptr(src, (size_t)n * 4, 4, h->dev))) return s;
    if ((s = check_ptr(dst, (size_t)n * 4, 4, h->dev))) return s;
    return cuda_status(launch_kv_copy(h->view, h->layers_dev, src, dst, nullptr, n, nullptr, h->nsm,
                                      (cudaStream_t)stream));
}

pi_status_t pi_kv_compact(pi_kv_t *h, int32_t *n_live, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, 0))) return s;
    if (n_live && (s = check_ptr(n_live, 4, 4, h->dev))) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const KvCopyList l{h->list_src, h->list_dst, h->list_count};
    if ((s = cuda_status(launch_kv_compact(h->view, l, h->page_map, n_live, st)))) return s;
    return cuda_status(launch_kv_copy(h->view, h->layers_dev, l.src, l.dst, l.count, h->desc.n_pages / 2, h->page_map,
                                      h->nsm, st));
}

}  // extern "C"
