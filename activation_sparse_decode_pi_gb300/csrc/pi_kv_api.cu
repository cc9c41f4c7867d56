// pi_kv_api.cu -- host side of the paged-cache C ABI declared in include/pi_kv.h.
//
// Validates every argument before launching anything, owns the workspace (partials of sequences
// whose cache is split over CTAs, page lists, status word) and the tensor maps of the pools.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <new>
#include <vector>

#include "pi_internal.h"
#include "pi_kv_internal.h"

using namespace pi;

struct pi_kv {
    pi_kv_desc_t desc;
    std::vector<KvLayerDev> layers;
    std::vector<CUtensorMap> map_k, map_v, box_k, box_v;   // of 64-position tiles; of 16 rows
    KvView view;
    int dev = 0, nsm = 0;
    void *ws = nullptr;
    float *part = nullptr, *part_ml = nullptr;
    float *rows_part = nullptr, *rows_ml = nullptr, *prior = nullptr, *short_part = nullptr, *short_ml = nullptr;
    uint32_t *tickets = nullptr, *rows_tickets = nullptr, *short_tickets = nullptr, *status = nullptr;
    KvLayerDev *layers_dev = nullptr;
    int32_t *list_src = nullptr, *list_dst = nullptr, *list_count = nullptr, *page_map = nullptr;
};

namespace pi {

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, or NULL
static EncodeFn tensor_map_encoder()
{
    static std::atomic<EncodeFn> found{nullptr};   // (looked up until it is there)
    if (EncodeFn fn = found.load(std::memory_order_relaxed)) return fn;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
        found.store((EncodeFn)p, std::memory_order_relaxed);
        return (EncodeFn)p;
    }
    cudaGetLastError();
    return nullptr;
}

bool encode_bytes(CUtensorMap *m, const void *base, int64_t rows, int64_t width, int box_rows, int box_width, CUtensorMapSwizzle swizzle)
{
    const EncodeFn fn = tensor_map_encoder();
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width};
    const cuuint32_t box[2] = {(cuuint32_t)box_width, (cuuint32_t)box_rows}, one[2] = {1, 1};
    const auto encode = [&]() {
        return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    // a thread that has no context yet: the runtime gives it the device's
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return encode();
}

}  // namespace pi

namespace {

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

// Pool of one layer as rows of head_dim bytes; boxes of one 64-position tile's share of a page (or of `rows` of it) and
// 128 bytes (64 for head_dim 64), swizzled so that the kernels' reads spread over the banks.
bool encode_pool(CUtensorMap *m, const pi_kv_desc_t &d, const void *base, int rows = KV_TILE)
{
    return encode_bytes(m, base, (int64_t)d.n_pages * d.n_kv_heads * d.page_tokens, d.head_dim, std::min(d.page_tokens, rows),
                        std::min(d.head_dim, 128), d.head_dim < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D>
cudaError_t setup_of()
{
    for (cudaError_t e : {split_setup<D, 1, 1, false>(), split_setup<D, 1, 2, false>(), split_setup<D, 2, 1, false>(),
                          split_setup<D, 2, 2, false>(), rows_setup<D, 1, false, false>(), rows_setup<D, 2, false, false>(),
                          rows_setup<D, 1, true, false>(), rows_setup<D, 2, true, false>()})
        if (e != cudaSuccess) return e;
    if constexpr (D <= 128) {
        for (cudaError_t e : {short_setup<D, 1>(), short_setup<D, 2>(), rows_setup<D, 1, true, true>(), rows_setup<D, 2, true, true>()})
            if (e != cudaSuccess) return e;
    } else {
        for (cudaError_t e : {split_setup<D, 1, 2, true>(), split_setup<D, 2, 2, true>()})
            if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Sequences with at least this many rows (new tokens x heads of a group) are worth a 128-row tile. Measured, 16 sequences
// of 4096, 64 query heads on 8, split / rows kernel: 16 rows 45 / 79 us, 32 rows 71 / 83 us, 48 rows 95 / 72 us, 64 rows
// 120 / 73 us; fp32: 32 rows 99 / 118 us, 64 rows 173 / 109 us.
constexpr int ROWS_FROM = 33;

// The kernels of one call: the split kernel for sequences with few rows, the rows kernel for the others.
template <int D, bool SHARED>
cudaError_t attend_of(const pi_kv *h, int layer, KvAttendArgs a, cudaStream_t s)
{
    const int64_t n = a.b.n, group = a.c.hq / a.c.hkv, rows = (int64_t)a.b.n_tokens * group;
    // the host knows the rows' total only: one sequence has them all, and a token each is a decode step
    const bool many = rows >= ROWS_FROM && (n == 1 || a.b.n_tokens > n), few = n > 1 || !many;
    a.rows_from = many ? (few ? ROWS_FROM : 0) : INT32_MAX;
    cudaError_t e = cudaSuccess;
    if constexpr (SHARED && D <= 128) {
        if (few) {
            KvAttendArgs b = a;
            b.part = h->short_part;
            b.part_ml = h->short_ml;
            b.tickets = h->short_tickets;
            const CUtensorMap &bk = h->box_k[layer], &bv = h->box_v[layer];
            e = a.dtype == PI_F32 ? short_launch<D, 2>(b, bk, bv, h->nsm, s) : short_launch<D, 1>(b, bk, bv, h->nsm, s);
        }
    } else if (few) {
        // 16 rows to a tile where the rows of a sequence (on average: all that the host knows) fill more than 8: the cache
        // is then read once instead of twice (64 sequences, 16 heads to a group: 229 / 323 us with 16 / 8; 8 heads, 128
        // sequences: 381 / 330 us, since 16 leave room for fewer warps)
        const bool wide = (many && !SHARED) || rows > 8 * n;
        auto run = wide ? split_launch<D, 2, 2, SHARED> : split_launch<D, 1, 2, SHARED>;
        if constexpr (!SHARED)
            if (a.dtype == PI_BF16) run = wide ? split_launch<D, 2, 1, false> : split_launch<D, 1, 1, false>;
        e = run(a, h->map_k[layer], h->map_v[layer], h->nsm, s);
    }
    if (many && e == cudaSuccess) {
        // (sequence, kv head, run of rows): at most one partly filled run to each sequence that has ROWS_FROM rows
        const int64_t runs = rows / rows_per_item(D, a.few), items = (runs + n) * a.c.hkv;
        const int64_t grid = a.rows_from ? std::min(runs + n, rows / a.rows_from) * a.c.hkv : items;
        int64_t splits = items < h->nsm ? std::min<int64_t>(16, 2 * h->nsm / items) : 1;
        if (a.pass == 1) splits = a.parts;
        const CUtensorMap &mk = h->map_k[layer], &mv = h->map_v[layer];
        if constexpr (SHARED && D <= 128)
            if (a.few) {
                const auto run = a.dtype == PI_F32 ? rows_launch<D, 2, true, true> : rows_launch<D, 1, true, true>;
                return run(a, mk, mv, (unsigned)grid, (unsigned)splits, s);
            }
        e = a.dtype == PI_F32 ? rows_launch<D, 2, SHARED, false>(a, mk, mv, (unsigned)grid, (unsigned)splits, s)
                              : rows_launch<D, 1, SHARED, false>(a, mk, mv, (unsigned)grid, (unsigned)splits, s);
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
    h->box_k.resize(d.n_layers);
    h->box_v.resize(d.n_layers);
    for (int l = 0; l < d.n_layers; ++l) {
        h->layers.push_back({(uint8_t *)layers[l].k, (uint8_t *)layers[l].v, layers[l].k_scale, layers[l].v_scale});
        if (!encode_pool(&h->map_k[l], d, layers[l].k) || !encode_pool(&h->map_v[l], d, layers[l].v) ||
            !encode_pool(&h->box_k[l], d, layers[l].k, 16) || !encode_pool(&h->box_v[l], d, layers[l].v, 16))
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
    const size_t prior = up((size_t)nsm * rows_per_item(d.head_dim) * (d.head_dim + 2) * 4);
    // (head dim 256 has no such kernel)
    const size_t shorts = d.head_dim <= 128 ? (size_t)SHORT_CTAS * nsm : 0, spart = up(2 * shorts * 8 * d.head_dim * 4), sml = up(2 * shorts * 8 * 2 * 4);
    const size_t total = 3 * list + part + ml + rpart + rml + prior + spart + sml + (3 + SHORT_CTAS) * tick + lay + 2 * 256;
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
    h->prior = (float *)take(prior);
    h->short_part = (float *)take(spart);
    h->short_ml = (float *)take(sml);
    h->tickets = (uint32_t *)take(tick);
    h->rows_tickets = (uint32_t *)take(2 * tick);
    h->short_tickets = (uint32_t *)take(SHORT_CTAS * tick);
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

int elt_size(int32_t dtype) { return dtype == PI_F32 ? 4 : dtype == PI_BF16 || dtype == PI_F16 ? 2 : 0; }

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

// `bytes` of memory as an array
Strided flat(const void *p, int64_t bytes) { return {p, 1, bytes, bytes, 1}; }

// Whether an element of x may be one of the others', or of what the call reads besides: its batch, the handle's state and, of a
// layer, the pools.
bool touches(const pi_kv_t *h, const Strided &x, int layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
             std::initializer_list<Strided> others)
{
    const pi_kv_desc_t &d = h->desc;
    const int64_t blocks = (int64_t)d.n_pages * d.n_kv_heads, pool = blocks * d.page_tokens * d.head_dim;
    for (const Strided &o : others)
        if (may_overlap(x, o)) return true;
    for (const Strided &o : {flat(seqs, n * 4ll), flat(tok_start, n * 4ll + 4), flat(h->view.table, (int64_t)d.max_seqs * d.max_pages * 4),
                             flat(h->view.length, d.max_seqs * 4ll), flat(h->view.ref, d.n_pages * 4ll)})
        if (may_overlap(x, o)) return true;
    if (layer < 0) return false;
    const KvLayerDev &l = h->layers[layer];
    for (const Strided &o : {flat(l.k, pool), flat(l.v, pool), flat(l.ks, blocks * 4), flat(l.vs, blocks * 4)})
        if (may_overlap(x, o)) return true;
    return false;
}

// The arguments of an attention, checked; a is filled where there is something to do.
pi_status_t attend_args(const pi_kv_t *h, int32_t layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
                        int32_t n_tokens, const void *q, int64_t ld_q, void *out, int64_t ld_out, float *lse, int32_t dtype,
                        float scale, int32_t window, int32_t sinks, KvAttendArgs *to)
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
    KvAttendArgs &a = *to;
    a.c = h->view;
    a.b = {seqs, tok_start, n, n_tokens, nullptr, nullptr, nullptr};
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
    return PI_OK;
}

cudaError_t attend(const pi_kv_t *h, int32_t layer, const KvAttendArgs &a, cudaStream_t s)
{
    const int d = h->desc.head_dim;
    const auto run = a.pass ? (d == 64 ? attend_of<64, true> : d == 128 ? attend_of<128, true> : attend_of<256, true>)
                            : (d == 64 ? attend_of<64, false> : d == 128 ? attend_of<128, false> : attend_of<256, false>);
    return run(h, layer, a, s);
}

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
    if (v == PI_ERR_TIMEOUT && (s = cuda_status(cudaMemset(h->tickets, 0, (3 + SHORT_CTAS) * up((size_t)h->nsm * 4))))) return s;
    return (pi_status_t)v;
}

pi_status_t pi_kv_reserve(pi_kv_t *h, const int32_t *seqs, const int32_t *tok_start, int32_t n, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    if (n == 0) return PI_OK;
    if ((s = check_batch(h, seqs, tok_start, n))) return s;
    return cuda_status(launch_kv_reserve(h->view, {seqs, tok_start, n, INT32_MAX, nullptr, nullptr, nullptr}, h->list_dst, (cudaStream_t)stream));
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
    return cuda_status(launch_kv_append(h->view, {seqs, tok_start, n, n_tokens, nullptr, nullptr, nullptr}, h->layers[layer], k_new, v_new, ld,
                                        dtype, h->nsm, (cudaStream_t)stream));
}

pi_status_t pi_kv_append_rotated(pi_kv_t *h, int32_t layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
                                 int32_t n_tokens, const pi_rotary_t *rotary, const void *q, int64_t ld_q, void *q_out,
                                 int64_t ld_q_out, const void *k_new, const void *v_new, int64_t ld, int32_t dtype,
                                 void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    const int es = elt_size(dtype);
    if (layer < 0 || layer >= h->desc.n_layers || n_tokens < 0 || n_tokens > KV_MAX_LEN || !es) return PI_ERR_INVALID_ARG;
    KvAppendRotArgs a = {};
    if ((s = check_rotary(rotary, h->desc.head_dim, h->dev, &a.r))) return s;
    if (n == 0 || n_tokens == 0) return PI_OK;
    if ((s = check_batch(h, seqs, tok_start, n))) return s;
    const int64_t width = (int64_t)h->desc.n_kv_heads * h->desc.head_dim, wide = (int64_t)h->desc.n_heads * h->desc.head_dim;
    if ((s = check_rows(h, k_new, n_tokens, width, ld, es))) return s;
    if ((s = check_rows(h, v_new, n_tokens, width, ld, es))) return s;
    if ((s = check_rows(h, q, n_tokens, wide, ld_q, es))) return s;
    if ((s = check_rows(h, q_out, n_tokens, wide, ld_q_out, es))) return s;
    const Strided sq{q, n_tokens, wide, ld_q, es}, so{q_out, n_tokens, wide, ld_q_out, es};
    const Strided sk{k_new, n_tokens, width, ld, es}, sv{v_new, n_tokens, width, ld, es};
    if ((!same_place(sq, so) && may_overlap(sq, so)) ||
        touches(h, so, layer, seqs, tok_start, n,
                {sk, sv, flat(a.r.turns, a.r.rot * 4ll), flat(a.r.norm ? a.r.qn : nullptr, h->desc.head_dim * 4ll),
                 flat(a.r.norm ? a.r.kn : nullptr, h->desc.head_dim * 4ll)}))
        return PI_ERR_INVALID_ARG;
    a.c = h->view;
    a.b = {seqs, tok_start, n, n_tokens, nullptr, nullptr, nullptr};
    a.l = h->layers[layer];
    a.q = q;
    a.k = k_new;
    a.v = v_new;
    a.qo = q_out;
    a.ldq = ld_q;
    a.ldqo = ld_q_out;
    a.ld = ld;
    return cuda_status(launch_kv_append_rot(a, dtype, h->nsm, (cudaStream_t)stream));
}

pi_status_t pi_kv_attend(pi_kv_t *h, int32_t layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
                         int32_t n_tokens, const void *q, int64_t ld_q, void *out, int64_t ld_out, float *lse,
                         int32_t dtype, float scale, int32_t window, int32_t sinks, void *stream)
{
    pi_status_t s;
    KvAttendArgs a = {};
    if ((s = attend_args(h, layer, seqs, tok_start, n, n_tokens, q, ld_q, out, ld_out, lse, dtype, scale, window, sinks, &a)))
        return s;
    if (n == 0 || n_tokens == 0) return PI_OK;
    return cuda_status(attend(h, layer, a, (cudaStream_t)stream));
}

pi_status_t pi_kv_share(pi_kv_t *h, const int32_t *seqs, const int32_t *tok_start, int32_t n, const int32_t *group_start,
                        int32_t n_groups, int32_t *plan, void *stream)
{
    pi_status_t s;
    if ((s = check_call(h, n))) return s;
    if (n_groups < 0 || n_groups > n) return PI_ERR_INVALID_ARG;
    if (n == 0) return PI_OK;
    if ((s = check_batch(h, seqs, tok_start, n))) return s;
    if ((s = check_ptr(group_start, ((size_t)n_groups + 1) * 4, 4, h->dev))) return s;
    if ((s = check_ptr(plan, (size_t)PI_KV_SHARE_INTS(n, n_groups) * 4, 4, h->dev))) return s;
    if (touches(h, flat(plan, PI_KV_SHARE_INTS(n, n_groups) * 4ll), -1, seqs, tok_start, n, {flat(group_start, n_groups * 4ll + 4)}))
        return PI_ERR_INVALID_ARG;
    return cuda_status(launch_kv_share(h->view, {seqs, tok_start, n, KV_MAX_LEN, nullptr, nullptr, nullptr}, group_start,
                                       n_groups, plan, (cudaStream_t)stream));
}

pi_status_t pi_kv_attend_shared(pi_kv_t *h, int32_t layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
                                int32_t n_tokens, const int32_t *plan, int32_t n_groups, const void *q, int64_t ld_q,
                                void *out, int64_t ld_out, float *lse, int32_t dtype, float scale, void *work, void *stream)
{
    pi_status_t s;
    KvAttendArgs a = {};
    if (n_groups < 0 || n_groups > n) return PI_ERR_INVALID_ARG;
    if ((s = attend_args(h, layer, seqs, tok_start, n, n_tokens, q, ld_q, out, ld_out, lse, dtype, scale, 0, 0, &a))) return s;
    if (n == 0 || n_tokens == 0) return PI_OK;
    if ((s = check_ptr(plan, (size_t)PI_KV_SHARE_INTS(n, n_groups) * 4, 4, h->dev))) return s;
    const int64_t rows = (int64_t)n_tokens * h->desc.n_heads;
    if ((s = check_ptr(work, (size_t)rows * (h->desc.head_dim + 2) * 4, 16, h->dev))) return s;
    // Prefixes of many rows are split along their positions over what the GPU holds (at most one partly filled run of rows
    // to each group but one); their parts lie in the workspace then, which has room for them: parts * most * run <= nsm * 256.
    const int64_t group_rows = (int64_t)n_tokens * (h->desc.n_heads / h->desc.n_kv_heads);
    // Up to 128 rows to a group on average take items of 128 rows (measured, 8 prefixes of 36 rows, 40 heads of 128, fp16, the
    // whole call: 247 us, with items of 256 rows 315 us; fp32 330 and 326).
    const bool few = h->desc.head_dim <= 128 && group_rows <= (int64_t)128 * n_groups;
    const int64_t run = rows_per_item(h->desc.head_dim, few), most = ((group_rows + run - 1) / run + n_groups - 1) * h->desc.n_kv_heads;
    a.parts = n_groups > 0 && group_rows >= ROWS_FROM ? (int)std::max<int64_t>(1, std::min<int64_t>(16, h->nsm / most)) : 1;
    const int64_t wide = (int64_t)h->desc.n_heads * h->desc.head_dim;
    const int es = elt_size(dtype);
    const Strided sq{q, n_tokens, wide, ld_q, es}, so{out, n_tokens, wide, ld_out, es}, sl = flat(lse, rows * 4),
        sp = flat(plan, PI_KV_SHARE_INTS(n, n_groups) * 4ll);
    if ((!same_place(sq, so) && may_overlap(sq, so)) || touches(h, so, layer, seqs, tok_start, n, {sl, sp}) ||
        touches(h, sl, layer, seqs, tok_start, n, {sq, sp}) ||
        touches(h, flat(work, rows * (h->desc.head_dim + 2) * 4), layer, seqs, tok_start, n, {sq, so, sl, sp}))
        return PI_ERR_INVALID_ARG;
    a.prior = a.parts > 1 ? h->prior : (float *)work;
    a.prior_ml = a.prior + a.parts * rows * h->desc.head_dim;
    const int32_t *lead = plan, *start = lead + n_groups, *len = start + n_groups + 1, *skip = len + n_groups, *was = skip + n;
    if (n_groups > 0) {
        KvAttendArgs first = a;
        first.pass = 1;
        first.few = few;
        first.b = {lead, start, n_groups, n_tokens, len, nullptr, nullptr};
        if ((s = cuda_status(attend(h, layer, first, (cudaStream_t)stream)))) return s;
    }
    a.pass = 2;
    a.b.skip = skip;
    a.b.was = was;
    return cuda_status(attend(h, layer, a, (cudaStream_t)stream));
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
