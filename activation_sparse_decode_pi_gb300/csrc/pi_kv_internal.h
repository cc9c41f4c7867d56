// pi_kv_internal.h -- what the paged-cache host side (pi_kv_api.cu) and its kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pi_kv.h"

namespace pi {

constexpr int KV_TILE = 64;        // positions per tile of the attention kernels
constexpr int KV_MAX_LEN = 1 << 30;   // positions of a sequence and tokens of a call: differences stay 32-bit
constexpr int KV_MIN_EXP = -120;   // smallest exponent of a block scale

// The cache as the kernels see it.
struct KvView {
    int n_layers, hq, hkv, dim, page, n_pages, max_seqs, max_pages;
    int32_t *table, *length, *ref;
    uint32_t *status;
};

// One layer's arrays.
struct KvLayerDev {
    uint8_t *k, *v;
    float *ks, *vs;
};

// The call's ragged batch.
struct KvBatch {
    const int32_t *seqs, *start;
    int n, n_tokens;
};

struct KvAttendArgs {
    KvView c;
    KvBatch b;
    KvLayerDev l;
    const void *q;
    void *out;
    float *lse;
    int64_t ldq, ldo;          // elements
    int dtype;
    float scale_log2;          // scale * log2(e)
    int window, sinks;         // window KV_MAX_LEN: none
    float *part;               // partial numerators [2 * grid][rows][dim]
    float *part_ml;            // their running maximum and sum [2 * grid][rows][2]
    uint32_t *tickets;         // [grid], zero on entry, left zero
    int rows_from;             // sequences with at least so many rows (new tokens x heads of a group) go to the
                               // rows kernel, the others to the split kernel
    float *rows_part;          // rows kernel, split items: numerators [items * splits][rows][dim]
    float *rows_ml;            // their references and sums [items * splits][rows][2]
    uint32_t *rows_tickets;    // [items], zero on entry, left zero
};

// The split kernel (pi_kv_split.cuh) of one head dim; QN: runs of 8 rows per tile, T: 16-bit terms.
template <int D, int QN, int T>
cudaError_t split_setup();   // shared-memory opt-in
template <int D, int QN, int T>
cudaError_t split_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int grid, cudaStream_t s);
#define PI_KV_EXTERN(D, QN, T)                       \
    extern template cudaError_t split_setup<D, QN, T>(); \
    extern template cudaError_t split_launch<D, QN, T>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t);
#define PI_KV_EXTERN4(D) PI_KV_EXTERN(D, 1, 1) PI_KV_EXTERN(D, 1, 2) PI_KV_EXTERN(D, 2, 1) PI_KV_EXTERN(D, 2, 2)
PI_KV_EXTERN4(64) PI_KV_EXTERN4(128) PI_KV_EXTERN4(256)
#undef PI_KV_EXTERN4
#undef PI_KV_EXTERN

// The rows kernel (pi_kv_rows.cuh): QT 16-bit terms of queries and weights. items: an upper bound of the
// call's (sequence, kv head, run of rows_per_item rows); splits: parts of each item's cache.
constexpr int rows_per_item(int dim) { return dim == 256 ? 128 : 256; }
template <int D, int QT>
cudaError_t rows_setup();
template <int D, int QT>
cudaError_t rows_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, unsigned items,
                        unsigned splits, cudaStream_t s);
#define PI_KV_EXTERN(D, QT)                        \
    extern template cudaError_t rows_setup<D, QT>(); \
    extern template cudaError_t rows_launch<D, QT>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, unsigned, unsigned, cudaStream_t);
PI_KV_EXTERN(64, 1) PI_KV_EXTERN(64, 2) PI_KV_EXTERN(128, 1)
PI_KV_EXTERN(128, 2) PI_KV_EXTERN(256, 1) PI_KV_EXTERN(256, 2)
#undef PI_KV_EXTERN

cudaError_t launch_kv_append(const KvView &c, const KvBatch &b, const KvLayerDev &l, const void *k_new,
                             const void *v_new, int64_t ld, int dtype, int nsm, cudaStream_t s);

struct KvCopyList {
    int32_t *src, *dst, *count;   // device; count: one int32
};
cudaError_t launch_kv_reserve(const KvView &c, const KvBatch &b, int32_t *list, cudaStream_t s);
cudaError_t launch_kv_fork(const KvView &c, const int32_t *src, const int32_t *dst, int n, const KvCopyList &l,
                           cudaStream_t s);
cudaError_t launch_kv_free(const KvView &c, const int32_t *seqs, int n, cudaStream_t s);
cudaError_t launch_kv_trim(const KvView &c, const int32_t *seqs, int n, int window, int sinks, cudaStream_t s);
cudaError_t launch_kv_compact(const KvView &c, const KvCopyList &l, int32_t *map, int32_t *n_live, cudaStream_t s);
// Copies the listed pages in every layer (layers: device array) and, with map, renames every table entry.
// max_count: an upper bound of *count known to the host.
cudaError_t launch_kv_copy(const KvView &c, const KvLayerDev *layers, const int32_t *src, const int32_t *dst,
                           const int32_t *count, int max_count, const int32_t *map, int nsm, cudaStream_t s);

}  // namespace pi
