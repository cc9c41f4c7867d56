// pi_kv_internal.h -- what the paged-cache host side (pi_kv_api.cu) and its kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pi_kv.h"
#include "pi_proj_internal.h"

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
    const int32_t *len;    // lengths to take in place of the sequences' own, or NULL
    const int32_t *skip;   // positions of each sequence that another pass attends to, or NULL
    const int32_t *was;    // with skip: [n] table rows and [n + 1] starts that the plan was made for
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
    // Attention in two passes (pi_kv_attend_shared): the first leaves every row's numerators, maximum and sum, the second
    // adds them to its own.
    int pass;                  // 0: one pass alone; 1: the first, whose rows all see positions [0, length); 2: the second
    float *prior, *prior_ml;   // [parts][n_tokens x hq][dim], [parts][n_tokens x hq][2]
    int parts;                 // of a row that the first pass has split along its prefix
    bool few;                  // first pass: the rows kernel's items have up to 128 rows
};
constexpr int KV_SHARE = 128;   // a shared prefix is a multiple of this: whole tiles of both kernels, whole pages

// The split kernel (pi_kv_split.cuh) of one head dim; QN: runs of 8 rows per tile, T: 16-bit terms, SHARED: for a pass of
// pi_kv_attend_shared (head dim 256, two terms; the others have pi_kv_short.cuh).
template <int D, int QN, int T, bool SHARED>
cudaError_t split_setup();   // shared-memory opt-in
template <int D, int QN, int T, bool SHARED>
cudaError_t split_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int grid, cudaStream_t s);
#define PI_KV_SPLIT1(WORD, D, QN, T, S)                  \
    WORD template cudaError_t split_setup<D, QN, T, S>(); \
    WORD template cudaError_t split_launch<D, QN, T, S>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t);
#define PI_KV_SPLIT(WORD, D) \
    PI_KV_SPLIT1(WORD, D, 1, 1, false) PI_KV_SPLIT1(WORD, D, 1, 2, false) PI_KV_SPLIT1(WORD, D, 2, 1, false) PI_KV_SPLIT1(WORD, D, 2, 2, false)
#define PI_KV_SPLIT_SHARED(WORD) PI_KV_SPLIT1(WORD, 256, 1, 2, true) PI_KV_SPLIT1(WORD, 256, 2, 2, true)
PI_KV_SPLIT(extern, 64) PI_KV_SPLIT(extern, 128) PI_KV_SPLIT(extern, 256) PI_KV_SPLIT_SHARED(extern)

// The rows kernel (pi_kv_rows.cuh): QT 16-bit terms of queries, and of weights (SHARED: two of these). items: an upper bound of the
// call's (sequence, kv head, run of rows_per_item rows); splits: parts of each item's cache.
constexpr int rows_per_item(int dim, bool few = false) { return dim == 256 || few ? 128 : 256; }
template <int D, int QT, bool SHARED, bool FEW>
cudaError_t rows_setup();
template <int D, int QT, bool SHARED, bool FEW>
cudaError_t rows_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, unsigned items,
                        unsigned splits, cudaStream_t s);
#define PI_KV_ROWS1(WORD, D, QT, S, F)                  \
    WORD template cudaError_t rows_setup<D, QT, S, F>(); \
    WORD template cudaError_t rows_launch<D, QT, S, F>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, unsigned, unsigned, cudaStream_t);
#define PI_KV_ROWS(WORD, D, S) PI_KV_ROWS1(WORD, D, 1, S, false) PI_KV_ROWS1(WORD, D, 2, S, false)
#define PI_KV_ROWS_FEW(WORD, D) PI_KV_ROWS1(WORD, D, 1, true, true) PI_KV_ROWS1(WORD, D, 2, true, true)
PI_KV_ROWS_FEW(extern, 64) PI_KV_ROWS_FEW(extern, 128)
PI_KV_ROWS(extern, 64, false) PI_KV_ROWS(extern, 128, false) PI_KV_ROWS(extern, 256, false)
PI_KV_ROWS(extern, 64, true) PI_KV_ROWS(extern, 128, true) PI_KV_ROWS(extern, 256, true)

// The kernel of few rows behind a shared prefix (pi_kv_short.cuh): head dims 64 and 128, T 16-bit terms of queries, maps of 16-row
// boxes. part, part_ml and
// tickets: [2 * grid][8][dim], [2 * grid][8][2] and [grid] for a grid of SHORT_CTAS * nsm at most.
constexpr int SHORT_CTAS = 4;
template <int D, int T>
cudaError_t short_setup();
template <int D, int T>
cudaError_t short_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int nsm, cudaStream_t s);
#define PI_KV_EXTERN(D, T)                           \
    extern template cudaError_t short_setup<D, T>(); \
    extern template cudaError_t short_launch<D, T>(const KvAttendArgs &, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t);
PI_KV_EXTERN(64, 1) PI_KV_EXTERN(64, 2) PI_KV_EXTERN(128, 1) PI_KV_EXTERN(128, 2)
#undef PI_KV_EXTERN

cudaError_t launch_kv_append(const KvView &c, const KvBatch &b, const KvLayerDev &l, const void *k_new,
                             const void *v_new, int64_t ld, int dtype, int nsm, cudaStream_t s);

struct KvAppendRotArgs {
    KvView c;
    KvBatch b;
    KvLayerDev l;
    RotaryDev r;
    const void *q, *k, *v;
    void *qo;
    int64_t ldq, ldqo, ld;   // elements
    int cap, slices_q, warps;   // the launch's: new tokens of a page at most; CTAs that share a page's queries; warps to one
                                // of its heads
};
cudaError_t launch_kv_append_rot(const KvAppendRotArgs &a, int dtype, int nsm, cudaStream_t s);

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
// plan: see pi_kv_share in pi_kv.h
cudaError_t launch_kv_share(const KvView &c, const KvBatch &b, const int32_t *groups, int n_groups, int32_t *plan, cudaStream_t s);
cudaError_t launch_kv_copy(const KvView &c, const KvLayerDev *layers, const int32_t *src, const int32_t *dst,
                           const int32_t *count, int max_count, const int32_t *map, int nsm, cudaStream_t s);

}  // namespace pi
