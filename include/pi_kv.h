/*
 * pi_kv.h -- C ABI of libpi_ffn.so: a paged 8-bit key/value cache on one GB300 (sm_103a), the
 * attention that reads it, the append that fills it and the moves of its pages. Next to pi_ffn.h,
 * whose sparse FFN is the other half of a transformer layer's decode step.
 *
 * The cache
 *  - A page holds page_tokens consecutive positions of one sequence, for every layer. Per layer the
 *    caller lends four arrays: k and v, e4m3 (1 sign, 4 exponent, 3 mantissa bits, largest value
 *    448) [n_pages x n_kv_heads x page_tokens x head_dim], and k_scale and v_scale, fp32
 *    [n_pages x n_kv_heads]: the value is code * scale of its page and head, the scale a number >= 0.
 *  - Shared by all layers: table int32 [max_seqs x max_pages] (row s, column c: the page of
 *    positions [c * page_tokens, (c + 1) * page_tokens) of sequence s, -1 for none), length int32
 *    [max_seqs] (tokens held), ref int32 [n_pages] (how many table entries name the page; 0 = free).
 *    A new cache has table = -1, length = 0, ref = 0. Columns at or past a sequence's last page are -1.
 *  - Pages held by more than one sequence are full ones: pi_kv_fork copies a partly filled last page.
 *
 * Conventions
 *  - Those of pi_ffn.h: tensor pointers are device pointers, borrowed; calls are asynchronous on
 *    `stream` and validate their arguments on the host before any launch; errors that kernels find
 *    go to a status word (pi_kv_get_status) and the offending entry is skipped; no C++ exception
 *    crosses the boundary; not thread-safe per handle, and the calls of one handle share its
 *    workspace, so they are ordered on one stream (or by events).
 *  - seqs: int32 [n] device, table rows, 0 <= n <= PI_KV_MAX_CALL_SEQS; tok_start: int32 [n + 1]
 *    device, ascending from 0: sequence i's new tokens are rows tok_start[i] .. tok_start[i + 1] of
 *    the call's token arrays (n_tokens <= 2^30 rows; what lies past them is not touched, and flagged).
 *    Except for pi_kv_attend, a sequence appears at most once in a call.
 *  - A step: pi_kv_reserve once (lengths grow, pages are found), then per layer pi_kv_append and
 *    pi_kv_attend. No call allocates, synchronises or reads back: a step can be captured in a graph.
 */
#ifndef PI_KV_H
#define PI_KV_H

#include "pi_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PI_KV_MAX_CALL_SEQS 1024

typedef struct {
    int32_t n_layers;      /* >= 1 */
    int32_t n_heads;       /* query heads, a multiple of n_kv_heads; query head h reads kv head h / (n_heads / n_kv_heads) */
    int32_t n_kv_heads;    /* >= 1 */
    int32_t head_dim;      /* 64, 128 or 256 */
    int32_t page_tokens;   /* 16, 32, 64 or 128 */
    int32_t n_pages;       /* pages of the pool, >= 1; n_pages * n_kv_heads * page_tokens < 2^31 */
    int32_t max_seqs;      /* rows of the table, >= 1 */
    int32_t max_pages;     /* columns of the table, >= 1; max_pages * page_tokens <= 2^30 */
} pi_kv_desc_t;

typedef struct {
    void *k, *v;               /* e4m3 [n_pages x n_kv_heads x page_tokens x head_dim], 128-byte aligned */
    float *k_scale, *v_scale;  /* [n_pages x n_kv_heads] */
} pi_kv_layer_t;

typedef struct {
    int32_t *table;            /* [max_seqs x max_pages] */
    int32_t *length;           /* [max_seqs] */
    int32_t *ref;              /* [n_pages] */
} pi_kv_state_t;

typedef struct pi_kv pi_kv_t;

/*
 * Create a handle over the caller's pools (host array of n_layers descriptors, copied) and state.
 * Allocates the workspace (partial results of split sequences, page lists, status word) on the
 * current device. On failure *out = NULL: PI_ERR_INVALID_ARG / PI_ERR_UNSUPPORTED / PI_ERR_OOM /
 * PI_ERR_CUDA. PI_FAULT (pi_ffn.h) injects the same host-side failures here.
 */
pi_status_t pi_kv_create(pi_kv_t **out, const pi_kv_desc_t *desc, const pi_kv_layer_t *layers,
                         const pi_kv_state_t *state);

/* Free the workspace and the handle (waits for the device first). NULL is a no-op. */
void pi_kv_destroy(pi_kv_t *h);

/* Wait for all work on the device, return the first kernel-recorded error and clear it. */
pi_status_t pi_kv_get_status(pi_kv_t *h);

/*
 * Room for new tokens: sequence seqs[i] grows by n_i = tok_start[i + 1] - tok_start[i] tokens
 * (length += n_i), and the pages it lacks are taken from the free ones, lowest id first, in the
 * order of the call's sequences and then of positions. Where the pool or the table row is too
 * short for a sequence, it keeps its length and pages (and from the first that the pool cannot
 * serve, so does every later one that needs a page); the status word records PI_ERR_OOM.
 */
pi_status_t pi_kv_reserve(pi_kv_t *h, const int32_t *seqs, const int32_t *tok_start, int32_t n, void *stream);

/*
 * Write the new tokens' keys and values into layer `layer`: sequence i's rows go to its last n_i
 * positions (pi_kv_reserve has made the room). k_new, v_new: [n_tokens x n_kv_heads x head_dim] of
 * dtype PI_F32, PI_BF16 or PI_F16; row t starts at element t * ld (ld >= n_kv_heads * head_dim, so
 * parts of a fused projection need no copy); base and row stride multiples of 16 bytes.
 * Per page and head, with a = max |x| over the call's finite values there:
 *   s_new = 2^e, the smallest power of two with a <= 448 s_new, e >= -120;
 *   s = s_new if the page held nothing before, else max(s_old, s_new);
 *   the page's earlier codes c become rn(c * s_old / s) where s > s_old; new codes are rn(x / s),
 *   saturated to +-448 (an infinity too); NaN stays NaN.
 * With powers of two x / s is exact, so a value is rounded once (again only when its page's scale
 * grows, and then only where the code falls among the subnormals).
 */
pi_status_t pi_kv_append(pi_kv_t *h, int32_t layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
                         int32_t n_tokens, const void *k_new, const void *v_new, int64_t ld, int32_t dtype,
                         void *stream);

/*
 * Attention of each sequence's last n_i tokens over the sequence's cache in layer `layer`. The
 * query at position p (the last n_i positions, in order) sees position j <= p of its sequence when
 *   window <= 0, or p - j < window, or j < sinks
 * and
 *   out = sum_j softmax_j(scale * q . k_j) v_j   over what it sees,  lse = log sum_j exp(scale * q . k_j).
 * A query that sees nothing (its position is negative) gives 0 and -infinity. What no query of the
 * call sees is not read, so it may be absent, stale or NaN; a page that is seen but absent (-1, or
 * no page of the pool), or has for the head a scale that is not a number >= 0, is left out and
 * flagged. q, out: [n_tokens x n_heads x head_dim] of `dtype`
 * (PI_F32, PI_BF16 or PI_F16), row t at element t * ld_q (ld_out); bases and row strides multiples
 * of 16 bytes. lse: fp32 [n_tokens x n_heads] or NULL. scale * log2(e) is
 * finite in fp32. Scores, the softmax's statistics and the output sums are fp32; the output is
 * rounded to `dtype` once. Queries and weights enter the products as f16 terms, the weights in units
 * that follow the largest value scale: two terms (22 bits) for PI_F32, and for PI_F16 where a
 * sequence has few rows (new tokens x heads of a group); else one (11 bits of a weight, while a
 * PI_BF16 or PI_F16 query is exact in one). The sums are divided last: values whose weighted sum over
 * the cache leaves fp32 give infinities.
 * The same call gives the same bits, whatever the GPU does besides (another set of sequences may cut
 * the caches elsewhere).
 */
pi_status_t pi_kv_attend(pi_kv_t *h, int32_t layer, const int32_t *seqs, const int32_t *tok_start, int32_t n,
                         int32_t n_tokens, const void *q, int64_t ld_q, void *out, int64_t ld_out, float *lse,
                         int32_t dtype, float scale, int32_t window, int32_t sinks, void *stream);

/*
 * dst[i] becomes a copy of sequence src[i]: what dst[i] held is given back (as by pi_kv_free), src's
 * full pages are shared (ref + 1), a partly filled last page is copied, whole and in every layer,
 * into the lowest free page (in the order of i). src, dst: int32 [n] device; the dst are distinct
 * and none of them is a src. Where no page is left for the copy dst[i] stays empty (PI_ERR_OOM).
 */
pi_status_t pi_kv_fork(pi_kv_t *h, const int32_t *src, const int32_t *dst, int32_t n, void *stream);

/* Give back the sequences' pages (ref - 1 each, free at 0); their rows become -1, their lengths 0. */
pi_status_t pi_kv_free(pi_kv_t *h, const int32_t *seqs, int32_t n, void *stream);

/*
 * Give back what a window no longer sees: every page of sequence s without one of the first `sinks`
 * positions, whose last position is <= length[s] - window (so that the next token, at position
 * length[s], cannot see it, nor can any later one). Its table entry becomes -1; the length stays.
 * window >= 1, sinks >= 0.
 */
pi_status_t pi_kv_trim(pi_kv_t *h, const int32_t *seqs, int32_t n, int32_t window, int32_t sinks, void *stream);

/*
 * Copy page src[i] to page dst[i] (codes and scales, every layer). Table and ref are not touched.
 * src, dst: int32 [n] device, n >= 0; no dst is a src or another dst. Ids outside the pool are
 * skipped and flagged.
 */
pi_status_t pi_kv_copy_pages(pi_kv_t *h, const int32_t *src, const int32_t *dst, int32_t n, void *stream);

/*
 * Make the pool dense: with m pages in use (ref > 0), the used pages with id >= m move, in
 * ascending order, into the free ids < m, in ascending order; ref and every table entry follow.
 * Afterwards pages [0, m) are the ones in use. n_live: one int32, device, out (m), or NULL.
 */
pi_status_t pi_kv_compact(pi_kv_t *h, int32_t *n_live, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PI_KV_H */
