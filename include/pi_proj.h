/*
 * pi_proj.h -- C ABI of libpi_ffn.so: what a decoder does between its hidden state and its attention on one GB300
 * (sm_103a): projections with 4-bit weights, and the norms of query and key heads with their position rotation. Next
 * to pi_ffn.h (the sparse FFN) and pi_kv.h (the paged cache, whose pi_kv_append_rotated writes rotated keys).
 *
 * Conventions: those of pi_ffn.h, without a handle. Tensor pointers are device pointers of the current device, borrowed;
 * calls validate their arguments on the host before any launch and are asynchronous on `stream`; none allocates,
 * synchronises or keeps anything between calls, so any number may run at once and be captured in graphs; no C++
 * exception crosses the boundary.
 */
#ifndef PI_PROJ_H
#define PI_PROJ_H

#include "pi_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PI_INT4_MAX_ROWS 256

/*
 * y = x W^T (+ bias) (+ add):  y[b, i] = sum_k x[b, k] W[i, k] + bias[i] + add[b, i].
 * W: PI_INT4_G128 as in pi_ffn.h, n rows (up to 2^30) of k elements, k a multiple of 128 up to 2^18: w [n x k/2] bytes (16-byte aligned), s
 * fp16 [n x k/128], the value q * s of its group. bias: fp32 [n] or NULL. x [rows x k], add and y [rows x n] of `dtype`
 * (PI_F32, PI_BF16 or PI_F16), row b at element b * ld of its array; x's base and row stride are multiples of 16 bytes,
 * those of add and y multiples of the element. 0 <= rows <= PI_INT4_MAX_ROWS. add: NULL, or y itself (same address
 * and stride), or an array that y does not touch; y overlaps neither x nor the weights.
 * Products are of the exact integers and x as f16 terms in units of a power of two for each row and group: one term for
 * PI_BF16 and PI_F16 (exact where an element is at least 2^-28 of its group's largest), two for PI_F32 (22 bits of an element,
 * or 2^-39 of its group's largest). Group sums, their scaling, bias and add are fp32; y is rounded to `dtype` once. Infinities
 * and NaN go where the formula takes them, 0 times an infinity too. The same call gives the same bits. (A kernel whose
 * bounded waits run out, which nothing but a fault makes them do, leaves NaN.)
 */
pi_status_t pi_int4_linear(const void *w, const void *s, const float *bias, int32_t n, int32_t k, const void *x,
                           int64_t ld_x, int32_t rows, const void *add, int64_t ld_add, void *y, int64_t ld_y,
                           int32_t dtype, void *stream);

/*
 * The rotation of heads by their position, after an optional norm. For a head x of head_dim elements at position p:
 *   x[j] *= weight[j] / sqrt(mean_j x[j]^2 + eps)                                        where norm is set,
 *   (x[a_i], x[b_i]) becomes amp * (x[a_i] cos - x[b_i] sin, x[b_i] cos + x[a_i] sin) of the angle p * f_i
 * for i < rot_dim / 2, the pairs (a_i, b_i) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) where interleaved is set; elements
 * from rot_dim on are not turned (nor multiplied by amp). turns[i] = round(f_i / (2 pi) * 2^64) mod 2^64: the fraction of
 * a turn that a step of one position makes, so that p * turns[i] mod 2^64 is the angle at any position, far ones too.
 * Arithmetic is fp32 (sums of squares among it), with one rounding at the end.
 */
typedef struct {
    const uint64_t *turns;   /* [rot_dim / 2] device, or NULL with rot_dim = 0 */
    const float *q_norm;     /* [head_dim] device: weights of the queries' norm, NULL: ones */
    const float *k_norm;     /* the same of the keys */
    int32_t rot_dim;         /* a multiple of 16, 0 .. head_dim */
    int32_t interleaved;     /* 0 or 1 */
    int32_t norm;            /* 0 or 1 */
    float amp;               /* finite */
    float eps;               /* finite, >= 0 (looked at where norm is set) */
} pi_rotary_t;

/*
 * q_out = the queries' heads and k_out = the keys' heads, rotated. q, q_out [n_tokens x n_heads x head_dim], k, k_out
 * [n_tokens x n_kv_heads x head_dim] of `dtype` (PI_F32, PI_BF16 or PI_F16), token t at element t * ld of its array (parts
 * of a fused projection need no copy), bases and row strides multiples of 16 bytes; head_dim 64, 128 or 256. n_kv_heads
 * 0: queries only (k and k_out are not looked at); n_heads 0 likewise. pos: int32 [n_tokens] device, any value. An output
 * is its input (same address and stride) or touches no other array of the call. 0 <= n_tokens <= 2^30.
 */
pi_status_t pi_rotate(const pi_rotary_t *rotary, const int32_t *pos, int32_t n_tokens, int32_t n_heads,
                      int32_t n_kv_heads, int32_t head_dim, const void *q, int64_t ld_q, void *q_out, int64_t ld_q_out,
                      const void *k, int64_t ld_k, void *k_out, int64_t ld_k_out, int32_t dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PI_PROJ_H */
