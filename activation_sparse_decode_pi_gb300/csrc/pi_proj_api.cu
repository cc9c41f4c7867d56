// pi_proj_api.cu -- host side of the C ABI declared in include/pi_proj.h: validates every argument before launching.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pi_proj_internal.h"

using namespace pi;

namespace {

pi_status_t cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return PI_OK;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? PI_ERR_OOM : PI_ERR_CUDA;
}

int elt_size(int32_t dtype) { return dtype == PI_F32 ? 4 : dtype == PI_BF16 || dtype == PI_F16 ? 2 : 0; }

// Bytes that `rows` rows of `width` elements of es bytes, ld elements apart, take up; -1 where no memory is that large.
int64_t extent(int64_t rows, int64_t width, int64_t ld, int es)
{
    if (ld < width || ld > ((int64_t)1 << 60) / rows) return -1;
    return ((rows - 1) * ld + width) * es;
}

}  // namespace

namespace pi {

bool same_place(const Strided &a, const Strided &b) { return a.p == b.p && (a.ld == b.ld || (a.rows == 1 && b.rows == 1)); }

bool may_overlap(const Strided &a, const Strided &b)
{
    if (!a.p || !b.p || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    const uintptr_t nx = (uintptr_t)(((a.rows - 1) * a.ld + a.width) * a.es), ny = (uintptr_t)(((b.rows - 1) * b.ld + b.width) * b.es);
    if (x >= y + ny || y >= x + nx) return false;
    if (a.ld * a.es != b.ld * b.es) return true;
    // rows of one stride: where b's begin within a's
    const int64_t ld = a.ld * a.es, wa = a.width * a.es, wb = b.width * b.es;
    const int64_t at = x <= y ? (int64_t)((y - x) % (uintptr_t)ld) : (ld - (int64_t)((x - y) % (uintptr_t)ld)) % ld;
    return at < wa || at + wb > ld;
}

pi_status_t check_rotary(const pi_rotary_t *r, int head_dim, int dev, RotaryDev *out)
{
    if (!r || r->rot_dim < 0 || r->rot_dim > head_dim || (r->interleaved & ~1) || (r->norm & ~1) || !std::isfinite(r->amp))
        return PI_ERR_INVALID_ARG;
    if (r->norm && !(std::isfinite(r->eps) && r->eps >= 0.f)) return PI_ERR_INVALID_ARG;
    if (r->rot_dim % 16) return PI_ERR_UNSUPPORTED;
    pi_status_t s;
    if (r->rot_dim > 0 && (s = check_ptr(r->turns, (size_t)r->rot_dim / 2 * 8, 8, dev))) return s;
    if (r->norm && r->q_norm && (s = check_ptr(r->q_norm, (size_t)head_dim * 4, 4, dev))) return s;
    if (r->norm && r->k_norm && (s = check_ptr(r->k_norm, (size_t)head_dim * 4, 4, dev))) return s;
    *out = {r->turns, r->q_norm, r->k_norm, r->rot_dim, r->interleaved, r->norm, r->amp, r->eps};
    return PI_OK;
}

}  // namespace pi

extern "C" {

pi_status_t pi_int4_linear(const void *w, const void *s, const float *bias, int32_t n, int32_t k, const void *x,
                           int64_t ld_x, int32_t rows, const void *add, int64_t ld_add, void *y, int64_t ld_y,
                           int32_t dtype, void *stream)
{
    const int es = elt_size(dtype);
    if (n < 1 || k < 1 || rows < 0 || rows > PI_INT4_MAX_ROWS || !es) return PI_ERR_INVALID_ARG;
    if (k % 128 || k > INT4_MAX_K || n > INT4_MAX_N) return PI_ERR_UNSUPPORTED;
    if (rows == 0) return PI_OK;
    const int64_t nw = (int64_t)n * (k / 2), ns = (int64_t)n * (k / 128) * 2;
    const int64_t nx = extent(rows, k, ld_x, es), ny = extent(rows, n, ld_y, es), na = add ? extent(rows, n, ld_add, es) : 0;
    if (nx < 0 || ny < 0 || na < 0 || (ld_x * es) % 16) return PI_ERR_INVALID_ARG;
    int dev = 0, nsm = 0;
    pi_status_t st;
    if ((st = cuda_status(cudaGetDevice(&dev)))) return st;
    if ((st = cuda_status(cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))) return st;
    if ((st = check_ptr(w, (size_t)nw, 16, dev))) return st;
    if ((st = check_ptr(s, (size_t)ns, 2, dev))) return st;
    if (bias && (st = check_ptr(bias, (size_t)n * 4, 4, dev))) return st;
    if ((st = check_ptr(x, (size_t)nx, 16, dev))) return st;
    if (add && (st = check_ptr(add, (size_t)na, es, dev))) return st;
    if ((st = check_ptr(y, (size_t)ny, es, dev))) return st;
    const Strided sy{y, rows, n, ld_y, es}, sa{add, rows, n, ld_add, es};
    for (const Strided &in : {Strided{x, rows, k, ld_x, es}, Strided{w, 1, nw, nw, 1}, Strided{s, 1, ns, ns, 1},
                              Strided{bias, 1, n, n, 4}})
        if (may_overlap(sy, in)) return PI_ERR_INVALID_ARG;
    if (add && !same_place(sy, sa) && may_overlap(sy, sa)) return PI_ERR_INVALID_ARG;
    Int4Args a = {};
    a.w = (const uint8_t *)w;
    a.s = (const __half *)s;
    a.bias = bias;
    a.x = x;
    a.add = add;
    a.y = y;
    a.ldx = ld_x;
    a.ldadd = ld_add;
    a.ldy = ld_y;
    a.n = n;
    a.k = k;
    a.rows = rows;
    return cuda_status(launch_int4_linear(a, dtype, nsm, (cudaStream_t)stream));
}

pi_status_t pi_rotate(const pi_rotary_t *rotary, const int32_t *pos, int32_t n_tokens, int32_t n_heads,
                      int32_t n_kv_heads, int32_t head_dim, const void *q, int64_t ld_q, void *q_out, int64_t ld_q_out,
                      const void *k, int64_t ld_k, void *k_out, int64_t ld_k_out, int32_t dtype, void *stream)
{
    const int es = elt_size(dtype);
    if (n_tokens < 0 || n_tokens > (1 << 30) || n_heads < 0 || n_kv_heads < 0 || head_dim < 1 || !es) return PI_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || n_heads > (1 << 16) || n_kv_heads > (1 << 16))
        return PI_ERR_UNSUPPORTED;
    int dev = 0, nsm = 0;
    pi_status_t st;
    if ((st = cuda_status(cudaGetDevice(&dev)))) return st;
    RotateArgs a = {};
    if ((st = check_rotary(rotary, head_dim, dev, &a.r))) return st;
    if (n_tokens == 0 || (n_heads == 0 && n_kv_heads == 0)) return PI_OK;
    if ((st = cuda_status(cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))) return st;
    if ((st = check_ptr(pos, (size_t)n_tokens * 4, 4, dev))) return st;
    const Strided all[4] = {{q, n_heads ? n_tokens : 0, (int64_t)n_heads * head_dim, ld_q, es},
                            {q_out, n_heads ? n_tokens : 0, (int64_t)n_heads * head_dim, ld_q_out, es},
                            {k, n_kv_heads ? n_tokens : 0, (int64_t)n_kv_heads * head_dim, ld_k, es},
                            {k_out, n_kv_heads ? n_tokens : 0, (int64_t)n_kv_heads * head_dim, ld_k_out, es}};
    for (const Strided &x : all) {
        if (x.rows == 0) continue;
        const int64_t bytes = extent(x.rows, x.width, x.ld, es);
        if (bytes < 0 || (x.ld * es) % 16) return PI_ERR_INVALID_ARG;
        if ((st = check_ptr(x.p, (size_t)bytes, 16, dev))) return st;
    }
    const Strided read[4] = {{pos, 1, n_tokens, n_tokens, 4}, {a.r.turns, 1, a.r.rot / 2, a.r.rot / 2, 8},
                             {a.r.norm ? a.r.qn : nullptr, 1, head_dim, head_dim, 4}, {a.r.norm ? a.r.kn : nullptr, 1, head_dim, head_dim, 4}};
    for (int i = 1; i < 4; i += 2) {
        for (int j = 0; j < 4; ++j)
            if (j != i && !(j == i - 1 && same_place(all[i], all[j])) && may_overlap(all[i], all[j])) return PI_ERR_INVALID_ARG;
        for (const Strided &x : read)
            if (may_overlap(all[i], x)) return PI_ERR_INVALID_ARG;
    }
    a.pos = pos;
    a.q = q;
    a.qo = q_out;
    a.k = k;
    a.ko = k_out;
    a.ldq = ld_q;
    a.ldqo = ld_q_out;
    a.ldk = ld_k;
    a.ldko = ld_k_out;
    a.n_tokens = n_tokens;
    a.hq = n_heads;
    a.hk = n_kv_heads;
    return cuda_status(launch_rotate(a, head_dim, dtype, nsm, (cudaStream_t)stream));
}

}  // extern "C"
