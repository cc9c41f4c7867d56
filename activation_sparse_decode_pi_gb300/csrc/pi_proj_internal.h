// pi_proj_internal.h -- what the host side of pi_proj.h (pi_proj_api.cu) and its kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>

#include "pi_internal.h"
#include "pi_proj.h"

namespace pi {

// A map for TMA copies of boxes out of `rows` rows of `width` bytes, dense; false: the driver has none (pi_kv_api.cu).
bool encode_bytes(CUtensorMap *m, const void *base, int64_t rows, int64_t width, int box_rows, int box_width, CUtensorMapSwizzle swizzle);

// Lets a kernel have `bytes` of dynamic shared memory on the current device, once for each device (safe from any thread).
template <auto kernel>
cudaError_t allow_smem(int bytes)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (done.load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
    const cudaError_t f = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (f == cudaSuccess) done.fetch_or((uint64_t)1 << dev, std::memory_order_release);
    return f;
}

struct Int4Args {
    const uint8_t *w;      // [n x k/2]
    const __half *s;       // [n x k/128]
    const float *bias;     // [n] or NULL
    const void *x, *add;   // add: or NULL
    void *y;
    int64_t ldx, ldadd, ldy;   // elements
    int n, k, rows;
    // the launch's: warps and CTAs along k, rows of x to a CTA, groups of its share of k at most, boxes of a warp,
    // where the barriers lie
    int kw, cluster, rows_per, groups, slots, bar_at;
};
cudaError_t launch_int4_linear(const Int4Args &a, int dtype, int nsm, cudaStream_t s);   // k <= INT4_MAX_K
constexpr int INT4_MAX_K = 1 << 18;   // a row of x in the shared memory of a cluster
constexpr int INT4_MAX_N = 1 << 30;   // rows of tiles are counted in 32 bits

struct RotaryDev {
    const uint64_t *turns;
    const float *qn, *kn;
    int rot, interleaved, norm;
    float amp, eps;
};

struct RotateArgs {
    RotaryDev r;
    const int32_t *pos;
    const void *q, *k;
    void *qo, *ko;
    int64_t ldq, ldqo, ldk, ldko;   // elements
    int n_tokens, hq, hk;
    int parts;                      // the launch's: warps that share a token's heads
};
cudaError_t launch_rotate(const RotateArgs &a, int dim, int dtype, int nsm, cudaStream_t s);

// The arguments that pi_rotate and pi_kv_append_rotated share (pi_proj_api.cu).
pi_status_t check_rotary(const pi_rotary_t *r, int head_dim, int dev, RotaryDev *out);

// Two strided arrays on the device: es bytes an element, `rows` rows of `width` elements ld apart.
struct Strided {
    const void *p;
    int64_t rows, width, ld;
    int es;
};
bool same_place(const Strided &a, const Strided &b);
// Whether an element of one may be one of the other (parts of one row layout, side by side, are not).
bool may_overlap(const Strided &a, const Strided &b);

}  // namespace pi
