// pi_kv_device.cuh -- device helpers of the paged-cache kernels (sm_103a).
#pragma once

#include <cuda_bf16.h>

#include "pi_async.cuh"
#include "pi_kv_internal.h"

namespace pi {

// ---------------------------------------------------------------- the ragged batch ----------

struct KvSeq {
    int row, len, start, n;   // table row, tokens held, first row of the call's arrays, new tokens
    int skip;                 // positions below this are another pass's
};

// Sequence i of the call, its fields brought into range; what was out of range is flagged and reads
// as a sequence without new tokens.
// SHARED: in a pass of pi_kv_attend_shared, whose batches may have lengths of their own and positions to skip.
template <bool SHARED = false>
__device__ __forceinline__ KvSeq kv_sequence(const KvView &c, const KvBatch &b, int i, bool flag)
{
    KvSeq s;
    s.row = b.seqs[i];
    const int s0 = b.start[i], s1 = b.start[i + 1];
    bool bad = s.row < 0 || s.row >= c.max_seqs || s0 < 0 || s1 < s0 || s1 > b.n_tokens;
    s.start = s0;
    s.n = s1 - s0;
    s.len = s.skip = 0;
    if (SHARED && b.skip && (b.was[i] != s.row || b.was[b.n + i] != s0 || b.was[b.n + i + 1] != s1)) bad = true;
    if (bad) {
        s.row = s.start = s.n = 0;
    } else {
        s.len = SHARED && b.len ? b.len[i] : c.length[s.row];
        if (s.len < 0 || s.len > c.max_pages * c.page) {
            s.len = s.n = 0;
            bad = true;
        }
        if (SHARED && b.len && s.len == 0) s.n = 0;   // nothing shared
        if (SHARED && b.skip) {
            s.skip = b.skip[i];
            if (s.skip < 0 || s.skip % KV_SHARE || (s.skip > 0 && s.skip > s.len - s.n)) {
                s.skip = s.len = s.n = 0;
                bad = true;
            }
        }
    }
    if (bad && flag) set_status(c.status, ST_DEVICE_CHECK);
    return s;
}

// Whether a block scale is one: a number >= 0. A page in view without one is left out, as an absent page is.
__device__ __forceinline__ bool is_scale(float s) { return s >= 0.f && s <= 3.402823466e38f; }

// ---------------------------------------------------------------- waiting -------------------

// mbar_wait by a whole warp, whose lanes leave it together and with one answer: a lane leaves its own polling loop when it
// has seen the phase, and what follows a wait (tcgen05, mma.sync, movmatrix, bar.sync) takes the warp as one.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// ---------------------------------------------------------------- e4m3 ----------------------

// Two codes (low byte first) as two f16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// The four codes of a word, low bytes first.
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Codes of (lo, hi): nearest, saturated to +-448, NaN kept.
__device__ __forceinline__ uint16_t f32x2_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Whether one of the four codes of w is NaN (all exponent and mantissa bits set).
__device__ __forceinline__ bool e4m3_any_nan(uint32_t w)
{
    return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
}

// The word with 0 for every NaN code.
__device__ __forceinline__ uint32_t e4m3_no_nan(uint32_t w)
{
    const uint32_t n = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // top bit of every NaN code
    return w & ~((n - (n >> 7)) | n);
}

// ---------------------------------------------------------------- numbers -------------------

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// |x|, or 0 where x is infinite or NaN
__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

// (a.x + b.x, a.y + b.y) in one instruction
__device__ __forceinline__ float2 fadd2(float2 a, float2 b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// (x, y) = hi + lo, f16 pairs
__device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 b = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = pack_f16(x - b.x, y - b.y);
}

// 16 consecutive elements of a 16- or 32-bit array (offset in elements, on a 16-byte boundary)
__device__ __forceinline__ void load16(const void *p, int dtype, int64_t at, float (&x)[16])
{
    if (dtype == DT_F32) {
        const uint4 *s = (const uint4 *)((const float *)p + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4];
            unpack<DT_F32>(s[i], v);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * i + e] = v[e];
        }
    } else {
        const uint4 *s = (const uint4 *)((const uint16_t *)p + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v[8];
            if (dtype == DT_BF16) unpack<DT_BF16>(s[i], v);
            else unpack<DT_F16>(s[i], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 * i + e] = v[e];
        }
    }
}

// ---------------------------------------------------------------- block scales --------------

// Smallest e >= KV_MIN_EXP with a <= 448 * 2^e = 1.75 * 2^(8 + e), a finite and >= 0.
__device__ __forceinline__ int block_exponent(float a)
{
    const uint32_t b = __float_as_uint(a);
    const int k = (int)(b >> 23) - 127;   // a = 1.m * 2^k (subnormals land far below KV_MIN_EXP)
    return max(k - 8 + ((b & 0x7fffffu) > 0x600000u), KV_MIN_EXP);
}

// The codes of n words in a unit 1 / f times as large, by `threads` threads th.
__device__ __forceinline__ void recode(uint8_t *codes, int n, float f, int th, int threads)
{
    for (int x = th; x < n; x += threads) {
        const uint32_t w = ((const uint32_t *)codes)[x];
        const uint32_t a0 = e4m3x2_f16x2((uint16_t)w), a1 = e4m3x2_f16x2((uint16_t)(w >> 16));
        const float2 x0 = __half22float2(u32_h2(a0)), x1 = __half22float2(u32_h2(a1));
        ((uint32_t *)codes)[x] = f32x2_e4m3x2(x0.x * f, x0.y * f) | (uint32_t)f32x2_e4m3x2(x1.x * f, x1.y * f) << 16;
    }
}

// ---------------------------------------------------------------- tensor-core product -------

// d += a b: 16 x 8 fp32 += (16 x 16 f16) (16 x 8 f16)
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit elements that the warp holds (row lane / 4, columns 2 (lane % 4) and on), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t word4(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// ---------------------------------------------------------------- TMA -----------------------

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Box at (x, y) of a 2-D tensor map into shared memory; completes on `bar` as transaction bytes.
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *m, int x, int y, uint64_t *bar)
{
    uint32_t d = (uint32_t)__cvta_generic_to_shared(dst), b = (uint32_t)__cvta_generic_to_shared(bar);
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(d),
        "l"(m), "r"(x), "r"(y), "r"(b)
        : "memory");
}

// ---------------------------------------------------------------- tile geometry -------------

// Column of dim that row n + 8 h of value product j stands for (a lane's bytes of a value row, two to a product).
template <int D>
__device__ __forceinline__ int out_col(int j, int n, int h)
{
    return D == 64 ? 8 * n + 2 * j + h : (j >> 3) * 128 + 16 * n + 2 * (j & 7) + h;
}

// Byte of (token, column) inside a swizzled 64-position tile.
template <int D>
__device__ __forceinline__ int tile_byte(int tok, int d)
{
    if (D == 64) return tok * 64 + (((d >> 4) ^ ((tok >> 1) & 3)) << 4) + (d & 15);
    return (d >> 7) * KV_TILE * 128 + tok * 128 + ((((d >> 4) & 7) ^ (tok & 7)) << 4) + (d & 15);
}

template <int N>
__device__ __forceinline__ void poison(float (&acc)[N][4], int j, int e)
{
#pragma unroll
    for (int jj = 0; jj < N; ++jj)
#pragma unroll
        for (int ee = 0; ee < 4; ++ee)
            if (jj == j && ee == e) acc[jj][ee] = __int_as_float(0x7fc00000);
}

// ---------------------------------------------------------------- output --------------------

template <int N>
__device__ __forceinline__ void store_f32(float *p, const float (&f)[N])
{
#pragma unroll
    for (int e = 0; e < N; e += 4) *(float4 *)(p + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
}

// N consecutive outputs (a multiple of 4; 8-byte aligned for 16-bit types) at element `at`.
template <int N>
__device__ __forceinline__ void store_out(const KvAttendArgs &a, int64_t at, const float (&f)[N])
{
    if (a.dtype == DT_F32) {
        store_f32((float *)a.out + at, f);
        return;
    }
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
        if (a.dtype == DT_BF16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            w[e] = *(const uint32_t *)&x;
        } else {
            w[e] = pack_f16(f[2 * e], f[2 * e + 1]);
        }
    }
    uint16_t *p = (uint16_t *)a.out + at;
    if constexpr (N % 8 == 0) {
#pragma unroll
        for (int e = 0; e < N / 2; e += 4) *(uint4 *)(p + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < N / 2; e += 2) *(uint2 *)(p + 2 * e) = make_uint2(w[e], w[e + 1]);
    }
}

// log of a row's sum of exponentials: maximum (or reference) M in base 2, sum S relative to it
__device__ __forceinline__ float row_lse(float M, float S)
{
    return S == 0.f ? -INFINITY : (M + log2f(S)) * 0.6931471805599453f;
}

// Weight of a partial sum s with maximum (or reference) m against the maximum M of all. One whose maximum is -infinity
// counts only where its sum is not 0 (it is NaN then).
__device__ __forceinline__ float part_weight(float m, float s, float M) { return m == -INFINITY ? (s != 0.f ? 1.f : 0.f) : ex2(m - M); }

// Joins a row's numerators o (four columns), maximum M and sum S with the parts that the first pass left of it.
__device__ __forceinline__ void join_prior(const KvAttendArgs &a, int64_t row, int D, int d, float4 &o, float &M, float &S)
{
    const int64_t rows = (int64_t)a.b.n_tokens * a.c.hq;
    const float2 *const ml = (const float2 *)a.prior_ml + row;
    const float *const num = a.prior + row * D + d;
    float top = M;
#pragma unroll 4
    for (int x = 0; x < a.parts; ++x) top = fmaxf(top, __ldcg(ml + x * rows).x);
    const float w0 = part_weight(M, S, top);
    o = make_float4(o.x * w0, o.y * w0, o.z * w0, o.w * w0);
    S *= w0;
    M = top;
#pragma unroll 4
    for (int x = 0; x < a.parts; ++x) {
        const float2 p = __ldcg(ml + x * rows);
        const float w = part_weight(p.x, p.y, top);
        const float4 v = __ldcg((const float4 *)(num + x * rows * D));
        S += w * p.y;
        if (w != 0.f) o.x += v.x * w, o.y += v.y * w, o.z += v.z * w, o.w += v.w * w;   // (an empty part has no numerators)
    }
}

// Four columns (from d) of row `r` (query token r / G, head r % G of kv head h) of the sequence f (table row,
// length, start, new tokens): numerators o over the sum S, and with d = 0 the row's log of the sum.
template <bool SHARED>
__device__ __forceinline__ void store_row(const KvAttendArgs &a, const int4 &f, int h, int G, int D, int r, int d,
                                          float4 o, float M, float S, bool join = false)
{
    const int64_t tok = (int64_t)f.z + r / G;
    const int head = h * G + r % G;
    if (SHARED && a.pass == 1) {   // the row's one part
        const int64_t row = tok * a.c.hq + head, rows = (int64_t)a.b.n_tokens * a.c.hq;
        *(float4 *)(a.prior + row * D + d) = o;
        if (d == 0) {
            *((float2 *)a.prior_ml + row) = make_float2(M, S);
            for (int x = 1; x < a.parts; ++x) *((float2 *)a.prior_ml + row + x * rows) = make_float2(-INFINITY, 0.f);
        }
        return;
    }
    if (SHARED && join) join_prior(a, tok * a.c.hq + head, D, d, o, M, S);
    const float inv = 1.f / S;
    // S = 0: nothing seen. (A NaN sum stays: it is not equal to 0.)
    const float v[4] = {S == 0.f ? 0.f : o.x * inv, S == 0.f ? 0.f : o.y * inv, S == 0.f ? 0.f : o.z * inv,
                        S == 0.f ? 0.f : o.w * inv};
    store_out<4>(a, tok * a.ldo + (int64_t)head * D + d, v);
    if (a.lse && d == 0) a.lse[tok * a.c.hq + head] = row_lse(M, S);
}

__device__ __forceinline__ void store_nan(const KvAttendArgs &a, const int4 &f, int h, int G, int D, int r, int d)
{
    const int64_t at = ((int64_t)f.z + r / G) * a.ldo + (int64_t)(h * G + r % G) * D + d;
    if (a.dtype == DT_F32) ((uint32_t *)a.out)[at] = 0x7fc00000u;
    else ((uint16_t *)a.out)[at] = a.dtype == DT_BF16 ? 0x7fc0u : 0x7e00u;
}

}  // namespace pi
