// pi_kv_append.cu -- new keys and values into the paged 8-bit cache (sm_103a).
//
// Per page and kv head the block scale is the smallest power of two that brings the largest value to
// at most 448; x / s is then exact and the rounding to e4m3 the only one. One warp owns one (page,
// head) of K or V: it reads the new rows once for their maximum and once to write the codes (from
// registers when they fit), so the bytes of the new values bound it.
#include <algorithm>

#include "pi_kv_device.cuh"

namespace pi {

constexpr int AP_NT = 256, AP_NW = AP_NT / 32;
constexpr int AP_BUF = 8;   // 16-byte vectors of new values a lane keeps between the two passes

// Smallest e >= KV_MIN_EXP with a <= 448 * 2^e = 1.75 * 2^(8 + e), a finite and >= 0.
__device__ __forceinline__ int block_exponent(float a)
{
    const uint32_t b = __float_as_uint(a);
    const int k = (int)(b >> 23) - 127;   // a = 1.m * 2^k (subnormals land far below KV_MIN_EXP)
    return max(k - 8 + ((b & 0x7fffffu) > 0x600000u), KV_MIN_EXP);
}

template <int DT>
__global__ void __launch_bounds__(AP_NT) k_kv_append(const KvView c, const KvBatch b, const KvLayerDev l,
                                                     const void *k_new, const void *v_new, int64_t ld)
{
    constexpr int VE = Vec<DT>::N;   // elements of a 16-byte vector
    __shared__ int wsum[AP_NW], s_i, s_col;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = c.page;
    pdl_wait();
    pdl_launch_dependents();

    // the blockIdx.x-th touched page of the call: sequence s_i, column s_col of its row
    if (tid == 0) s_i = -1;
    __syncthreads();
    int before = 0;
    for (int base = 0; base < b.n && before <= (int)blockIdx.x; base += AP_NT) {
        const int i = base + tid;
        int cnt = 0, first = 0;
        if (i < b.n) {
            const KvSeq q = kv_sequence(c, b, i, blockIdx.x == 0 && blockIdx.y == 0);
            first = (q.len - q.n) / P;
            if (q.n > 0 && q.len >= q.n) cnt = (q.len - 1) / P - first + 1;
            else if (q.n > 0 && blockIdx.x == 0 && blockIdx.y == 0) set_status(c.status, ST_DEVICE_CHECK);
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int at = before + inc - cnt;
        for (int w = 0; w < AP_NW; ++w) {
            at += w < warp ? wsum[w] : 0;
            before += wsum[w];
        }
        if (at <= (int)blockIdx.x && (int)blockIdx.x < at + cnt) {
            s_i = i;
            s_col = first + (int)blockIdx.x - at;
        }
        __syncthreads();
    }
    if (s_i < 0) return;
    const int hv = blockIdx.y * AP_NW + warp;
    if (hv >= 2 * c.hkv) return;
    const bool val = hv >= c.hkv;
    const int h = val ? hv - c.hkv : hv, D = c.dim;
    const KvSeq q = kv_sequence(c, b, s_i, false);
    const int page = c.table[(size_t)q.row * c.max_pages + s_col];
    if (page < 0 || page >= c.n_pages) {
        if (lane == 0) set_status(c.status, ST_DEVICE_CHECK);
        return;
    }
    const int first = q.len - q.n;
    const int p0 = max(first - s_col * P, 0), p1 = min(q.len - s_col * P, P);   // new slots of the page
    const int64_t row0 = (int64_t)q.start + s_col * P + p0 - first;             // their first row in the call
    const uint8_t *src = (const uint8_t *)(val ? v_new : k_new);
    constexpr int ES = 16 / VE;
    uint8_t *codes = (val ? l.v : l.k) + ((size_t)page * c.hkv + h) * P * D;
    float *scale = (val ? l.vs : l.ks) + (size_t)page * c.hkv + h;
    const int vpr = D / VE, nv = (p1 - p0) * vpr;   // vectors of a row, of the block
    auto vec = [&](int v) {
        return *(const uint4 *)(src + ((row0 + v / vpr) * ld + (int64_t)h * D + (v % vpr) * VE) * ES);
    };

    uint4 buf[AP_BUF];
    float top = 0.f;
    const float was = p0 > 0 ? *scale : 0.f;
#pragma unroll
    for (int x = 0; x < AP_BUF; ++x) {
        const int v = x * 32 + lane;
        if (v < nv) buf[x] = vec(v);
    }
#pragma unroll
    for (int x = 0; x < AP_BUF; ++x)
        if (x * 32 + lane < nv) {
            float f[VE];
            unpack<DT>(buf[x], f);
#pragma unroll
            for (int e = 0; e < VE; ++e) top = fmaxf(top, finite_abs(f[e]));
        }
#pragma unroll 4
    for (int v = AP_BUF * 32 + lane; v < nv; v += 32) {
        float f[VE];
        unpack<DT>(vec(v), f);
#pragma unroll
        for (int e = 0; e < VE; ++e) top = fmaxf(top, finite_abs(f[e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float s = exp2i(block_exponent(top));
    if (p0 > 0) {
        s = fmaxf(was, s);
        if (s > was) {   // the page's earlier codes in the new unit
            const float f = was / s;
            for (int x = lane; x < p0 * D / 4; x += 32) {
                const uint32_t w = ((const uint32_t *)codes)[x];
                const uint32_t a0 = e4m3x2_f16x2((uint16_t)w), a1 = e4m3x2_f16x2((uint16_t)(w >> 16));
                const float2 x0 = __half22float2(u32_h2(a0)), x1 = __half22float2(u32_h2(a1));
                ((uint32_t *)codes)[x] =
                    f32x2_e4m3x2(x0.x * f, x0.y * f) | (uint32_t)f32x2_e4m3x2(x1.x * f, x1.y * f) << 16;
            }
        }
    }
    if (lane == 0 && (p0 == 0 || s > was)) *scale = s;

    // x / s: the reciprocal of a power of two is exact (a scale the caller put there may be another number)
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
    const float rcp = 1.f / s;
    auto put = [&](int v, const uint4 &raw) {
        float f[VE];
        unpack<DT>(raw, f);
        uint32_t w[VE / 4];
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = pow2 ? f[e] * rcp : f[e] / s;
#pragma unroll
        for (int e = 0; e < VE / 4; ++e)
            w[e] = f32x2_e4m3x2(f[4 * e], f[4 * e + 1]) | (uint32_t)f32x2_e4m3x2(f[4 * e + 2], f[4 * e + 3]) << 16;
        uint8_t *dst = codes + (size_t)(p0 + v / vpr) * D + (v % vpr) * VE;
        if constexpr (VE == 4) *(uint32_t *)dst = w[0];
        else *(uint2 *)dst = make_uint2(w[0], w[1]);
    };
#pragma unroll
    for (int x = 0; x < AP_BUF; ++x)
        if (x * 32 + lane < nv) put(x * 32 + lane, buf[x]);
#pragma unroll 4
    for (int v = AP_BUF * 32 + lane; v < nv; v += 32) put(v, vec(v));
}

cudaError_t launch_kv_append(const KvView &c, const KvBatch &b, const KvLayerDev &l, const void *k_new,
                             const void *v_new, int64_t ld, int dtype, cudaStream_t s)
{
    // touched pages: at most one per token, and for each sequence a run of whole pages and two ends
    const int64_t pages = std::min<int64_t>(b.n_tokens, b.n_tokens / c.page + 2 * (int64_t)b.n);
    Launch L;
    L.grid = dim3((unsigned)pages, (2 * c.hkv + AP_NW - 1) / AP_NW);
    L.block = dim3(AP_NT);
    L.smem = 0;
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    switch (dtype) {
    case DT_F32: return launch_ex(L, k_kv_append<DT_F32>, c, b, l, k_new, v_new, ld);
    case DT_BF16: return launch_ex(L, k_kv_append<DT_BF16>, c, b, l, k_new, v_new, ld);
    default: return launch_ex(L, k_kv_append<DT_F16>, c, b, l, k_new, v_new, ld);
    }
}

}  // namespace pi
