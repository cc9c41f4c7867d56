// pi_kv_append.cu -- new keys and values into the paged 8-bit cache (sm_103a).
//
// Per page and kv head the block scale is the smallest power of two that brings the largest value to
// at most 448; x / s is then exact and the rounding to e4m3 the only one. W warps own one (page, head)
// of K or V: they read the new rows once for their maximum and keep what fits in registers for the
// codes, so the bytes of the new values bound it. One warp is enough for a decode step's single rows;
// a prompt's whole pages take four, so that a page is one round of loads. Measured: 7 prompts of 1015..3351
// tokens, 8 heads of 128, bf16 31 us = 3.0 TB/s (four warps; 52 us with one), bound by the latency of a page's
// loads, maximum and stores; 64 single tokens of 40 heads, fp32 7.7 us, which is the host's time.
#include <algorithm>

#include "pi_async.cuh"
#include "pi_kv_device.cuh"

namespace pi {

constexpr int AP_NT = 256, AP_NW = AP_NT / 32;
// 16-byte vectors of new values a lane keeps between the two passes, and CTAs that an SM then has room for: a step's
// rows are one or two vectors a lane, and what counts is how many are on their way.
template <int W>
struct AppendCfg {
    static constexpr int BUF = W == 1 ? 2 : 8, CTAS = W == 1 ? 6 : 3;
};

template <int DT, int W>
__global__ void __launch_bounds__(AP_NT, AppendCfg<W>::CTAS) k_kv_append(const KvView c, const KvBatch b, const KvLayerDev l,
                                                     const void *k_new, const void *v_new, int64_t ld)
{
    constexpr int VE = Vec<DT>::N;   // elements of a 16-byte vector
    constexpr int BUF = AppendCfg<W>::BUF;
    __shared__ float s_top[AP_NW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = c.page;
    pdl_wait();
    pdl_launch_dependents();
    // sequence blockIdx.x of the call: every gridDim.y-th of the pages it touches, every gridDim.z-th of their units
    const bool flag = blockIdx.y == 0 && blockIdx.z == 0;
    const KvSeq q = kv_sequence(c, b, blockIdx.x, flag);
    if (q.n == 0) return;
    const int first = q.len - q.n;   // position of the first new token
    if (first < 0) {                 // no room was reserved
        if (flag && tid == 0) set_status(c.status, ST_DEVICE_CHECK);
        return;
    }
    constexpr int ES = 16 / VE, NTH = W * 32;
    const int th = tid % NTH, D = c.dim, vs = __ffs(D / VE) - 1, vm = D / VE - 1, ps = __ffs(P) - 1;
    for (int col = (first >> ps) + blockIdx.y; col <= (q.len - 1) >> ps; col += gridDim.y) {
        const int page = c.table[(size_t)q.row * c.max_pages + col];
        if (page < 0 || page >= c.n_pages) {
            if (tid == 0) set_status(c.status, ST_DEVICE_CHECK);
            continue;
        }
        const int p0 = max(first - col * P, 0), p1 = min(q.len - col * P, P);   // new slots of the page
        const int64_t row0 = (int64_t)q.start + col * P + p0 - first;           // their first row in the call
        // (head, K or V) units: W warps to each
        for (int u = blockIdx.z * (AP_NW / W) + warp / W; u < 2 * c.hkv; u += gridDim.z * (AP_NW / W)) {
            const bool val = u >= c.hkv;
            const int h = val ? u - c.hkv : u;
            const uint8_t *src = (const uint8_t *)(val ? v_new : k_new);
            uint8_t *codes = (val ? l.v : l.k) + ((size_t)page * c.hkv + h) * P * D;
            float *scale = (val ? l.vs : l.ks) + (size_t)page * c.hkv + h;
            const int nv = (p1 - p0) << vs;   // vectors of the block, 2^vs to a row
            auto vec = [&](int v) {
                return *(const uint4 *)(src + ((row0 + (v >> vs)) * ld + h * D + (v & vm) * VE) * ES);
            };

            uint4 buf[BUF];
            float top = 0.f;
            const float was = p0 > 0 ? *scale : 0.f;
#pragma unroll
            for (int x = 0; x < BUF; ++x) {
                const int v = x * NTH + th;
                if (v < nv) buf[x] = vec(v);
            }
#pragma unroll
            for (int x = 0; x < BUF; ++x)
                if (x * NTH + th < nv) {
                    float f[VE];
                    unpack<DT>(buf[x], f);
#pragma unroll
                    for (int e = 0; e < VE; ++e) top = fmaxf(top, finite_abs(f[e]));
                }
#pragma unroll 4
            for (int v = BUF * NTH + th; v < nv; v += NTH) {
                float f[VE];
                unpack<DT>(vec(v), f);
#pragma unroll
                for (int e = 0; e < VE; ++e) top = fmaxf(top, finite_abs(f[e]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if constexpr (W > 1) {   // over the unit's warps (a second barrier ends the unit, so s_top is free again)
                if (lane == 0) s_top[warp] = top;
                bar_sync(1 + warp / W, NTH);
#pragma unroll
                for (int w = 0; w < W; ++w) top = fmaxf(top, s_top[warp / W * W + w]);
            }
            float s = exp2i(block_exponent(top));
            if (p0 > 0) {
                s = fmaxf(was, s);
                if (s > was) recode(codes, p0 * D / 4, was / s, th, NTH);   // the page's earlier codes in the new unit
            }
            if (th == 0 && (p0 == 0 || s > was)) *scale = s;

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
                uint8_t *dst = codes + (p0 + (v >> vs)) * D + (v & vm) * VE;
                if constexpr (VE == 4) *(uint32_t *)dst = w[0];
                else *(uint2 *)dst = make_uint2(w[0], w[1]);
            };
#pragma unroll
            for (int x = 0; x < BUF; ++x)
                if (x * NTH + th < nv) put(x * NTH + th, buf[x]);
#pragma unroll 4
            for (int v = BUF * NTH + th; v < nv; v += NTH) put(v, vec(v));
            if constexpr (W > 1) bar_sync(1 + warp / W, NTH);
        }
    }
}

cudaError_t launch_kv_append(const KvView &c, const KvBatch &b, const KvLayerDev &l, const void *k_new,
                             const void *v_new, int64_t ld, int dtype, int nsm, cudaStream_t s)
{
    // Four warps to a unit where sequences bring 4 tokens or more on average (measured, d 5120 fp32: 64 x 1 tokens 8.2 us
    // with one and 14.3 with four; 7 prompts of ~2000 tokens 52 and 29 us).
    const bool wide = (int64_t)b.n_tokens >= 4 * (int64_t)b.n;
    // pages of a sequence (half as many again as the average has) and units of a page side by side: about two rounds
    // of what the GPU holds
    const int64_t pages = std::min<int64_t>((int64_t)b.n_tokens / c.page + 2, (int64_t)b.n_tokens / ((int64_t)b.n * c.page) * 3 / 2 + 1);
    const int64_t per = AP_NW / (wide ? 4 : 1), most = (2 * c.hkv + per - 1) / per;
    const int64_t fill = std::max<int64_t>(1, (wide ? 12 : 24) * (int64_t)nsm / (pages * b.n));
    Launch L;
    L.grid = dim3((unsigned)b.n, (unsigned)std::min<int64_t>(pages, 65535), (unsigned)std::min(most, fill));
    L.block = dim3(AP_NT);
    L.smem = 0;
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    const auto run = [&](auto one, auto four) {
        return wide ? launch_ex(L, four, c, b, l, k_new, v_new, ld) : launch_ex(L, one, c, b, l, k_new, v_new, ld);
    };
    switch (dtype) {
    case DT_F32: return run(k_kv_append<DT_F32, 1>, k_kv_append<DT_F32, 4>);
    case DT_BF16: return run(k_kv_append<DT_BF16, 1>, k_kv_append<DT_BF16, 4>);
    default: return run(k_kv_append<DT_F16, 1>, k_kv_append<DT_F16, 4>);
    }
}

}  // namespace pi
