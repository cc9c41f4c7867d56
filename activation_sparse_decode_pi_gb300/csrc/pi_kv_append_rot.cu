// pi_kv_append_rot.cu -- one pass from a fused projection into the attention: queries and keys normed and rotated by
// their positions, keys and values coded into the paged 8-bit cache (sm_103a).
//
// Each element is read once and written once (a query in its type, a key or value as a code), and those bytes bound it.
// A CTA has the new tokens of one page of one sequence and a slice of their heads. It works out the tokens' cosines and
// sines once, into shared memory; W warps then own one (page, head) of K or V as in pi_kv_append.cu (largest value, block
// scale, codes, what fits in registers between the two); queries go a token to a warp.
#include <algorithm>

#include "pi_rotary.cuh"

namespace pi {

constexpr int AR_NT = 256, AR_NW = AR_NT / 32;
// Groups of eight values that a lane keeps between a block's maximum and its codes, and bytes of the table of cosines and
// sines (tokens past it work theirs out for every head).
template <int W>
struct AppendRotCfg {
    static constexpr int BUF = W == 1 ? 1 : 4, CTAS = 2, TABLE = W == 1 ? 16 * 1024 : 64 * 1024;
};

// turn_cos_sin out of line, for tokens without a place in the table
__device__ __noinline__ float2 turn_cos_sin_call(uint64_t turns, int p, float amp) { return turn_cos_sin(turns, p, amp); }

template <int DT, int D, int W>
__global__ void __launch_bounds__(AR_NT, AppendRotCfg<W>::CTAS) k_kv_append_rot(const KvAppendRotArgs a)
{
    constexpr int LPR = D / 8, BUF = AppendRotCfg<W>::BUF, NTH = W * 32, ES = DT == DT_F32 ? 4 : 2;
    extern __shared__ __align__(16) float table[];   // [a.cap][rot / 2] cosines, then sines
    __shared__ float s_top[AR_NW];
    const KvView &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = c.page;
    pdl_wait();
    pdl_launch_dependents();
    const bool flag = blockIdx.y == 0 && blockIdx.z == 0;
    const KvSeq q = kv_sequence(c, a.b, blockIdx.x, flag);
    if (q.n == 0) return;
    const int first = q.len - q.n;   // position of the first new token
    if (first < 0) {                 // no room was reserved
        if (flag && tid == 0) set_status(c.status, ST_DEVICE_CHECK);
        return;
    }
    const int th = tid % NTH, ps = __ffs(P) - 1, half = a.r.rot / 2, slice = blockIdx.z, slices = gridDim.z;
    const int hq0 = (int)((int64_t)c.hq * slice / slices), hq1 = (int)((int64_t)c.hq * (slice + 1) / slices);
    const RotaryLane l = rotary_lane<D>(a.r, lane);
    float *const cosv = table, *const sinv = table + a.cap * half;
    auto pair_cos_sin = [&](int row, int pos, float2 (&cs)[4]) {   // of the lane's four pairs, at the page's row-th new token
        if (!l.turned) return;
        if (row < a.cap) {
            const float4 c4 = *(const float4 *)(cosv + row * half + l.pair0), s4 = *(const float4 *)(sinv + row * half + l.pair0);
            cs[0] = make_float2(c4.x, s4.x), cs[1] = make_float2(c4.y, s4.y);
            cs[2] = make_float2(c4.z, s4.z), cs[3] = make_float2(c4.w, s4.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) cs[i] = turn_cos_sin_call(a.r.turns[l.pair0 + i], pos, a.r.amp);
        }
    };

    for (int col = (first >> ps) + blockIdx.y; col <= (q.len - 1) >> ps; col += gridDim.y) {
        const int p0 = max(first - col * P, 0), p1 = min(q.len - col * P, P), rows = p1 - p0;   // new slots of the page
        const int pos0 = col * P + p0;
        const int64_t row0 = (int64_t)q.start + pos0 - first;   // their first row in the call
        __syncthreads();   // (the last page's table has been read)
        for (int x = tid; x < min(rows, a.cap) * half; x += AR_NT) {
            const int r = x / half, i = x - r * half;
            const float2 cs = turn_cos_sin(a.r.turns[i], pos0 + r, a.r.amp);
            cosv[x] = cs.x;
            sinv[x] = cs.y;
        }
        __syncthreads();
        int page = c.table[(size_t)q.row * c.max_pages + col];
        if (page < 0 || page >= c.n_pages) {
            if (tid == 0) set_status(c.status, ST_DEVICE_CHECK);
            page = -1;
        }
        // ---------------------------------------------------------------- keys and values: W warps to a head
        for (int u = slice * (AR_NW / W) + warp / W; page >= 0 && u < 2 * c.hkv; u += slices * (AR_NW / W)) {
            const bool val = u >= c.hkv;
            const int h = val ? u - c.hkv : u;
            const uint8_t *src = (const uint8_t *)(val ? a.v : a.k) + (row0 * a.ld + h * D + l.off_a) * ES;
            uint8_t *codes = (val ? a.l.v : a.l.k) + ((size_t)page * c.hkv + h) * P * D;
            float *scale = (val ? a.l.vs : a.l.ks) + (size_t)page * c.hkv + h;
            const int nv = rows * LPR;   // groups of eight of the block
            auto fetch = [&](int v) {
                Eight<DT> raw;
                const uint8_t *const at = src + ((v / LPR) * a.ld) * ES;
                if (v < nv) raw.load(at, at + (l.off_b - l.off_a) * ES);
                else raw.clear();
                return raw;
            };
            auto finish = [&](const Eight<DT> &raw, int v, float2 (&f)[4]) {   // by the whole warp
                if (val) {
                    raw.widen(f);
                    return;
                }
                float2 cs[4];
                const int row = min(v / LPR, rows - 1);
                pair_cos_sin(row, pos0 + row, cs);
                rotate_eight<DT, D>(a.r, l, raw, rotary_coef(a.r, l, a.r.kn, cs), f);
            };
            auto largest = [](float top, const float2 (&f)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(finite_abs(f[e].x), finite_abs(f[e].y)));
                return top;
            };
            float2 buf[BUF][4];
            float top = 0.f;
            const float was = p0 > 0 ? *scale : 0.f;
            const int v0 = th & ~31;   // the warp's first
            constexpr int LD = BUF < 2 ? BUF : 2;   // loads under way at a time
#pragma unroll
            for (int x0 = 0; x0 < BUF; x0 += LD) {
                Eight<DT> raw[LD];
#pragma unroll
                for (int x = 0; x < LD; ++x) raw[x] = fetch((x0 + x) * NTH + th);
#pragma unroll
                for (int x = 0; x < LD; ++x)
                    if ((x0 + x) * NTH + v0 < nv) {
                        finish(raw[x], (x0 + x) * NTH + th, buf[x0 + x]);
                        if ((x0 + x) * NTH + th < nv) top = largest(top, buf[x0 + x]);
                    }
            }
            for (int v = BUF * NTH; v + v0 < nv; v += NTH) {
                float2 f[4];
                finish(fetch(v + th), v + th, f);
                if (v + th < nv) top = largest(top, f);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if constexpr (W > 1) {   // over the unit's warps (a second barrier ends the unit, so s_top is free again)
                if (lane == 0) s_top[warp] = top;
                bar_sync(1 + warp / W, NTH);
#pragma unroll
                for (int y = 0; y < W; ++y) top = fmaxf(top, s_top[warp / W * W + y]);
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
            auto put = [&](int v, float2 (&f)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = pow2 ? fmul2(f[e], make_float2(rcp, rcp)) : make_float2(f[e].x / s, f[e].y / s);
                uint32_t o[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    o[e] = f32x2_e4m3x2(f[2 * e].x, f[2 * e].y) | (uint32_t)f32x2_e4m3x2(f[2 * e + 1].x, f[2 * e + 1].y) << 16;
                if (v < nv) {
                    uint8_t *const to = codes + (size_t)(p0 + v / LPR) * D;
                    *(uint32_t *)(to + l.off_a) = o[0];
                    *(uint32_t *)(to + l.off_b) = o[1];
                }
            };
#pragma unroll
            for (int x = 0; x < BUF; ++x)
                if (x * NTH + v0 < nv) put(x * NTH + th, buf[x]);
            for (int v = BUF * NTH; v + v0 < nv; v += NTH) {
                float2 f[4];
                finish(fetch(v + th), v + th, f);
                put(v + th, f);
            }
            if constexpr (W > 1) bar_sync(1 + warp / W, NTH);
        }
        // ---------------------------------------------------------------- queries: a token to a warp
        for (int t = warp; t < rows; t += AR_NW) {
            float2 cs[4];
            pair_cos_sin(t, pos0 + t, cs);
            rotate_heads<DT, D, W == 1 ? 2 : 4>(a.r, l, rotary_coef(a.r, l, a.r.qn, cs), (const uint8_t *)a.q + (row0 + t) * a.ldq * ES,
                                                (uint8_t *)a.qo + (row0 + t) * a.ldqo * ES, hq0, hq1, lane);
        }
    }
}

namespace {

template <int DT, int D, int W>
cudaError_t launch_of(const KvAppendRotArgs &in, int nsm, cudaStream_t s)
{
    KvAppendRotArgs a = in;
    const int64_t n = a.b.n, T = a.b.n_tokens;
    const int half = a.r.rot / 2, room = half ? AppendRotCfg<W>::TABLE / (half * 8) : 0;
    a.cap = (int)std::min<int64_t>(std::min<int64_t>(a.c.page, T), room);
    // pages of a sequence (half as many again as the average has) and slices of a page's heads: about two rounds of
    // what the GPU holds
    const int64_t pages = std::min<int64_t>(T / a.c.page + 2, T / (n * a.c.page) * 3 / 2 + 1);
    const int64_t per = AR_NW / W, most = std::max<int64_t>((2 * a.c.hkv + per - 1) / per, (a.c.hq + 7) / 8);
    const int64_t fill = std::max<int64_t>(1, (W == 1 ? 16 : 8) * (int64_t)nsm / (pages * n));
    const size_t smem = (size_t)a.cap * half * 8;
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k_kv_append_rot<DT, D, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   AppendRotCfg<W>::TABLE);
        if (e != cudaSuccess) return e;
    }
    Launch L;
    L.grid = dim3((unsigned)n, (unsigned)std::min<int64_t>(pages, 65535), (unsigned)std::min(most, fill));
    L.block = dim3(AR_NT);
    L.smem = smem;
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    return launch_ex(L, k_kv_append_rot<DT, D, W>, a);
}

template <int DT, int D>
cudaError_t launch_w(const KvAppendRotArgs &a, int nsm, cudaStream_t s)
{
    // Four warps to a unit where sequences bring 4 tokens or more on average, as in pi_kv_append.cu.
    return a.b.n_tokens >= 4 * (int64_t)a.b.n ? launch_of<DT, D, 8>(a, nsm, s) : launch_of<DT, D, 1>(a, nsm, s);
}

template <int DT>
cudaError_t launch_dim(const KvAppendRotArgs &a, int nsm, cudaStream_t s)
{
    return a.c.dim == 64 ? launch_w<DT, 64>(a, nsm, s) : a.c.dim == 128 ? launch_w<DT, 128>(a, nsm, s) : launch_w<DT, 256>(a, nsm, s);
}

}  // namespace

cudaError_t launch_kv_append_rot(const KvAppendRotArgs &a, int dtype, int nsm, cudaStream_t s)
{
    return dtype == DT_F32 ? launch_dim<DT_F32>(a, nsm, s) : dtype == DT_BF16 ? launch_dim<DT_BF16>(a, nsm, s) : launch_dim<DT_F16>(a, nsm, s);
}

}  // namespace pi
