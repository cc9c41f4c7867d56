// pi_kv_append_rot.cu -- one pass from a fused projection into the attention: queries and keys normed and rotated by
// their positions, keys and values coded into the paged 8-bit cache (sm_103a).
//
// Each element is read once and written once (a query in its type, a key or value as a code), and those bytes bound it.
// A CTA has the new tokens of one page of one sequence and a slice of their queries, or of their keys and values (pages of
// all sequences are counted through, so that ragged prompts fill the GPU evenly). Queries: a
// token and a part of its heads to a warp, as in pi_rotate.cu. Keys and values: one to eight warps to one (page, head), as in
// pi_kv_append.cu (largest value, block scale, codes), keys with cosines and sines that the CTA works out once for all its
// heads.
// Measured: 7 prompts of 1015..3351 tokens, 32 heads on 8 of 128, bf16 96 us = 3.5 TB/s; queries alone (the other CTAs out)
// took 62 us, keys and values 60 us, and both want issue slots. 64 tokens of 40 + 80 heads, fp32 6.3 us; one token 3.1 us.
#include <algorithm>

#include "pi_rotary.cuh"

namespace pi {

constexpr int AR_NT = 256, AR_NW = AR_NT / 32;
// U: loads of eight elements that a thread has under way at a time
template <int DT, int D, int U>
__global__ void __launch_bounds__(AR_NT, 3) k_kv_append_rot(const KvAppendRotArgs a)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ES = DT == DT_F32 ? 4 : 2;
    extern __shared__ __align__(16) float table[];   // [tokens of a page][rot / 2] cosines, then sines
    __shared__ float s_top[AR_NW];
    __shared__ int s_item, s_sum[AR_NW];
    __shared__ KvSeq s_seq;
    const KvView &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = c.page;
    pdl_wait();
    pdl_launch_dependents();
    // the blockIdx.x-th page that new tokens of the call fall into
    const int ps = __ffs(P) - 1;
    if (tid == 0) s_item = -1;
    const bool flag = blockIdx.x == 0 && blockIdx.y == 0;   // the CTA that looks at every sequence, for what is out of range
    int before = 0;
    for (int b0 = 0; b0 < a.b.n && (flag || before <= (int)blockIdx.x); b0 += AR_NT) {
        const int i = b0 + tid;
        KvSeq s = {};
        int cnt = 0;
        if (i < a.b.n) {
            s = kv_sequence(c, a.b, i, flag);
            if (s.n > 0 && s.n <= s.len) cnt = ((s.len - 1) >> ps) - ((s.len - s.n) >> ps) + 1;
            else if (s.n > 0 && flag) set_status(c.status, ST_DEVICE_CHECK);   // no room was reserved
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        int at = before + inc - cnt;
#pragma unroll
        for (int x = 0; x < AR_NW; ++x) {
            at += x < warp ? s_sum[x] : 0;
            before += s_sum[x];
        }
        if (at <= (int)blockIdx.x && (int)blockIdx.x < at + cnt) {
            s_item = (int)blockIdx.x - at;
            s_seq = s;
        }
        __syncthreads();
    }
    if (s_item < 0) return;
    const KvSeq q = s_seq;
    const int first = q.len - q.n, col = (first >> ps) + s_item;   // position of the first new token; the page's column
    const int p0 = max(first - col * P, 0), p1 = min(q.len - col * P, P), rows = p1 - p0;   // new slots of the page
    const int pos0 = col * P + p0;
    const int64_t row0 = (int64_t)q.start + pos0 - first;   // their first row in the call
    const RotaryLane l = rotary_lane<D>(a.r, lane);
    if ((int)blockIdx.y < a.slices_q) {
        // ---------------------------------------------------------------- queries
        const int warps = AR_NW * a.slices_q;
        const int parts = max(1, min(warps / rows, (c.hq + RPW - 1) / RPW));   // few tokens: several warps to one
        for (int item = blockIdx.y * AR_NW + warp; item < rows * parts; item += warps) {
            const int t = item / parts, part = item - t * parts;
            const int h0 = c.hq * part / parts, h1 = c.hq * (part + 1) / parts;
            float2 cs[4];
            if (l.turned) {
#pragma unroll
                for (int i = 0; i < 4; ++i) cs[i] = turn_cos_sin(a.r.turns[l.pair0 + i], pos0 + t, a.r.amp);
            }
            rotate_heads<DT, D, U == 1 ? 2 : 4>(a.r, l, rotary_coef(a.r, l, a.r.qn, cs), (const uint8_t *)a.q + (row0 + t) * a.ldq * ES,
                                                (uint8_t *)a.qo + (row0 + t) * a.ldqo * ES, h0, h1, lane);
        }
        return;
    }
    // -------------------------------------------------------------------- keys and values
    const int W = a.warps, NTH = W * 32, th = tid & (NTH - 1), unit0 = warp / W, per = AR_NW / W;   // W: a power of two
    const int half = a.r.rot / 2, slice = blockIdx.y - a.slices_q, slices = gridDim.y - a.slices_q;
    float *const cosv = table, *const sinv = table + a.cap * half;
    float w[8];
    rotary_weights(a.r, l, a.r.kn, w);
    const int page = c.table[(size_t)q.row * c.max_pages + col];
    if (page < 0 || page >= c.n_pages) {
        if (tid == 0) set_status(c.status, ST_DEVICE_CHECK);
        return;
    }
    for (int x = tid; x < rows * half; x += AR_NT) {
        const int r = x / half, i = x - r * half;
        const float2 cs = turn_cos_sin(a.r.turns[i], pos0 + r, a.r.amp);
        cosv[x] = cs.x;
        sinv[x] = cs.y;
    }
    __syncthreads();
    // W warps to a head
    for (int u = slice * per + unit0; u < 2 * c.hkv; u += slices * per) {
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
            raw.widen(f);
            if (val) return;
            const int at = min(v / LPR, rows - 1) * half + l.pair0;
            float2 cc[2], ss[2];
            if (l.turned) {
                const float4 c4 = *(const float4 *)(cosv + at), s4 = *(const float4 *)(sinv + at);
                cc[0] = make_float2(c4.x, c4.y), cc[1] = make_float2(c4.z, c4.w);
                ss[0] = make_float2(s4.x, s4.y), ss[1] = make_float2(s4.z, s4.w);
            }
            rotate_once<D>(a.r, l, w, cc, ss, f);
        };
        const float was = p0 > 0 ? *scale : 0.f;
        const int v0 = th & ~31;   // the warp's first
        float2 f[4];               // of the unit's last eight of this thread
        // `use` of every group of eight, U loads under way at a time
        auto over_rows = [&](auto use) {
            for (int v = 0; v + v0 < nv; v += U * NTH) {
                Eight<DT> raw[U];
#pragma unroll
                for (int x = 0; x < U; ++x) raw[x] = fetch(v + x * NTH + th);
#pragma unroll
                for (int x = 0; x < U; ++x) {
                    if (v + x * NTH + v0 >= nv) break;
                    finish(raw[x], v + x * NTH + th, f);
                    use(v + x * NTH + th);
                }
            }
        };
        float top = 0.f;
        over_rows([&](int v) {   // (fmaxf leaves NaN out)
            if (v < nv) {
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
            }
        });
        auto over_unit = [&](float x) {   // the largest of the unit's threads
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (W > 1) {
                if (lane == 0) s_top[warp] = x;
                bar_sync(1 + unit0, NTH);
                for (int y = 0; y < W; ++y) x = fmaxf(x, s_top[unit0 * W + y]);
                bar_sync(1 + unit0, NTH);   // (s_top is free again)
            }
            return x;
        };
        top = over_unit(top);
        if (top > 3.402823466e38f) {   // an infinity: once more without (rare)
            top = 0.f;
            over_rows([&](int v) {
                if (v < nv) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(finite_abs(f[e].x), finite_abs(f[e].y)));
                }
            });
            top = over_unit(top);
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
        auto put = [&](int v) {
            uint32_t o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float2 x = fmul2(f[2 * e], make_float2(rcp, rcp)), y = fmul2(f[2 * e + 1], make_float2(rcp, rcp));
                if (!pow2) x = make_float2(f[2 * e].x / s, f[2 * e].y / s), y = make_float2(f[2 * e + 1].x / s, f[2 * e + 1].y / s);
                o[e] = f32x2_e4m3x2(x.x, x.y) | (uint32_t)f32x2_e4m3x2(y.x, y.y) << 16;
            }
            if (v < nv) {
                uint8_t *const to = codes + (size_t)(p0 + v / LPR) * D;
                *(uint32_t *)(to + l.off_a) = o[0];
                *(uint32_t *)(to + l.off_b) = o[1];
            }
        };
        // one eight to a thread is still there; more are read again (from the caches: a page's head is some kilobytes)
        if (nv <= NTH) {
            if (v0 < nv) put(th);
        } else {
            over_rows(put);
        }
    }
}

namespace {

template <int DT, int D, int U>
cudaError_t launch_of(const KvAppendRotArgs &in, int nsm, cudaStream_t s)
{
    KvAppendRotArgs a = in;
    const int64_t n = a.b.n, T = a.b.n_tokens;
    // Pages that T tokens of n sequences touch, at most.
    const int64_t pages = std::min(T, T / a.c.page + 2 * n);
    // Warps to a page's head: one where that makes enough of them (48 to an SM), and no more than its rows fill (measured,
    // 7 prompts of ~2000 tokens, 8 heads of 128, bf16, where the rule takes two: 110, 102, 96 and 95 us with eight, four, two
    // and one; 64 single tokens, which fill one: 6.3 us, 10.4 with two).
    a.warps = 1;
    while (a.warps < AR_NW && pages * 2 * a.c.hkv * a.warps < 48 * (int64_t)nsm && std::min<int64_t>(a.c.page, T / n) * D > a.warps * 256 * U)
        a.warps *= 2;
    // Slices of a page's queries and of its keys and values, by their number: about eight rounds of what the GPU holds.
    const int64_t fill = (int64_t)24 * nsm / pages, heads = a.c.hq + 2 * a.c.hkv, round = 256 / D;
    const auto slices = [&](int64_t part, int64_t most) { return std::max<int64_t>(1, std::min(most, fill * part / heads)); };
    a.slices_q = (int)slices(a.c.hq, (a.c.hq + AR_NW * round - 1) / (AR_NW * round));
    const int64_t per = AR_NW / a.warps, slices_kv = slices(2 * a.c.hkv, (2 * a.c.hkv + per - 1) / per);
    a.cap = (int)std::min<int64_t>(a.c.page, T);
    const size_t smem = (size_t)a.cap * a.r.rot * 4;   // at most 128 x 256 x 4
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_smem<k_kv_append_rot<DT, D, U>>(128 * D * 4);
        if (e != cudaSuccess) return e;
    }
    Launch L;
    L.grid = dim3((unsigned)pages, (unsigned)(a.slices_q + slices_kv));
    L.block = dim3(AR_NT);
    L.smem = smem;
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    return launch_ex(L, k_kv_append_rot<DT, D, U>, a);
}

template <int DT, int D>
cudaError_t launch_w(const KvAppendRotArgs &a, int nsm, cudaStream_t s)
{
    // Several loads at a time where sequences bring 4 tokens or more on average: fewer have no more than one to a thread.
    // Four of 16 bits; two of fp32, of which four spill (7 prompts of ~2000 tokens 161 us with four, 132 with two).
    constexpr int U = DT == DT_F32 ? 2 : 4;
    return a.b.n_tokens >= 4 * (int64_t)a.b.n ? launch_of<DT, D, U>(a, nsm, s) : launch_of<DT, D, 1>(a, nsm, s);
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
