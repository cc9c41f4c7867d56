// pi_rotate.cu -- norms of query and key heads with the position rotation (sm_103a).
//
// Each element is read and written once, and the bytes bound it. A warp takes a token and some of its heads (all of one
// array): it works out the token's coefficients once, then streams heads, four rounds of loads at a time.
#include <algorithm>

#include "pi_rotary.cuh"

namespace pi {

constexpr int RO_NT = 256, RO_NW = RO_NT / 32;

template <int DT, int D>
__global__ void __launch_bounds__(RO_NT) k_rotate(const RotateArgs a)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
    const int lane = threadIdx.x & 31, sub = lane / LPR;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t item = (int64_t)blockIdx.x * RO_NW + (threadIdx.x >> 5);
    const int parts = a.parts_q + a.parts_k;
    if (item >= (int64_t)a.n_tokens * parts) return;
    const int64_t tok = item / parts;
    const int part = (int)(item % parts);
    const bool key = part >= a.parts_q;
    const int heads = key ? a.hk : a.hq, n = key ? a.parts_k : a.parts_q, x = key ? part - a.parts_q : part;
    const int h0 = (int)((int64_t)heads * x / n), h1 = (int)((int64_t)heads * (x + 1) / n);
    const uint8_t *src = (const uint8_t *)(key ? a.k : a.q);
    uint8_t *dst = (uint8_t *)(key ? a.ko : a.qo);
    const int64_t at = tok * (key ? a.ldk : a.ldq) + lane % LPR * 8, to = tok * (key ? a.ldko : a.ldqo) + lane % LPR * 8;

    Eight<DT> raw[U];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = h + u * RPW + sub;
            if (r < h1) raw[u].load(src, at + (int64_t)r * D);
            else raw[u].clear();
        }
    };
    load(h0);
    const RotaryLane l = rotary_lane<D>(a.r, lane);
    float wc[8], ws[8];
    norm_weights<D>(a.r, l, key ? a.r.kn : a.r.qn, lane, wc, ws);
    if (l.turned) {
        const int p = a.pos[tok];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (a.r.interleaved && (e & 1)) continue;
            const float2 cs = turn_cos_sin(a.r.turns[l.pair0 + (a.r.interleaved ? e / 2 : e)], p, a.r.amp);
            wc[e] *= cs.x;
            ws[e] *= l.second ? cs.y : -cs.y;
            if (a.r.interleaved) {
                wc[e + 1 & 7] *= cs.x;
                ws[e + 1 & 7] *= cs.y;
            }
        }
    }
    for (int h = h0; h < h1; h += U * RPW) {
        Eight<DT> now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = raw[u];
        if (h + U * RPW < h1) load(h + U * RPW);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = h + u * RPW + sub;
            if (h + u * RPW >= h1) break;
            float out[8];
            rotate_eight<DT, D>(a.r, l, now[u], wc, ws, out);
            if (r < h1) Eight<DT>::store(dst, to + (int64_t)r * D, out);
        }
    }
}

cudaError_t launch_rotate(const RotateArgs &in, int dim, int dtype, int nsm, cudaStream_t s)
{
    RotateArgs a = in;
    // Warps: about 32 to an SM where the tokens are few (a warp takes one round of heads at least), else one to a token
    // and array.
    const int64_t want = std::max<int64_t>(1, (int64_t)32 * nsm / a.n_tokens);
    const int heads = a.hq + a.hk, round = 256 / dim;
    const auto parts = [&](int h) {
        return h == 0 ? 0 : (int)std::max<int64_t>(1, std::min<int64_t>((h + round - 1) / round, want * h / heads));
    };
    a.parts_q = parts(a.hq);
    a.parts_k = parts(a.hk);
    const int64_t items = (int64_t)a.n_tokens * (a.parts_q + a.parts_k);
    Launch L;
    L.grid = dim3((unsigned)((items + RO_NW - 1) / RO_NW));
    L.block = dim3(RO_NT);
    L.smem = 0;
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    const auto run = [&](auto k64, auto k128, auto k256) {
        return dim == 64 ? launch_ex(L, k64, a) : dim == 128 ? launch_ex(L, k128, a) : launch_ex(L, k256, a);
    };
    switch (dtype) {
    case DT_F32: return run(k_rotate<DT_F32, 64>, k_rotate<DT_F32, 128>, k_rotate<DT_F32, 256>);
    case DT_BF16: return run(k_rotate<DT_BF16, 64>, k_rotate<DT_BF16, 128>, k_rotate<DT_BF16, 256>);
    default: return run(k_rotate<DT_F16, 64>, k_rotate<DT_F16, 128>, k_rotate<DT_F16, 256>);
    }
}

}  // namespace pi
