// pi_rotate.cu -- norms of query and key heads with the position rotation (sm_103a).
//
// Each element is read and written once, and the bytes bound it. A warp takes a token and some of its heads: it works out
// the cosines and sines of its columns once, then streams queries and keys, four rounds of loads at a time.
// Measured: 8191 tokens of 64 + 8 heads of 128, bf16, with norms 56 us = 5.4 TB/s (issue slots and memory are both near
// their end); 1003 tokens of 40 + 40 heads of 64, fp32 11 us; one token 2.7 us of the GPU's time (and 15 of the host's).
#include <algorithm>

#include "pi_rotary.cuh"

namespace pi {

constexpr int RO_NT = 256, RO_NW = RO_NT / 32;

template <int DT, int D>
__global__ void __launch_bounds__(RO_NT, DT == DT_F32 ? 3 : 4) k_rotate(const RotateArgs a)
{
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t item = (int64_t)blockIdx.x * RO_NW + (threadIdx.x >> 5);
    if (item >= (int64_t)a.n_tokens * a.parts) return;
    const int64_t tok = item / a.parts;
    const int part = (int)(item - tok * a.parts), heads = a.hq + a.hk;
    const int h_lo = (int)((int64_t)heads * part / a.parts), h_hi = (int)((int64_t)heads * (part + 1) / a.parts);
    const RotaryLane l = rotary_lane<D>(a.r, lane);
    float2 cs[4];
    if (l.turned) {
        const int p = a.pos[tok];
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = turn_cos_sin(a.r.turns[l.pair0 + i], p, a.r.amp);
    }
    if (h_lo < a.hq)
        rotate_heads<DT, D, 4>(a.r, l, rotary_coef(a.r, l, a.r.qn, cs), (const uint8_t *)a.q + tok * a.ldq * ES,
                               (uint8_t *)a.qo + tok * a.ldqo * ES, h_lo, min(h_hi, a.hq), lane);
    if (h_hi > a.hq)
        rotate_heads<DT, D, 4>(a.r, l, rotary_coef(a.r, l, a.r.kn, cs), (const uint8_t *)a.k + tok * a.ldk * ES,
                               (uint8_t *)a.ko + tok * a.ldko * ES, max(h_lo, a.hq) - a.hq, h_hi - a.hq, lane);
}

cudaError_t launch_rotate(const RotateArgs &in, int dim, int dtype, int nsm, cudaStream_t s)
{
    RotateArgs a = in;
    // Warps to a token: 32 to an SM in all where the tokens are few (and a round of heads to each at least).
    const int64_t rounds = (a.hq + a.hk + 256 / dim - 1) / (256 / dim);
    a.parts = (int)std::max<int64_t>(1, std::min(rounds, (int64_t)32 * nsm / a.n_tokens));
    const int64_t items = (int64_t)a.n_tokens * a.parts;
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
