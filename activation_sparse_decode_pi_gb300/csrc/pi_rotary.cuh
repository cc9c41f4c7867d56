// pi_rotary.cuh -- norm and position rotation of a head, eight elements to a lane (sm_103a).
//
// A head of D elements lies in D / 8 neighbouring lanes of a warp, each with two runs of four elements, A and B. In the half
// layout the first rot / 8 lanes take A from the first half of what is turned and B from the same place of the second, so
// an element's partner is in the same lane; neighbouring pairs are anyway. With w the norm's weights, c and s the
// angle's cosine and sine times amp (s negative for a pair's first),
//   out = inv (x w c + x' w' s),   inv = 1 / sqrt(mean x^2 + eps):
// the two coefficients of an element depend on the token only, and serve all its heads.
#pragma once

#include "pi_kv_device.cuh"
#include "pi_proj_internal.h"

namespace pi {

// A lane's eight elements, as they lie in memory.
template <int DT>
struct Eight {
    static constexpr int W = DT == DT_F32 ? 4 : 2;   // 32-bit words of a run
    uint32_t w[2][W];

    __device__ __forceinline__ void load(const uint8_t *a, const uint8_t *b)   // where its runs lie
    {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if constexpr (DT == DT_F32) {
                const uint4 v = *(const uint4 *)(r ? b : a);
                w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
            } else {
                const uint2 v = *(const uint2 *)(r ? b : a);
                w[r][0] = v.x, w[r][1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < W; ++i) w[r][i] = 0;
    }
    // elements 2 i, 2 i + 1 of A (i < 2) and of B (i >= 2)
    __device__ __forceinline__ void widen(float2 (&f)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t *const v = w[i >> 1];
            if constexpr (DT == DT_F32) {
                f[i] = make_float2(__uint_as_float(v[2 * (i & 1)]), __uint_as_float(v[2 * (i & 1) + 1]));
            } else if constexpr (DT == DT_BF16) {
                f[i] = make_float2(__uint_as_float(v[i & 1] << 16), __uint_as_float(v[i & 1] & 0xffff0000u));
            } else {
                f[i] = __half22float2(u32_h2(v[i & 1]));
            }
        }
    }
    static __device__ __forceinline__ void store(uint8_t *a, uint8_t *b, const float2 (&f)[4])
    {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float2 x = f[2 * r], y = f[2 * r + 1];
            if constexpr (DT == DT_F32) {
                *(float4 *)(r ? b : a) = make_float4(x.x, x.y, y.x, y.y);
            } else {
                uint2 o;
                if constexpr (DT == DT_BF16) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y), k = __floats2bfloat162_rn(y.x, y.y);
                    o = make_uint2(*reinterpret_cast<const uint32_t *>(&h), *reinterpret_cast<const uint32_t *>(&k));
                } else {
                    o = make_uint2(pack_f16(x.x, x.y), pack_f16(y.x, y.y));
                }
                *(uint2 *)(r ? b : a) = o;
            }
        }
    }
};

// Cosine and sine of position p's angle, times amp. The angle in 2^-32 of a turn is a whole number; what is left of it
// next to a multiple of a quarter turn, u eighths of a turn with |u| <= 1, goes into polynomials in u^2 (fitted to
// sin(pi u / 4) / u and cos(pi u / 4) for the smallest largest error: 2.5e-9 and 5e-11, in fp32 6e-8 of a value).
__device__ __forceinline__ float2 turn_cos_sin(uint64_t turns, int p, float amp)
{
    const uint32_t x = (uint32_t)((turns * (uint64_t)(int64_t)p) >> 32), quarter = (x + 0x20000000u) >> 30;
    const float u = (float)(int)(x - (quarter << 30)) * 0x1p-29f, v = u * u;
    const float s = amp * (u * fmaf(v, fmaf(v, fmaf(v, -0x1.2d9bb8p-15f, 0x1.465ec6p-9f), -0x1.4abbbap-4f), 0x1.921fb6p-1f));
    const float c = amp * fmaf(v, fmaf(v, fmaf(v, fmaf(v, 0x1.d9c364p-19f, -0x1.55c57cp-12f), 0x1.03c1dcp-6f), -0x1.3bd3ccp-2f), 1.f);
    const float a = quarter & 1 ? -s : c, b = quarter & 1 ? c : s;   // a quarter turn: (c, s) -> (-s, c)
    return quarter & 2 ? make_float2(-a, -b) : make_float2(a, b);
}

// Which elements of a head a lane has.
struct RotaryLane {
    int off_a, off_b;   // first elements of its runs
    int pair0;          // first of its four pairs
    bool turned;
};

template <int D>
__device__ __forceinline__ RotaryLane rotary_lane(const RotaryDev &r, int lane)
{
    const int l = lane % (D / 8);
    RotaryLane o;
    o.turned = 8 * l < r.rot;
    o.pair0 = o.turned ? 4 * l : 0;
    const bool halves = o.turned && !r.interleaved;
    o.off_a = halves ? 4 * l : 8 * l;
    o.off_b = halves ? r.rot / 2 + 4 * l : 8 * l + 4;
    return o;
}

// Coefficients of a lane's elements, as its runs lie: x's own, and its partner's.
struct RotaryCoef {
    float2 own[4], other[4];
};

// A norm's weights of the lane's elements (NULL: ones).
__device__ __forceinline__ void rotary_weights(const RotaryDev &r, const RotaryLane &l, const float *weight, float (&w)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (r.norm && weight) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = weight[e < 4 ? l.off_a + e : l.off_b + e - 4];
    }
}

// From a norm's weights (NULL: ones) and the cosines and sines, times amp, of the lane's four pairs.
__device__ __forceinline__ RotaryCoef rotary_coef(const RotaryDev &r, const RotaryLane &l, const float *weight, const float2 (&cs)[4])
{
    float w[8];
    rotary_weights(r, l, weight, w);
    RotaryCoef o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o.own[i] = make_float2(w[2 * i], w[2 * i + 1]);
        o.other[i] = make_float2(0.f, 0.f);
    }
    if (!l.turned) return o;
    if (r.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // pair i: elements 2 i and 2 i + 1
            o.own[i] = make_float2(w[2 * i] * cs[i].x, w[2 * i + 1] * cs[i].x);
            o.other[i] = make_float2(-w[2 * i + 1] * cs[i].y, w[2 * i] * cs[i].y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // pairs 2 i and 2 i + 1: their firsts in A, their seconds in B
            const float2 u = cs[2 * i], v = cs[2 * i + 1];
            o.own[i] = make_float2(w[2 * i] * u.x, w[2 * i + 1] * v.x);
            o.own[2 + i] = make_float2(w[4 + 2 * i] * u.x, w[5 + 2 * i] * v.x);
            o.other[i] = make_float2(-w[4 + 2 * i] * u.y, -w[5 + 2 * i] * v.y);
            o.other[2 + i] = make_float2(w[2 * i] * u.y, w[2 * i + 1] * v.y);
        }
    }
    return o;
}

// 1 / sqrt(mean x^2 + eps) of the head that the lane's D / 8 lanes hold
template <int D>
__device__ __forceinline__ float head_inv(const RotaryDev &r, const float2 (&x)[4])
{
    float2 q = fmul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) q = ffma2(x[i], x[i], q);
    float s = q.x + q.y;
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return rsqrtf(s * (1.f / D) + r.eps);
}

// The lane's eight outputs. The whole warp takes part.
template <int DT, int D>
__device__ __forceinline__ void rotate_eight(const RotaryDev &r, const RotaryLane &l, const Eight<DT> &raw, const RotaryCoef &k,
                                             float2 (&out)[4])
{
    float2 x[4];
    raw.widen(x);
    float inv = 1.f;
    if (r.norm) inv = head_inv<D>(r, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = fmul2(x[i], k.own[i]);
    if (l.turned) {   // (not turned: nothing that lies beside it may meet a zero, for 0 * infinity)
        if (r.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = ffma2(make_float2(x[i].y, x[i].x), k.other[i], out[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = ffma2(x[i ^ 2], k.other[i], out[i]);
        }
    }
    if (r.norm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = fmul2(out[i], make_float2(inv, inv));
    }
}

// The same, to the bit, from a norm's weights and the cosines and sines of the lane's pairs (first two, last two): for tokens
// that differ from lane to lane, where sixteen coefficients a token would only fill registers (7 prompts of ~2000 tokens, 8
// heads of 128, 125 us so).
template <int D>
__device__ __forceinline__ void rotate_once(const RotaryDev &r, const RotaryLane &l, const float (&w)[8], const float2 (&c)[2],
                                            const float2 (&s)[2], float2 (&x)[4])
{
    float inv = 1.f;
    if (r.norm) inv = head_inv<D>(r, x);
    if (!l.turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmul2(x[i], make_float2(w[2 * i], w[2 * i + 1]));
    } else if (r.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float cc = i & 1 ? c[i >> 1].y : c[i >> 1].x, ss = i & 1 ? s[i >> 1].y : s[i >> 1].x;
            const float2 ww = make_float2(w[2 * i], w[2 * i + 1]), sw = make_float2(-w[2 * i + 1], w[2 * i]);
            x[i] = ffma2(make_float2(x[i].y, x[i].x), fmul2(sw, make_float2(ss, ss)), fmul2(x[i], fmul2(ww, make_float2(cc, cc))));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 a = x[i], b = x[2 + i];
            const float2 wa = make_float2(w[2 * i], w[2 * i + 1]), wb = make_float2(w[4 + 2 * i], w[5 + 2 * i]);
            x[i] = ffma2(b, fmul2(wb, make_float2(-s[i].x, -s[i].y)), fmul2(a, fmul2(wa, c[i])));
            x[2 + i] = ffma2(a, fmul2(wa, s[i]), fmul2(b, fmul2(wb, c[i])));
        }
    }
    if (r.norm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmul2(x[i], make_float2(inv, inv));
    }
}

// Heads [h0, h1) of one token: src and dst are where the token's heads of the array begin, k its coefficients. A warp has
// 256 / D heads to a round, and U rounds of loads under way.
template <int DT, int D, int U>
__device__ __forceinline__ void rotate_heads(const RotaryDev &r, const RotaryLane &l, const RotaryCoef &k, const void *src,
                                             void *dst, int h0, int h1, int lane)
{
    constexpr int RPW = 256 / D, ES = DT == DT_F32 ? 4 : 2, ROUND = RPW * D * ES;
    const int sub = lane / (D / 8), mine = h0 * D + sub * D;
    const uint8_t *sa = (const uint8_t *)src + (int64_t)(mine + l.off_a) * ES, *sb = sa + (l.off_b - l.off_a) * ES;
    uint8_t *da = (uint8_t *)dst + (int64_t)(mine + l.off_a) * ES, *db = da + (l.off_b - l.off_a) * ES;
    for (int left = h1 - h0; left > 0; left -= U * RPW) {
        Eight<DT> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * RPW + sub < left) raw[u].load(sa + u * ROUND, sb + u * ROUND);
            else raw[u].clear();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u * RPW >= left) break;
            float2 out[4];
            rotate_eight<DT, D>(r, l, raw[u], k, out);
            if (u * RPW + sub < left) Eight<DT>::store(da + u * ROUND, db + u * ROUND, out);
        }
        sa += U * ROUND, sb += U * ROUND, da += U * ROUND, db += U * ROUND;
    }
}

}  // namespace pi
