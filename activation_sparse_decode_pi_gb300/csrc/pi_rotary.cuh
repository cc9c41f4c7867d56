// pi_rotary.cuh -- norm and position rotation of a head, eight elements to a lane (sm_103a).
//
// A head of D elements lies in D / 8 neighbouring lanes of a warp. Pairs are eight elements or a multiple apart (rot_dim is
// a multiple of 16) or neighbours, so an element's partner is in another lane at the same place or in its own lane.
// With w the norm's weights, c and s the angle's cosine and sine times amp (s negative for a pair's first),
//   out = inv (x w c + x' w' s),   inv = 1 / sqrt(mean x^2 + eps):
// the two coefficients of an element depend on the token only, and serve all its heads.
#pragma once

#include "pi_kv_device.cuh"
#include "pi_proj_internal.h"

namespace pi {

// Eight consecutive elements, as they lie in memory.
template <int DT>
struct Eight {
    static constexpr int W = DT == DT_F32 ? 8 : 4;   // 32-bit words
    uint32_t w[W];

    __device__ __forceinline__ void load(const void *p, int64_t at)
    {
        const uint4 *s = (const uint4 *)((const uint8_t *)p + at * (DT == DT_F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 v = s[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const
    {
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        } else {
            unpack<DT>(make_uint4(w[0], w[1], w[2], w[3]), f);
        }
    }
    __device__ __forceinline__ Eight from_lane(int lane) const
    {
        Eight r;
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = __shfl_sync(0xffffffffu, w[i], lane);
        return r;
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, const float (&f)[8])
    {
        uint4 *d = (uint4 *)((uint8_t *)p + at * (DT == DT_F32 ? 4 : 2));
        if constexpr (DT == DT_F32) {
            d[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            d[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
        } else {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == DT_BF16) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    o[i] = *reinterpret_cast<const uint32_t *>(&h);
                } else {
                    o[i] = pack_f16(f[2 * i], f[2 * i + 1]);
                }
            }
            d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
};

// Cosine and sine of position p's angle, times amp. The angle in 2^-32 of a turn is a whole number; what is left of it
// next to a multiple of a quarter turn goes to the functions, so its rounding to fp32 is at most 2^-26 of a turn.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t turns, int p, float amp)
{
    const int x = (int)(uint32_t)((turns * (uint64_t)(int64_t)p) >> 32);
    const int quarter = (int)(((uint32_t)x + 0x20000000u) >> 30);
    const int left = (int)((uint32_t)x - ((uint32_t)quarter << 30));
    float s, c;
    sincospif((float)left * 0x1p-31f, &s, &c);
    const float a = quarter & 1 ? -s : c, b = quarter & 1 ? c : s;   // a quarter turn: (c, s) -> (-s, c)
    return quarter & 2 ? make_float2(-a * amp, -b * amp) : make_float2(a * amp, b * amp);
}

// What a lane knows of its eight elements' columns.
struct RotaryLane {
    int pair0;        // pair of its first element (interleaved: of its first two)
    int partner;      // lane with the partners (itself: interleaved, or not turned)
    bool turned, second;
};

template <int D>
__device__ __forceinline__ RotaryLane rotary_lane(const RotaryDev &r, int lane)
{
    constexpr int LPR = D / 8;
    const int l = lane % LPR, col = l * 8, half = r.rot / 2;
    RotaryLane o;
    o.turned = col < r.rot;
    o.second = o.turned && !r.interleaved && col >= half;
    o.pair0 = !o.turned ? 0 : r.interleaved ? col / 2 : o.second ? col - half : col;
    o.partner = !o.turned || r.interleaved ? lane : o.second ? lane - half / 8 : lane + half / 8;
    return o;
}

// 1 / sqrt(mean x^2 + eps) of the head that the lane's D / 8 lanes hold
template <int D>
__device__ __forceinline__ float head_inv(const float (&x)[8], float eps)
{
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(x[e], x[e], q);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    return rsqrtf(q * (1.f / D) + eps);
}

// The lane's eight outputs: own coefficients wc, partners' ws. The whole warp takes part.
template <int DT, int D>
__device__ __forceinline__ void rotate_eight(const RotaryDev &r, const RotaryLane &l, const Eight<DT> &raw,
                                             const float (&wc)[8], const float (&ws)[8], float (&out)[8])
{
    float x[8], y[8];
    raw.widen(x);
    const float inv = r.norm ? head_inv<D>(x, r.eps) : 1.f;
    if (r.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
    } else {
        raw.from_lane(l.partner).widen(y);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float v = x[e] * wc[e];
        if (l.turned) v = fmaf(y[e], ws[e], v);   // (not turned: its partner's infinity must not meet a zero)
        out[e] = v * inv;
    }
}

// Weights of the lane's eight elements and of their partners (ones without a norm).
template <int D>
__device__ __forceinline__ void norm_weights(const RotaryDev &r, const RotaryLane &l, const float *weight, int lane,
                                             float (&w)[8], float (&wp)[8])
{
    constexpr int LPR = D / 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
    if (!r.norm || !weight) return;
    const float *a = weight + lane % LPR * 8, *b = weight + l.partner % LPR * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        w[e] = a[e];
        wp[e] = r.interleaved ? a[e ^ 1] : b[e];
    }
}

}  // namespace pi
