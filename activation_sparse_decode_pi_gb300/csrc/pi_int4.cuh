// pi_int4.cuh -- what the two kernels of the int4 projections share (pi_int4.cu: few rows of x; pi_int4_rows.cu: more).
#pragma once

#include <algorithm>

#include "pi_proj_internal.h"
#include "pi_kv_device.cuh"

namespace pi {

constexpr int I4_GROUP = 128;
constexpr int I4_SMEM = 227 * 1024;    // of a CTA, one to an SM

// The eight nibbles of a word as f16 pairs (i, i + 4), each q 2^-10: a nibble in the low bits of a half reads as the subnormal
// (q + 8) 2^-24 (flipping its top bit turns two's complement into offset binary), one in bits 4..7 as 16 times that; one exact
// half-precision operation takes both to q 2^-10, a normal number: the tensor cores line products up by their operands'
// exponents, and a subnormal's says 2^-14 however small it is, so sums of subnormals lose low bits (1 x 12288 -> 36864, fp32,
// error against 64 bits: 7.3e-7 with q 2^-24). (With the offset left on and taken off each group's sum, groups of zeros did
// not give 0, and an infinity gave NaN everywhere.)
__device__ __forceinline__ void i4_word_h2(uint32_t w, uint32_t (&p)[4])
{
    const uint32_t w8 = w >> 8;
    const __half2 low = u32_h2(0x74007400u), high = u32_h2(0x64006400u), off = u32_h2(0xa000a000u);   // 2^14, 2^10; -8 2^-10
    const __half2 h[4] = {__hfma2(u32_h2(lop3_and_xor(w, 0x000F000Fu, 0x00080008u)), low, off),
                          __hfma2(u32_h2(lop3_and_xor(w, 0x00F000F0u, 0x00800080u)), high, off),
                          __hfma2(u32_h2(lop3_and_xor(w8, 0x000F000Fu, 0x00080008u)), low, off),
                          __hfma2(u32_h2(lop3_and_xor(w8, 0x00F000F0u, 0x00800080u)), high, off)};
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const uint32_t *>(&h[i]);
}

// Groups [g_lo, g_lo + gn) of rows [b0, b0 + nb) of x as f16 terms by `warps` warps: put(group, row, term, halves) gets the
// lane's four of a word's eight (word lane / 2; its pairs 0 and 1 in an even lane, 2 and 3 in an odd one), units(group, row,
// unit) 2 times the unit of x. The largest element of a row's group lies in [2^14, 2^15) of its unit, so a term's
// smallest step (2^-25 at most away) is 2^-39 of it.
template <int DT, int S, class Put, class Units>
__device__ __forceinline__ void i4_take_x(const Int4Args &a, int b0, int nb, int g_lo, int gn, int warp, int warps, int lane, Put put,
                                          Units units)
{
    // a warp to a row's group, four elements to a lane, S groups' loads under way at a time
    const uint64_t magic = 0xffffffffull / (uint32_t)nb + 1;   // it / nb, exactly for it < 2^32 / nb
    const int all = gn * nb;
    for (int it0 = warp; it0 < all; it0 += S * warps) {
        float f[S][4];
#pragma unroll
        for (int y = 0; y < S; ++y) {
            const int it = it0 + y * warps, gl = (int)(it * magic >> 32), b = it - gl * nb;
            if (it >= all) break;
            const int64_t at = (int64_t)(b0 + b) * a.ldx + (int64_t)(g_lo + gl) * I4_GROUP + lane * 4;
            if constexpr (DT == DT_F32) {
                const float4 v = *(const float4 *)((const float *)a.x + at);
                f[y][0] = v.x, f[y][1] = v.y, f[y][2] = v.z, f[y][3] = v.w;
            } else {
                const uint2 v = *(const uint2 *)((const uint16_t *)a.x + at);
                if constexpr (DT == DT_BF16) {
                    f[y][0] = __uint_as_float(v.x << 16), f[y][1] = __uint_as_float(v.x & 0xffff0000u);
                    f[y][2] = __uint_as_float(v.y << 16), f[y][3] = __uint_as_float(v.y & 0xffff0000u);
                } else {
                    const float2 lo = __half22float2(u32_h2(v.x)), hi = __half22float2(u32_h2(v.y));
                    f[y][0] = lo.x, f[y][1] = lo.y, f[y][2] = hi.x, f[y][3] = hi.y;
                }
            }
        }
        int ex[S];
#pragma unroll
        for (int y = 0; y < S; ++y) {
            uint32_t top = 0;   // the largest finite size, as bits
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t u = __float_as_uint(f[y][e]) & 0x7fffffffu;
                top = max(top, u < 0x7f800000u ? u : 0u);
            }
            // 2^ex <= top < 2^(ex + 1) (zeros and the smallest numbers below)
            ex[y] = max((int)(__reduce_max_sync(0xffffffffu, top) >> 23) - 127, -113);
        }
#pragma unroll
        for (int y = 0; y < S; ++y) {
            const int it = it0 + y * warps, gl = (int)(it * magic >> 32), b = it - gl * nb;
            if (it >= all) break;
            const float mul = exp2i(14 - ex[y]);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[y][e] *= mul;
            // a word's elements 0..3 lie in an even lane, 4..7 in the next: the even lane takes pairs (0, 4) and (1, 5)
            const bool odd = lane & 1;
            const float p0 = __shfl_xor_sync(0xffffffffu, odd ? f[y][0] : f[y][2], 1);
            const float p1 = __shfl_xor_sync(0xffffffffu, odd ? f[y][1] : f[y][3], 1);
            const float x0 = odd ? p0 : f[y][0], y0 = odd ? f[y][2] : p0, x1 = odd ? p1 : f[y][1], y1 = odd ? f[y][3] : p1;
            const uint32_t h0 = pack_f16(x0, y0), h1 = pack_f16(x1, y1);
            put(gl, b, 0, make_uint2(h0, h1));
            if constexpr (DT == DT_F32) {
                const float2 c0 = __half22float2(u32_h2(h0)), c1 = __half22float2(u32_h2(h1));
                // (an infinity or NaN is in the first term)
                const auto rest = [](float x, float c) { return fabsf(x) < INFINITY ? x - c : 0.f; };
                put(gl, b, 1, make_uint2(pack_f16(rest(x0, c0.x), rest(y0, c0.y)), pack_f16(rest(x1, c1.x), rest(y1, c1.y))));
            }
            if (lane == 0) units(gl, b, exp2i(ex[y] - 13));
        }
    }
}

// y's element of row b of x and row i of W
template <int DT>
__device__ __forceinline__ void i4_store(const Int4Args &a, float v, int b, int i)
{
    if (a.bias) v += a.bias[i];
    const int64_t at = (int64_t)b * a.ldy + i, at_add = (int64_t)b * a.ldadd + i;
    if constexpr (DT == DT_F32) {
        if (a.add) v += ((const float *)a.add)[at_add];
        ((float *)a.y)[at] = v;
    } else if constexpr (DT == DT_BF16) {
        if (a.add) v += __bfloat162float(((const __nv_bfloat16 *)a.add)[at_add]);
        ((__nv_bfloat16 *)a.y)[at] = __float2bfloat16_rn(v);
    } else {
        if (a.add) v += __half2float(((const __half *)a.add)[at_add]);
        ((__half *)a.y)[at] = __float2half_rn(v);
    }
}

// The kernel for many rows; false: k is too long for it (eight rows of x do not fit a cluster's shared memory).
bool launch_int4_rows(const Int4Args &a, int dtype, int nsm, cudaStream_t s, cudaError_t *e);

// Clusters of cs CTAs, one to an SM, that run at a time. A cluster's SMs lie in one group of the GPU's SMs, so 152 SMs hold
// (by the runtime's count) 15 of 8 and not 19.
inline int clusters_at_once(int nsm, int cs)
{
    constexpr int of_152[8] = {152, 76, 46, 36, 28, 23, 15, 15};
    return std::max(1, of_152[cs - 1] * nsm / 152);
}

}  // namespace pi
