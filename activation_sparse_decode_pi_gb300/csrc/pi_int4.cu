// pi_int4.cu -- projections of a few rows with int4 group-128 weights (sm_103a).
//
// y[b, i] = sum_g s[i, g] sum_{k in g} q[i, k] x[b, k]. Up to a dozen rows the bytes of W bound it (half a byte a weight;
// d 4096: 13 MB in 1.9 us), so the rest has to hide under its loads:
//  - products on mma.sync m16n8k16, 16 rows of W against up to 8 rows of x: 16 bytes of a row of W to a lane are 32
//    nibbles, four lanes' a group. The contraction may run in any order that both operands share, so nibbles are used
//    as they lie: a word's nibbles (i, i + 4) become an f16 pair by masking them into the mantissa of 1024, and x is
//    laid into shared memory in that order;
//  - x is cut to f16 in units of a power of two for each row and group (fp32: two terms), undone in fp32 with the
//    weights' scale, so a group's sum is of exact integers times f16 and nothing else is rounded before fp32;
//  - a CTA's warps split its rows of W (MW ways) and the contraction (KW ways); CTAs of a cluster split the
//    contraction further and add their sums through distributed shared memory, in the order of their ranks.
#include <cooperative_groups.h>

#include <algorithm>

#include "pi_proj_internal.h"
#include "pi_kv_device.cuh"

namespace pi {

namespace cg = cooperative_groups;

constexpr int I4_NT = 256, I4_NW = I4_NT / 32;
constexpr int I4_GROUP = 128;
constexpr int I4_SMEM = 112 * 1024;   // of a CTA, two to an SM

struct Int4Plan {
    int kw, cluster;
};

// One lane's 16 bytes of a row of W against its four 16-wide chunks: f16 pairs of nibbles (i, i + 4) of each word.
__device__ __forceinline__ void i4_word_h2(uint32_t w, uint32_t (&p)[4])
{
    const uint32_t w8 = w >> 8;
    const __half2 k1032 = u32_h2(0x64086408u);   // 1032
    const __half2 k16th = u32_h2(0x2C002C00u);   // 1 / 16
    const __half2 km72 = u32_h2(0xD480D480u);    // -72 = -(1024 / 16 + 8)
    const auto bits = [](__half2 h) { return *reinterpret_cast<uint32_t *>(&h); };
    p[0] = bits(__hsub2(u32_h2(lop3_and_xor(w, 0x000F000Fu, 0x64086408u)), k1032));
    p[1] = bits(__hfma2(u32_h2(lop3_and_xor(w, 0x00F000F0u, 0x64806480u)), k16th, km72));
    p[2] = bits(__hsub2(u32_h2(lop3_and_xor(w8, 0x000F000Fu, 0x64086408u)), k1032));
    p[3] = bits(__hfma2(u32_h2(lop3_and_xor(w8, 0x00F000F0u, 0x64806480u)), k16th, km72));
}

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) { return pack_f16(lo, hi); }

// MT: runs of 16 rows of W to a warp; NT: runs of 8 rows of x.
template <int DT, int MT, int NT>
__global__ void __launch_bounds__(I4_NT, 2) k_int4_linear(const Int4Args a)
{
    constexpr int T = DT == DT_F32 ? 2 : 1;
    constexpr int U = MT == 1 ? 4 : NT == 2 ? 2 : 1;   // groups whose weights are loaded at a time
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int kw = a.kw, mw = I4_NW / kw, R = 16 * MT * mw;
    const int cs = a.cluster, rank = blockIdx.x % cs, tile = blockIdx.x / cs;
    const int b0 = blockIdx.y * (8 * NT), nb = min(a.rows - b0, 8 * NT);
    const int G = a.k / I4_GROUP, g_lo = (int)((int64_t)G * rank / cs), g_hi = (int)((int64_t)G * (rank + 1) / cs);
    const int wk = warp % kw, wm = warp / kw;
    const int row0 = tile * R + wm * 16 * MT;
    const size_t row_bytes = (size_t)a.k / 2;

    // this lane's rows of W (rows past the last read the last: their results are not stored)
    const uint8_t *wp[MT][2];
    const __half *sp[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = min(row0 + m * 16 + h * 8 + g, a.n - 1);
            wp[m][h] = a.w + (size_t)r * row_bytes + q * 16;
            sp[m][h] = a.s + (size_t)r * G;
        }
    // Into L2 before the previous kernel's results are waited for (a hint: nothing is read yet).
    for (int r = tid; r < R; r += I4_NT) {
        const int at = tile * R + r;
        if (at < a.n && g_hi > g_lo) prefetch_l2(a.w + (size_t)at * row_bytes + (size_t)g_lo * 64, (uint32_t)(g_hi - g_lo) * 64u);
    }
    pdl_wait();
    pdl_launch_dependents();

    float tot[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) tot[m][n][e] = 0.f;

    uint8_t *const frag = smem;                                               // [group][word][term][row][64 bytes]
    float *const xf = (float *)(smem + (size_t)a.chunk * 256 * T * nb);   // [group][8 NT] units of x

    for (int c_lo = g_lo; c_lo < g_hi; c_lo += a.chunk) {
        const int c_hi = min(g_hi, c_lo + a.chunk);
        uint4 w[2][U][MT][2];
        float s[2][U][MT][2];
        auto load = [&](int buf, int g0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int gr = g0 + u * kw;
                if (gr < c_hi) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            w[buf][u][m][h] = ld_stream((const uint4 *)(wp[m][h] + (size_t)gr * 64));
                            s[buf][u][m][h] = __half2float(__ldg(sp[m][h] + gr));
                        }
                }
            }
        };
        load(0, c_lo + wk);
        if (c_lo > g_lo) __syncthreads();   // the last chunk's x has been read
        // x of the chunk: a warp to a row's group, four elements to a lane
        for (int it = warp; it < (c_hi - c_lo) * nb; it += I4_NW) {
            const int gl = it / nb, b = it % nb;
            const int64_t at = (int64_t)(b0 + b) * a.ldx + (int64_t)(c_lo + gl) * I4_GROUP + lane * 4;
            float f[4];
            if constexpr (DT == DT_F32) {
                const float4 v = *(const float4 *)((const float *)a.x + at);
                f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
            } else {
                const uint2 v = *(const uint2 *)((const uint16_t *)a.x + at);
                if constexpr (DT == DT_BF16) {
                    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
                    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
                } else {
                    const float2 lo = __half22float2(u32_h2(v.x)), hi = __half22float2(u32_h2(v.y));
                    f[0] = lo.x, f[1] = lo.y, f[2] = hi.x, f[3] = hi.y;
                }
            }
            float top = fmaxf(fmaxf(finite_abs(f[0]), finite_abs(f[1])), fmaxf(finite_abs(f[2]), finite_abs(f[3])));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // 2^ex <= top < 2^(ex + 1): the largest lies in [128, 256)
            const int ex = top > 0.f ? min(max(ilogbf(top), -118), 127) : 0;
            const float mul = exp2i(7 - ex);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] *= mul;
            // a word's elements 0..3 lie in an even lane, 4..7 in the next: the even lane takes pairs (0, 4) and (1, 5)
            const bool odd = lane & 1;
            const float p0 = __shfl_xor_sync(0xffffffffu, odd ? f[0] : f[2], 1);
            const float p1 = __shfl_xor_sync(0xffffffffu, odd ? f[1] : f[3], 1);
            const float x0 = odd ? p0 : f[0], y0 = odd ? f[2] : p0, x1 = odd ? p1 : f[1], y1 = odd ? f[3] : p1;
            const int word = (lane >> 1) & 3, qq = lane >> 3;
            uint8_t *const to = frag + (size_t)((gl * 4 + word) * T * nb + b) * 64 + qq * 16 + odd * 8;
            const uint32_t h0 = f16_pair(x0, y0), h1 = f16_pair(x1, y1);
            *(uint2 *)to = make_uint2(h0, h1);
            if constexpr (T == 2) {
                const float2 c0 = __half22float2(u32_h2(h0)), c1 = __half22float2(u32_h2(h1));
                // (an infinity has no second term)
                const auto rest = [](float v, float c) { return fabsf(c) <= 65504.f ? v - c : 0.f; };
                *(uint2 *)(to + 64 * nb) = make_uint2(f16_pair(rest(x0, c0.x), rest(y0, c0.y)),
                                                          f16_pair(rest(x1, c1.x), rest(y1, c1.y)));
            }
            if (lane == 0) xf[gl * (8 * NT) + b] = exp2i(ex - 7);
        }
        __syncthreads();

        auto step = [&](const uint4 (&wv)[MT][2], const float (&sv)[MT][2], int gl) {
            float d[T][MT][NT][4];
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[t][m][n][e] = 0.f;
#pragma unroll
            for (int word = 0; word < 4; ++word) {
                uint32_t pa[MT][2][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) i4_word_h2(word4(wv[m][h], word), pa[m][h]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        uint4 b = make_uint4(0, 0, 0, 0);   // rows past the last: nothing was stored
                        if (8 * n + g < nb)
                            b = *(const uint4 *)(frag + (size_t)(((gl * 4 + word) * T + t) * nb + 8 * n + g) * 64 + q * 16);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint32_t a0[4] = {pa[m][0][0], pa[m][1][0], pa[m][0][1], pa[m][1][1]};
                            const uint32_t a1[4] = {pa[m][0][2], pa[m][1][2], pa[m][0][3], pa[m][1][3]};
                            mma_f16(d[t][m][n], a0, b.x, b.y);
                            mma_f16(d[t][m][n], a1, b.z, b.w);
                        }
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 u = *(const float2 *)&xf[gl * (8 * NT) + 8 * n + 2 * q];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = d[0][m][n][e];
                        if constexpr (T == 2) v += d[T - 1][m][n][e];
                        tot[m][n][e] = fmaf(v * (e & 1 ? u.y : u.x), sv[m][e >> 1], tot[m][n][e]);
                    }
            }
        };
        auto batch = [&](int buf, int g0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (g0 + u * kw < c_hi) step(w[buf][u], s[buf][u], g0 + u * kw - c_lo);
        };
        for (int g0 = c_lo + wk; g0 < c_hi; g0 += 2 * U * kw) {
            if (g0 + U * kw < c_hi) load(1, g0 + U * kw);
            batch(0, g0);
            if (g0 + 2 * U * kw < c_hi) load(0, g0 + 2 * U * kw);
            if (g0 + U * kw < c_hi) batch(1, g0 + U * kw);
        }
    }

    // ---------------------------------------------------------------- sums of the warps and of the cluster
    __syncthreads();   // x is no longer needed: its place takes the sums [KW][8 NT][R + 1]
    float *const red = (float *)smem;
    const int ldr = R + 1;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = wm * 16 * MT + m * 16 + (e >> 1) * 8 + g, b = 8 * n + 2 * q + (e & 1);
                if (b < nb) red[(wk * (8 * NT) + b) * ldr + r] = tot[m][n][e];
            }
    cg::cluster_group cl = cg::this_cluster();
    if (cs > 1) cl.sync();
    else __syncthreads();
    const int per = R / cs;   // rows that this CTA adds up
    for (int x = tid; x < per * nb; x += I4_NT) {
        const int r = rank * per + x % per, b = x / per, i = tile * R + r;
        if (i >= a.n) continue;
        float v = 0.f;
        for (int c = 0; c < cs; ++c) {
            const float *from = cs > 1 ? cl.map_shared_rank(red, c) : red;
            for (int y = 0; y < kw; ++y) v += from[(y * (8 * NT) + b) * ldr + r];
        }
        if (a.bias) v += a.bias[i];
        const int64_t at = (int64_t)(b0 + b) * a.ldy + i, at_add = (int64_t)(b0 + b) * a.ldadd + i;
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
    if (cs > 1) cl.sync();   // the others have read this CTA's sums
}

namespace {

template <int DT, int MT, int NT>
cudaError_t launch_of(const Int4Args &in, const Int4Plan &p, cudaStream_t s)
{
    Int4Args a = in;
    constexpr int T = DT == DT_F32 ? 2 : 1;
    const int nb = std::min(a.rows, 8 * NT), R = 16 * MT * (I4_NW / p.kw), G = a.k / I4_GROUP;
    a.kw = p.kw;
    a.cluster = p.cluster;
    const int per_group = 256 * T * nb + 4 * 8 * NT;
    a.chunk = std::min((G + p.cluster - 1) / p.cluster, I4_SMEM / per_group);
    const int sums = p.kw * 8 * NT * (R + 1) * 4;
    const cudaError_t e =
        cudaFuncSetAttribute(k_int4_linear<DT, MT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, I4_SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.n + R - 1) / R * p.cluster), (unsigned)((a.rows + 8 * NT - 1) / (8 * NT)));
    cfg.blockDim = dim3(I4_NT);
    cfg.dynamicSmemBytes = (size_t)std::max(a.chunk * per_group, sums);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_int4_linear<DT, MT, NT>, a);
}

template <int DT>
cudaError_t launch_dt(const Int4Args &a, int nsm, cudaStream_t s)
{
    const int G = a.k / I4_GROUP, nt = a.rows <= 8 ? 1 : a.rows <= 16 ? 2 : 4, mt = nt == 1 ? 1 : 2;
    // A CTA brings its rows of x into shared memory, so it takes about as many bytes of W.
    const int bytes_x = std::min(a.rows, 8 * nt) * (DT == DT_F32 ? 4 : 2);
    int mw = 1;
    while (mw < I4_NW && 16 * mt * mw < bytes_x) mw *= 2;
    Int4Plan p;
    p.kw = I4_NW / mw;
    const int64_t tiles = (int64_t)((a.n + 16 * mt * mw - 1) / (16 * mt * mw)) * ((a.rows + 8 * nt - 1) / (8 * nt));
    p.cluster = 1;
    // two CTAs to an SM, as long as every warp has a group of its own
    while (p.cluster < 8 && tiles * p.cluster < 2 * nsm && G >= 2 * p.cluster * p.kw) p.cluster *= 2;
    return nt == 1 ? launch_of<DT, 1, 1>(a, p, s) : nt == 2 ? launch_of<DT, 2, 2>(a, p, s) : launch_of<DT, 2, 4>(a, p, s);
}

}  // namespace

cudaError_t launch_int4_linear(const Int4Args &a, int dtype, int nsm, cudaStream_t s)
{
    switch (dtype) {
    case DT_F32: return launch_dt<DT_F32>(a, nsm, s);
    case DT_BF16: return launch_dt<DT_BF16>(a, nsm, s);
    default: return launch_dt<DT_F16>(a, nsm, s);
    }
}

}  // namespace pi
