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
constexpr int I4_SMEM = 208 * 1024;   // of a CTA at most
constexpr int I4_BATCH = 4;           // runs of 16 rows by 128 of a warp that are loaded at a time

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

// MT: runs of 16 rows of W to a warp; NT: runs of 8 rows of x.
// CTAs to an SM, as registers allow, and places for a tile's sums.
template <int DT, int NT>
struct Int4Cfg {
    static constexpr int CTAS = NT == 4 || (NT == 2 && DT == DT_F32) ? 1 : 2, SUMS = NT == 4 ? 1 : 2;
};

template <int DT, int MT, int NT>
__global__ void __launch_bounds__(I4_NT, Int4Cfg<DT, NT>::CTAS) k_int4_linear(const Int4Args a)
{
    constexpr int T = DT == DT_F32 ? 2 : 1;
    constexpr int U = I4_BATCH / MT;   // groups whose weights are loaded at a time
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int kw = a.kw, mw = I4_NW / kw, R = 16 * MT * mw;
    const int cs = a.cluster, rank = blockIdx.x % cs, tile0 = blockIdx.x / cs, step_t = gridDim.x / cs;
    const int b0 = blockIdx.y * a.rows_per, nb = min(a.rows - b0, a.rows_per);
    const int G = a.k / I4_GROUP, g_lo = (int)((int64_t)G * rank / cs), gn = (int)((int64_t)G * (rank + 1) / cs) - g_lo;
    const int wk = warp % kw, wm = warp / kw;
    const size_t row_bytes = (size_t)a.k / 2;
    const int tiles = (a.n + R - 1) / R;

    uint8_t *const frag = smem;                                            // [group][word][term][row][64 bytes]
    float *const xf = (float *)(smem + (size_t)a.groups * 256 * T * nb);   // [group][8 NT] units of x
    float *const red = xf + a.groups * 8 * NT;                             // [SUMS][KW][8 NT][R + 1] sums

    // Into L2 before the previous kernel's results are waited for (a hint: nothing is read yet).
    for (int r = tid; r < R; r += I4_NT) {
        const int at = tile0 * R + r;
        if (at < a.n) prefetch_l2(a.w + (size_t)at * row_bytes + (size_t)g_lo * 64, (uint32_t)gn * 64u);
    }
    pdl_wait();
    pdl_launch_dependents();

    // Batches of U groups: every warp has the same number to a tile, the last ones partly or wholly past its groups. A
    // batch's weights are loaded while the one before is worked on, from one tile into the next.
    const int per_tile = max(1, ((gn + kw - 1) / kw + U - 1) / U);
    uint4 w[2][U][MT][2];
    __half s[2][U][MT][2];
    int lt = tile0, lb = 0;   // the next batch to load
    auto load = [&](int buf) {
        if (lt >= tiles) return;
        const int row0 = lt * R + wm * 16 * MT + g;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int gr = (lb * U + u) * kw + wk;
            if (gr < gn) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // (rows past the last read the last: their results are not stored)
                        const size_t r = (size_t)min(row0 + m * 16 + h * 8, a.n - 1);
                        w[buf][u][m][h] = ld_stream((const uint4 *)(a.w + r * row_bytes + (size_t)(g_lo + gr) * 64 + q * 16));
                        s[buf][u][m][h] = a.s[r * G + g_lo + gr];
                    }
            }
        }
        if (++lb == per_tile) {
            lb = 0;
            lt += step_t;
        }
    };
    load(0);

    // x: a warp to a row's group, four elements to a lane, four groups' loads under way at a time
    constexpr int S = 4;
    for (int it0 = warp; it0 < gn * nb; it0 += S * I4_NW) {
        float f[S][4];
#pragma unroll
        for (int y = 0; y < S; ++y) {
            const int it = it0 + y * I4_NW, gl = it / nb, b = it - gl * nb;
            if (it >= gn * nb) break;
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
        float top[S];
#pragma unroll
        for (int y = 0; y < S; ++y)
            top[y] = fmaxf(fmaxf(finite_abs(f[y][0]), finite_abs(f[y][1])), fmaxf(finite_abs(f[y][2]), finite_abs(f[y][3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int y = 0; y < S; ++y) top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], o));
#pragma unroll
        for (int y = 0; y < S; ++y) {
            const int it = it0 + y * I4_NW, gl = it / nb, b = it - gl * nb;
            if (it >= gn * nb) break;
            // 2^ex <= top < 2^(ex + 1): the largest lies in [128, 256) (zeros and the smallest numbers below)
            const int ex = max((int)(__float_as_uint(top[y]) >> 23) - 127, -118);
            const float mul = exp2i(7 - ex);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[y][e] *= mul;
            // a word's elements 0..3 lie in an even lane, 4..7 in the next: the even lane takes pairs (0, 4) and (1, 5)
            const bool odd = lane & 1;
            const float p0 = __shfl_xor_sync(0xffffffffu, odd ? f[y][0] : f[y][2], 1);
            const float p1 = __shfl_xor_sync(0xffffffffu, odd ? f[y][1] : f[y][3], 1);
            const float x0 = odd ? p0 : f[y][0], y0 = odd ? f[y][2] : p0, x1 = odd ? p1 : f[y][1], y1 = odd ? f[y][3] : p1;
            const int word = (lane >> 1) & 3, qq = lane >> 3;
            uint8_t *const to = frag + ((gl * 4 + word) * T * nb + b) * 64 + qq * 16 + odd * 8;
            const uint32_t h0 = pack_f16(x0, y0), h1 = pack_f16(x1, y1);
            *(uint2 *)to = make_uint2(h0, h1);
            if constexpr (T == 2) {
                const float2 c0 = __half22float2(u32_h2(h0)), c1 = __half22float2(u32_h2(h1));
                // (an infinity has no second term)
                const auto rest = [](float v, float c) { return fabsf(c) <= 65504.f ? v - c : 0.f; };
                *(uint2 *)(to + 64 * nb) = make_uint2(pack_f16(rest(x0, c0.x), rest(y0, c0.y)), pack_f16(rest(x1, c1.x), rest(y1, c1.y)));
            }
            if (lane == 0) xf[gl * (8 * NT) + b] = exp2i(ex - 7);
        }
    }
    __syncthreads();

    float tot[MT][NT][4];
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) tot[m][n][e] = 0.f;
    };
    clear();
    auto step = [&](const uint4 (&wv)[MT][2], const __half (&sv)[MT][2], int gl) {
        float d[T][MT][NT][4];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[t][m][n][e] = 0.f;
        const uint8_t *const xg = frag + gl * 4 * T * nb * 64 + g * 64 + q * 16;
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
                    if (8 * n + g < nb) b = *(const uint4 *)(xg + ((word * T + t) * nb + 8 * n) * 64);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint32_t a0[4] = {pa[m][0][0], pa[m][1][0], pa[m][0][1], pa[m][1][1]};
                        const uint32_t a1[4] = {pa[m][0][2], pa[m][1][2], pa[m][0][3], pa[m][1][3]};
                        mma_f16(d[t][m][n], a0, b.x, b.y);
                        mma_f16(d[t][m][n], a1, b.z, b.w);
                    }
                }
        }
        float sc[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) sc[m][h] = __half2float(sv[m][h]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 u = *(const float2 *)&xf[gl * (8 * NT) + 8 * n + 2 * q];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = d[0][m][n][e];
                    if constexpr (T == 2) v += d[T - 1][m][n][e];
                    tot[m][n][e] = fmaf(v * (e & 1 ? u.y : u.x), sc[m][e >> 1], tot[m][n][e]);
                }
        }
    };
    cg::cluster_group cl = cg::this_cluster();
    int ct = tile0, cb = 0, turn = 0;   // the batch that is worked on; sums alternate between two places
    auto batch = [&](int buf) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int gr = (cb * U + u) * kw + wk;
            if (gr < gn) step(w[buf][u], s[buf][u], gr);
        }
        if (++cb < per_tile) return;
        // the tile's end: sums of the warps and of the cluster
        cb = 0;
        float *const to = red + turn * (kw * 8 * NT * (R + 1));
        auto meet = [&]() {
            if (cs > 1) cl.sync();
            else __syncthreads();
        };
        if constexpr (Int4Cfg<DT, NT>::SUMS == 2) turn ^= 1;
        else if (ct != tile0) meet();   // the last tile's sums have been read
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = wm * 16 * MT + m * 16 + (e >> 1) * 8 + g, b = 8 * n + 2 * q + (e & 1);
                    if (b < nb) to[(wk * (8 * NT) + b) * (R + 1) + r] = tot[m][n][e];
                }
        clear();
        meet();
        const int per = R / cs;   // rows that this CTA adds up
        for (int x = tid; x < per * nb; x += I4_NT) {
            const int b = x / per, r = rank * per + x - b * per, i = ct * R + r;
            if (i >= a.n) continue;
            float v = 0.f;
            for (int c = 0; c < cs; ++c) {
                const float *from = cs > 1 ? cl.map_shared_rank(to, c) : to;
                for (int y = 0; y < kw; ++y) v += from[(y * (8 * NT) + b) * (R + 1) + r];
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
        ct += step_t;
    };
    while (ct < tiles) {
        load(1);
        batch(0);
        if (ct >= tiles) break;
        load(0);
        batch(1);
    }
    if (cs > 1) cl.sync();   // the others have read this CTA's sums
}

namespace {

struct Int4Plan {
    int mw, cluster, rows_per;
};

template <int DT, int MT, int NT>
cudaError_t launch_of(const Int4Args &in, const Int4Plan &p, int nsm, cudaStream_t s)
{
    Int4Args a = in;
    constexpr int T = DT == DT_F32 ? 2 : 1;
    const int nb = std::min(a.rows, p.rows_per), R = 16 * MT * p.mw, G = a.k / I4_GROUP;
    a.kw = I4_NW / p.mw;
    a.cluster = p.cluster;
    a.rows_per = p.rows_per;
    a.groups = (G + p.cluster - 1) / p.cluster;
    const auto kern = k_int4_linear<DT, MT, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, I4_SMEM);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)a.groups * (256 * T * nb + 4 * 8 * NT) + (size_t)Int4Cfg<DT, NT>::SUMS * a.kw * 8 * NT * (R + 1) * 4;
    // CTAs stay and go through tiles: as many as the GPU holds at a time
    const int slices = (a.rows + p.rows_per - 1) / p.rows_per, hold = smem <= I4_SMEM / 2 ? Int4Cfg<DT, NT>::CTAS * nsm : nsm;
    const int tiles = (a.n + R - 1) / R, room = std::max(1, hold / (p.cluster * slices));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(std::min(tiles, room) * p.cluster), (unsigned)slices);
    cfg.blockDim = dim3(I4_NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int DT>
cudaError_t launch_dt(const Int4Args &a, int nsm, cudaStream_t s)
{
    const int G = a.k / I4_GROUP, T = DT == DT_F32 ? 2 : 1;
    Int4Plan p;
    // rows of x that a CTA keeps: what 8 CTAs' shared memory holds of their whole length
    const int fit = (int)std::min<int64_t>(32, (int64_t)(I4_SMEM - 40 * 1024) / ((int64_t)(G + 7) / 8 * 256 * T));
    p.rows_per = std::min(a.rows, std::max(1, fit));
    const int nt = p.rows_per <= 8 ? 1 : p.rows_per <= 16 ? 2 : 4, mt = nt == 1 ? 1 : 2;
    // A CTA brings its rows of x into shared memory, so its share of W should be larger.
    p.mw = 1;
    while (p.mw < I4_NW && 16 * mt * p.mw < p.rows_per * 2 * T) p.mw *= 2;
    const int kw = I4_NW / p.mw, slices = (a.rows + p.rows_per - 1) / p.rows_per;
    const int64_t tiles = (int64_t)((a.n + 16 * mt * p.mw - 1) / (16 * mt * p.mw)) * slices;
    const size_t sums = (size_t)(nt == 4 ? 1 : 2) * kw * 8 * nt * (16 * mt * p.mw + 1) * 4;
    p.cluster = 1;
    while (p.cluster < 8 && (size_t)((G + p.cluster - 1) / p.cluster) * (256 * T * p.rows_per + 32 * nt) + sums > I4_SMEM) p.cluster *= 2;
    // two CTAs to an SM, as long as every warp has a group of its own
    while (p.cluster < 8 && tiles * p.cluster < nsm && G >= 2 * p.cluster * kw) p.cluster *= 2;
    return nt == 1   ? launch_of<DT, 1, 1>(a, p, nsm, s)
           : nt == 2 ? launch_of<DT, 2, 2>(a, p, nsm, s)
                     : launch_of<DT, 2, 4>(a, p, nsm, s);
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
