// pi_int4.cu -- projections of a few rows with int4 group-128 weights (sm_103a).
//
// y[b, i] = sum_g s[i, g] sum_{k in g} q[i, k] x[b, k]. Up to about eight rows the bytes of W bound it (half a byte a weight;
// d 12288: 226 MB in 34 us), so the rest has to hide under its loads:
//  - weights come by TMA, a box of 32 rows and two groups at a time, into places of each warp's own, so that no warp waits
//    for another's and a load costs no address arithmetic (loads to registers, 16 bytes a lane: 87 us where this takes 44);
//  - products on mma.sync m16n8k16, 16 rows of W against up to 8 rows of x: 16 bytes of a row of W to a lane are 32
//    nibbles, four lanes' a group. The contraction may run in any order that both operands share, so nibbles are used
//    as they lie: a word's nibbles (i, i + 4) become an f16 pair by a mask and one operation, and x is laid into shared
//    memory in that order. (pi_int4_rows.cu has tcgen05 products, whose hand-offs cost more than these up to 8 rows, or
//    16 of 16 bits where W has many rows.)
//  - x is cut to f16 in units of a power of two for each row and group (fp32: two terms), undone in fp32 with the
//    weights' scale, so a group's sum is of whole numbers times f16 and nothing else is rounded before fp32;
//  - one CTA to an SM stays and goes through tiles of W, x resident. Its 16 warps split a tile's rows and the
//    contraction (kw ways); CTAs of a cluster split the contraction further, where x is too large for one or the tiles are
//    few, and add their sums through distributed shared memory in the order of their ranks.
// Measured, one row (graph of calls back to back): 12288 -> 36864 bf16 45 us = 5.2 TB/s, fp32 55 us (second terms: twice the
// products; with weights left in offset binary, at five times the error, 42 and 52), 4096 -> 6144 bf16 6.7 us (launch, x, one
// tile and its sums in turn). 5120 -> 15360: 8 rows fp32 17 us, 16 rows bf16 21 us: there the products (mma.sync gives 1024 a
// cycle and SM) and the cluster's sums bound it.
#include <cooperative_groups.h>

#include <algorithm>

#include "pi_int4.cuh"

namespace pi {

namespace cg = cooperative_groups;

constexpr int I4_NT = 512, I4_NW = I4_NT / 32;
constexpr double I4_TILE_US = 0.5, I4_CLUSTER_US = 1.0, I4_X_US = 0.01;   // of the estimate below (measured)
constexpr int I4_BOX = 32 * 128;       // bytes of a box: 32 rows of W, two groups
constexpr int I4_SLOTS = 3;            // places for boxes of a warp, at most

// NT: runs of 8 rows of x.
template <int DT, int NT>
__global__ void __launch_bounds__(I4_NT, 1) k_int4_linear(const __grid_constant__ Int4Args a, const __grid_constant__ CUtensorMap map)
{
    constexpr int T = DT == DT_F32 ? 2 : 1;
    extern __shared__ __align__(1024) uint8_t smem[];   // no static shared memory beside it: it starts on its alignment
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int kw = a.kw, mw = I4_NW / kw, R = 32 * mw, slots = a.slots;
    const int cs = a.cluster, rank = blockIdx.x % cs, tile0 = blockIdx.x / cs, step_t = gridDim.x / cs;
    const int b0 = blockIdx.y * a.rows_per, nb = min(a.rows - b0, a.rows_per);
    const int G = a.k / I4_GROUP, g_lo = (int)((int64_t)G * rank / cs), gn = (int)((int64_t)G * (rank + 1) / cs) - g_lo;
    const int wk = warp % kw, wm = warp / kw;
    const int tiles = (a.n + R - 1) / R, pairs = (gn + 1) / 2;

    uint8_t *const ring = smem + warp * slots * I4_BOX;                    // the warp's boxes
    uint8_t *const frag = smem + I4_NW * slots * I4_BOX;                   // [group][word][term][row][64 bytes]
    float *const xf = (float *)(frag + (size_t)a.groups * 256 * T * nb);   // [group][8 NT]: 2 times the unit of x
    float *const red = xf + a.groups * 8 * NT;                             // [KW][8 NT][R + 1] sums
    uint64_t *const full = (uint64_t *)(smem + a.bar_at) + warp * slots;
    if (lane == 0) {
        for (int x = 0; x < slots; ++x) mbar_init(&full[x], 1);
        fence_mbar_init();
    }
    __syncwarp();
    if (tid == 0) prefetch_tensormap(&map);
    pdl_wait();
    pdl_launch_dependents();

    // The warp's boxes: of each of the CTA's tiles the pairs of groups wk, wk + kw, ... of its 32 rows
    struct Cursor {
        int tile, pair;
    };
    auto advance = [&](Cursor &c) {
        c.pair += kw;
        if (c.pair >= pairs) {
            c.pair = wk;
            c.tile += step_t;
        }
    };
    Cursor ask{wk < pairs ? tile0 : tiles, wk}, sc{ask};
    int asked = 0;   // boxes asked for
    auto request = [&](int slot) {   // the next box into a place (uniform over the warp)
        if (ask.tile >= tiles) return;
        if (lane == 0) {
            mbar_arrive_expect_tx(&full[slot], I4_BOX);
            tma_load_2d(ring + slot * I4_BOX, &map, (g_lo + 2 * ask.pair) * 64, ask.tile * R + wm * 32, &full[slot]);
        }
        ++asked;
        advance(ask);
    };
    for (int x = 0; x < slots; ++x) request(x);
    // Scales of a box, both groups of row `lane`, loaded two boxes ahead. (An odd share's last box has one group; what lies
    // behind it may be another CTA's or none.)
    const __half *sp = a.s;
    auto scale_row = [&]() { sp = a.s + (size_t)min(sc.tile * R + wm * 32 + lane, a.n - 1) * G + g_lo + 2 * wk; };
    scale_row();
    auto scale = [&]() {
        uint32_t v = 0;
        if (sc.tile < tiles) {
            v = __half_as_ushort(sp[0]);
            if (2 * sc.pair + 1 < gn) v |= (uint32_t)__half_as_ushort(sp[1]) << 16;
            sp += 2 * kw;
            const int was = sc.tile;
            advance(sc);
            if (sc.tile != was) scale_row();
        }
        return v;
    };
    uint32_t s0 = scale(), s1 = scale();

    i4_take_x<DT, 4>(a, b0, nb, g_lo, gn, warp, I4_NW, lane,
                  [&](int gl, int b, int term, uint2 v) {
                      const int word = (lane >> 1) & 3, qq = lane >> 3;
                      *(uint2 *)(frag + ((gl * 4 + word) * T * nb + b) * 64 + qq * 16 + (lane & 1) * 8 + term * 64 * nb) = v;
                  },
                  [&](int gl, int b, float unit) { xf[gl * (8 * NT) + b] = unit; });
    __syncthreads();

    // Row g of a product is row ((g & 1) << 2 | g >> 1) of a box (and 8 + that): so eight lanes' reads, two rows' halves, lie
    // in different banks of the swizzled box.
    const int rg = (g & 1) << 2 | g >> 1;
    const int wj0 = rg * 128 + ((q ^ rg) << 4), wj1 = rg * 128 + (((4 + q) ^ rg) << 4);   // the lane's chunks of a row's groups
    int xrow[NT];   // (rows past the last read another: their columns of the products are not looked at)
#pragma unroll
    for (int n = 0; n < NT; ++n) xrow[n] = min(8 * n + g, nb - 1) * 64 + q * 16;
    float tot[2][NT][4];   // of rows 16 m + ...
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) tot[m][n][e] = 0.f;
    };
    clear();
    auto step = [&](const uint8_t *box, int j, float sv, int gl) {   // group j of the box, gl of the CTA's share
        float d[T][2][NT][4];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[t][m][n][e] = 0.f;
        uint4 wv[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) wv[m][h] = *(const uint4 *)(box + m * 2048 + h * 1024 + (j ? wj1 : wj0));
        const uint8_t *const xg = frag + gl * 4 * T * nb * 64;
#pragma unroll
        for (int word = 0; word < 4; ++word) {
            uint32_t pa[2][2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) i4_word_h2(word4(wv[m][h], word), pa[m][h]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const uint4 b = *(const uint4 *)(xg + xrow[n] + (word * T + t) * nb * 64);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint32_t a0[4] = {pa[m][0][0], pa[m][1][0], pa[m][0][1], pa[m][1][1]};
                        const uint32_t a1[4] = {pa[m][0][2], pa[m][1][2], pa[m][0][3], pa[m][1][3]};
                        mma_f16(d[t][m][n], a0, b.x, b.y);
                        mma_f16(d[t][m][n], a1, b.z, b.w);
                    }
                }
        }
        float se[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) se[m][h] = __shfl_sync(0xffffffffu, sv, m * 16 + h * 8 + rg);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 u = *(const float2 *)&xf[gl * (8 * NT) + 8 * n + 2 * q];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = d[0][m][n][e];
                    if constexpr (T == 2) v += d[T - 1][m][n][e];
                    tot[m][n][e] = fmaf(v * (e & 1 ? u.y : u.x), se[m][e >> 1], tot[m][n][e]);
                }
        }
    };
    cg::cluster_group cl = cg::this_cluster();
    auto meet = [&]() {
        if (cs > 1) cl.sync();
        else __syncthreads();
    };
    int slot = 0;
    uint32_t parity = 0;
    bool dead = false;
    for (int tile = tile0; tile < tiles; tile += step_t) {
        for (int pair = wk; pair < pairs; pair += kw) {
            const float2 sv = __half22float2(u32_h2(s0));
            s0 = s1, s1 = scale();
            if (!dead && !warp_wait(&full[slot], parity)) dead = true;
            const uint8_t *const box = ring + slot * I4_BOX;
            // (x's unit is half of xf's, the weights' 2^-10)
            step(box, 0, sv.x * 512.f, 2 * pair);
            if (2 * pair + 1 < gn) step(box, 1, sv.y * 512.f, 2 * pair + 1);
            fence_proxy_async_smem();   // the next copy into the place comes after the loads
            __syncwarp();
            if (!dead) request(slot);
            if (++slot == slots) slot = 0, parity ^= 1;
        }
        if (dead) {   // a wait ran out: no number
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) tot[0][n][e] = tot[1][n][e] = __int_as_float(0x7fc00000);
        }
        // sums of the warps and of the cluster
        if (kw == 1 && cs == 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = tile * R + wm * 32 + m * 16 + (e >> 1) * 8 + rg, b = 8 * n + 2 * q + (e & 1);
                        if (b < nb && i < a.n) i4_store<DT>(a, tot[m][n][e], b0 + b, i);
                    }
        } else {
            if (tile != tile0) meet();   // the last tile's sums have been read
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = wm * 32 + m * 16 + (e >> 1) * 8 + rg, b = 8 * n + 2 * q + (e & 1);
                        if (b < nb) red[(wk * (8 * NT) + b) * (R + 1) + r] = tot[m][n][e];
                    }
            meet();
            const int r_lo = R * rank / cs, per = R * (rank + 1) / cs - r_lo;   // rows that this CTA adds up
            for (int x = tid; x < per * nb; x += I4_NT) {
                const int b = x / per, r = r_lo + x - b * per, i = tile * R + r;
                if (i >= a.n) continue;
                float v = 0.f;
                for (int c = 0; c < cs; ++c) {
                    const float *from = cs > 1 ? cl.map_shared_rank(red, c) : red;
                    for (int y = 0; y < kw; ++y) v += from[(y * (8 * NT) + b) * (R + 1) + r];
                }
                i4_store<DT>(a, v, b0 + b, i);
            }
        }
        clear();
    }
    if (dead)   // nothing may land after the CTA is gone: the last copy into each place (bounded)
        for (int x = 0; x < slots && x < asked; ++x) warp_wait(&full[x], ((asked - 1 - x) / slots) & 1);
    if (cs > 1) cl.sync();   // the others have read this CTA's sums
}

namespace {

struct Int4Plan {
    int kw, cluster, rows_per, slots;
    size_t smem, bar_at;
};

template <int DT, int NT>
cudaError_t launch_of(const Int4Args &in, const Int4Plan &p, const CUtensorMap &map, int nsm, cudaStream_t s)
{
    Int4Args a = in;
    const int R = 32 * (I4_NW / p.kw), G = a.k / I4_GROUP;
    a.kw = p.kw;
    a.cluster = p.cluster;
    a.rows_per = p.rows_per;
    a.slots = p.slots;
    a.groups = (G + p.cluster - 1) / p.cluster;
    a.bar_at = (int)p.bar_at;
    const auto kern = k_int4_linear<DT, NT>;
    cudaError_t e;
    if ((e = allow_smem<k_int4_linear<DT, NT>>(I4_SMEM)) != cudaSuccess) return e;
    // CTAs stay and go through tiles: as many as the GPU holds at a time
    const int slices = (a.rows + p.rows_per - 1) / p.rows_per, tiles = (a.n + R - 1) / R;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(std::min(tiles, std::max(1, clusters_at_once(nsm, p.cluster) / slices)) * p.cluster), (unsigned)slices);
    cfg.blockDim = dim3(I4_NT);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, map);
}

template <int DT>
cudaError_t launch_dt(const Int4Args &a, const CUtensorMap &map, int nsm, cudaStream_t s)
{
    const int G = a.k / I4_GROUP, T = DT == DT_F32 ? 2 : 1;
    Int4Plan p = {};
    // rows of x that a CTA keeps: what 8 CTAs' shared memory holds of their whole length
    const int fit = (int)std::min<int64_t>(T == 2 ? 8 : 16, (int64_t)(I4_SMEM - I4_NW * I4_BOX - 72 * 1024) / ((int64_t)(G + 7) / 8 * 256 * T));
    p.rows_per = std::min(a.rows, std::max(1, fit));
    const int nt = p.rows_per <= 8 ? 1 : 2;
    const int slices = (a.rows + p.rows_per - 1) / p.rows_per;
    // The fastest by an estimate: rounds of tiles, each as long as its bytes of W take (45 bytes a nanosecond to an SM), or
    // its products (16 NT T of 8 cycles to a warp's group, four warps to a scheduler), or a box's latency; and what a
    // tile's sums, a cluster's barriers and bringing in x cost.
    double best = 0;
    for (int cs = 1; cs <= 8; ++cs)
        for (int kw = 1; kw <= I4_NW; kw *= 2) {
            const int R = 32 * (I4_NW / kw), groups = (G + cs - 1) / cs;
            const size_t sums = kw == 1 && cs == 1 ? 0 : (size_t)kw * 8 * nt * (R + 1) * 4;
            const size_t rest = ((size_t)groups * (256 * T * p.rows_per + 32 * nt) + sums + 7) / 8 * 8 + 8 * I4_NW * I4_SLOTS;
            if (rest + I4_NW * I4_BOX > I4_SMEM) continue;
            const int n_slots = std::min<int>(I4_SLOTS, (int)((I4_SMEM - rest) / (I4_NW * I4_BOX)));
            const int64_t tiles = (int64_t)((a.n + R - 1) / R) * slices;
            const int64_t rounds = (tiles + clusters_at_once(nsm, cs) - 1) / clusters_at_once(nsm, cs);
            const int boxes = ((groups + 1) / 2 + kw - 1) / kw;
            const double tile_us = std::max({boxes * kw * (R / 32) * I4_BOX / 45e3, boxes * 2 * 0.27 * nt * T, boxes * 0.15});
            const double us = (double)rounds * (tile_us + I4_TILE_US * (sums > 0) + (cs > 1 ? I4_CLUSTER_US : 0.0)) +
                              (double)groups * p.rows_per * I4_X_US;
            if (p.cluster == 0 || us < best) {
                best = us;
                p.cluster = cs;
                p.kw = kw;
                p.slots = n_slots;
                p.bar_at = (size_t)I4_NW * n_slots * I4_BOX + rest - 8 * I4_NW * I4_SLOTS;
                p.smem = p.bar_at + (size_t)8 * I4_NW * n_slots;
            }
        }
    if (p.cluster == 0) return cudaErrorInvalidConfiguration;
    if constexpr (DT != DT_F32)
        if (nt == 2) return launch_of<DT, 2>(a, p, map, nsm, s);
    return launch_of<DT, 1>(a, p, map, nsm, s);
}

}  // namespace

cudaError_t launch_int4_linear(const Int4Args &a, int dtype, int nsm, cudaStream_t s)
{
    // The other kernel is faster for more than 8 rows of fp32 (two terms). Measured in us, this against that, 8 and 9 rows:
    // 5120 -> 15360 16.9 / 21.0 and 27.8 / 21.6, 12288 -> 36864 65 / 83 and 115 / 99, 5120 -> 5120 10.8 / 11.4 and 14.1 / 11.6,
    // 640 -> 40000 8.6 / 10.2 and 13.5 / 10.3 (1024 -> 2560 has it at 7 rows: 5.8 / 5.1). For more than 16 of 16 bits, 16 and 20 rows:
    // 20.8 / 22.8 and 36.4 / 25.6, 76 / 87 and 131 / 95, 640 -> 40000 10.0 / 10.8 and 15.5 / 13.1. But for more than 8 of 16 bits too
    // where W has few tiles, which this kernel spreads over clusters: 9 and 16 rows 5120 -> 5120 11.1 / 11.3 and 14.2 / 12.1,
    // 1024 -> 2560 6.7 / 5.3 and 8.5 / 5.6, 4096 -> 6144 (48 tiles of 128 rows) 12.0 / 11.8 and 12.7 / 12.9.
    const bool small = (a.n + 127) / 128 * 3 <= nsm;
    cudaError_t e;
    if (a.rows > (dtype == DT_F32 || small ? 8 : 16) && launch_int4_rows(a, dtype, nsm, s, &e)) return e;
    // W as rows of k / 2 bytes; boxes of 32 rows and 128 bytes, swizzled. What lies past its edges reads as zeros.
    CUtensorMap map;
    if (!encode_bytes(&map, a.w, a.n, a.k / 2, 32, 128, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorUnknown;
    switch (dtype) {
    case DT_F32: return launch_dt<DT_F32>(a, map, nsm, s);
    case DT_BF16: return launch_dt<DT_BF16>(a, map, nsm, s);
    default: return launch_dt<DT_F16>(a, map, nsm, s);
    }
}

}  // namespace pi
