// pi_int4_rows.cu -- projections of many rows with int4 group-128 weights, on tcgen05 (sm_103a).
//
// As pi_int4.cu (the same cut of x to f16 terms, the same f16 weights from nibbles), for batches whose products
// would bound mma.sync. A CTA has tiles of 128 rows of W and a share of the contraction, whose x stays in shared memory:
//  - weights come by TMA, boxes of 128 rows and two groups;
//  - a thread to a row turns a group's 64 bytes into 64 f16 pairs (nine operations for eight weights) and writes them to
//    tensor memory, where they are the product's A operand: nothing of the f16 weights passes through shared memory. 8 warps,
//    four to each group of a box;
//  - one thread issues a group's products, 128 x NP x 128, into an accumulator of the group's own;
//  - 8 warps, a thread to a row and half of the rows of x, read it and add it times the group's scale to the row's fp32 sums.
// Five or six groups are under way between these. CTAs of a cluster share the contraction, and send each other the sums of
// a tile: each adds up its part of the tile's rows in the order of
// the ranks, a tile later, when they have long come.
// Measured (5120 -> 15360): 16 rows fp32 23 us, 32 bf16 31, 64 fp32 45, 64 bf16 44; 12288 -> 36864: 32 bf16 120, 32 fp32 204.
// Neither the tensor pipe (13% active) nor issue slots (43%) bound it but the hand-offs: with one product of eight it took as
// long, and of a group's 750 cycles the warps of the sums worked 380, on a wait, a load, 8 to 16 sums and an arrival in turn, and
// a tile's exchange cost 2600 (stamped when the weights' offset was still in the sums). Bringing in x is 3 us (5120 in eight shares, 16 rows) to 12 us (12288,
// 32 rows), whether the first boxes are asked for before it or after.
#include <cooperative_groups.h>

#include "pi_int4.cuh"
#include "pi_umma.cuh"

namespace pi {

namespace cg = cooperative_groups;

constexpr int IR_ACC = 8, IR_COPY = IR_ACC + 8, IR_MMA = IR_COPY + 1, IR_NT = 32 * (IR_MMA + 1);   // warps
constexpr int IR_BOX = 128 * 128;   // bytes of a box: 128 rows of W, two groups
constexpr int IR_SLOTS = 4;         // places for boxes, at most
constexpr int IR_COLS = 512;
constexpr double IR_GROUP_US = 0.2, IR_TILE_US = 0.7, IR_X_US = 0.02;   // of the estimate below (measured)
// Of a CTA, at least: one to an SM. Two would wait for each other's tensor memory, and with their clusters' barriers for ever.
constexpr size_t IR_SMEM_MIN = 120 * 1024;

// NP: columns of the products, at least the rows of x that a CTA has.
template <int NP>
struct IrCfg {
    static constexpr int STAGES = NP == 32 ? 5 : 6;    // groups under way: 64 columns of weights each, NP of sums
    static_assert(STAGES * (64 + NP) <= IR_COLS);
};

struct RowsBars {
    uint64_t wfull[IR_SLOTS], wfree[IR_SLOTS], afull[6], done[6], dfree[6], sums[2];
    uint32_t tmem;
};

// A value to rank's copy of `to`, counted in bytes by rank's copy of `bar`.
__device__ __forceinline__ void send_to(float *to, float v, uint64_t *bar, int rank)
{
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\t"
        "mapa.shared::cluster.u32 a, %0, %3;\n\t"
        "mapa.shared::cluster.u32 b, %2, %3;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [a], %1, [b];\n\t}" ::"r"(smem_u32(to)),
        "r"(__float_as_uint(v)), "r"(smem_u32(bar)), "r"(rank)
        : "memory");
}

// warp_wait for a barrier that counts what other CTAs of the cluster send
__device__ __forceinline__ bool warp_wait_cluster(uint64_t *bar, uint32_t parity)
{
    auto ready = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        return ok != 0;
    };
    bool ok = ready();
    const unsigned long long t0 = globaltimer_ns();
    while (!ok && globaltimer_ns() - t0 <= WAIT_LIMIT_NS) ok = ready();
    return __all_sync(0xffffffffu, ok);
}

template <int DT, int NP>
__global__ void __launch_bounds__(IR_NT, 1) k_int4_rows(const __grid_constant__ Int4Args a, const __grid_constant__ CUtensorMap map)
{
    using C = IrCfg<NP>;
    constexpr int T = DT == DT_F32 ? 2 : 1;
    constexpr uint32_t ID = f16_idesc(0, 0, 0, 128, NP);
    extern __shared__ __align__(1024) uint8_t smem[];   // no static shared memory beside it: it starts on its alignment
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int cs = a.cluster, rank = blockIdx.x % cs, tile0 = blockIdx.x / cs, step_t = gridDim.x / cs;
    const int b0 = blockIdx.y * a.rows_per, nb = min(a.rows - b0, a.rows_per), R8 = (a.rows_per + 7) / 8 * 8;
    const int G = a.k / I4_GROUP, g_lo = (int)((int64_t)G * rank / cs), gn = (int)((int64_t)G * (rank + 1) / cs) - g_lo;
    const int tiles = (a.n + 127) / 128, pairs = (gn + 1) / 2, slots = a.slots;

    uint8_t *const ring = smem;
    uint8_t *const frag = smem + slots * IR_BOX;   // [group][term][64 columns of K][R8 rows][128 bytes], swizzled
    // (a product's columns from R8 on read on into what follows; nobody looks at them)
    float *const xu = (float *)(frag + (size_t)a.groups * T * 256 * R8 + (NP - R8) * 128);   // [group][NP]: 2 times x's unit
    float *const recv = xu + a.groups * NP;                                // [2][rank][row of x][row of W]: sums sent here
    RowsBars &bars = *(RowsBars *)(smem + a.bar_at);
    if (warp == IR_COPY && lane == 0) {
        for (int x = 0; x < slots; ++x) mbar_init(&bars.wfull[x], 1), mbar_init(&bars.wfree[x], 8);
        for (int x = 0; x < C::STAGES; ++x)
            mbar_init(&bars.afull[x], 4), mbar_init(&bars.done[x], 1), mbar_init(&bars.dfree[x], IR_ACC);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars.sums[x], 1);
            mbar_arrive_expect_tx(&bars.sums[x], 128 * nb * 4);   // a tile's sums of the rank's rows, from each rank
        }
        fence_mbar_init();
        prefetch_tensormap(&map);
    }
    __syncwarp();
    pdl_wait();
    if (warp == IR_MMA) tmem_alloc(&bars.tmem, IR_COLS);   // (not before: the last kernel may still want some)
    // A warp whose wait has run out makes no more arrivals, asks for no more copies and issues no more products; it waits
    // (again bounded) for those that it has under way and goes on to the end, where the tensor memory is freed.
    bool dead = false;   // the same in all lanes of a warp
    auto wait = [&](uint64_t *bar, uint32_t parity) {   // by the whole warp
        if (!dead && !warp_wait(bar, parity)) dead = true;
    };

    // boxes, by the loading warp
    int ask_tile = tile0, ask_pair = 0, asked = 0;
    auto request = [&]() {
        const int slot = asked % slots;
        if (lane == 0) {
            mbar_arrive_expect_tx(&bars.wfull[slot], IR_BOX);
            tma_load_2d(ring + slot * IR_BOX, &map, (g_lo + 2 * ask_pair) * 64, ask_tile * 128, &bars.wfull[slot]);
        }
        ++asked;
        if (++ask_pair == pairs) ask_pair = 0, ask_tile += step_t;
    };
    if (warp == IR_COPY)
        while (asked < slots && ask_tile < tiles) request();

    i4_take_x<DT, 8>(a, b0, nb, g_lo, gn, warp, IR_NT / 32, lane,
                  [&](int gl, int b, int term, uint2 v) {
                      const int word = lane >> 1;   // 16 bytes of a row to a word
                      uint8_t *const to = frag + ((size_t)gl * T + term) * 256 * R8 + (word >> 3) * (128 * R8);
                      *(uint2 *)(to + sw128_off(b, word & 7) + (lane & 1) * 8) = v;
                  },
                  [&](int gl, int b, float unit) { xu[gl * NP + b] = unit; });
    fence_proxy_async_smem();   // the products read it
    tc_fence_before();
    cg::cluster_group cl = cg::this_cluster();
    if (cs > 1) cl.sync();   // also: barriers are there before another rank arrives on them
    else __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();   // (a CTA of the next kernel that shares the SM may take tensor memory at its start)
    const uint32_t tmem = bars.tmem, tsum = tmem + C::STAGES * 64;

    if (warp < IR_ACC) {
        // ------------------------------------------------------------- sums: a thread to a row of W and half of the rows of x
        constexpr int H = NP / 2;
        const int half = warp >> 2, r = tid & 127, c0 = half * H;
        const uint32_t from = tsum + ((uint32_t)(warp & 3) << 21) + c0;   // (32 lanes, from bit 16 on)
        const int ro = 128 / cs, owner = r / ro;                          // the rank that adds the row up
        int it = 0;
        float sc[4], sn[4];
        auto scales = [&](int tile, int g, float (&v)[4]) {    // of four groups, or those of the next tile's first
            if (g >= gn) g = 0, tile += step_t;
            const __half *const p = a.s + (size_t)min(tile * 128 + r, a.n - 1) * G + g_lo;
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] = __half2float(p[min(g + y, gn - 1)]);
        };
        // Adds up and stores the rank's rows of its tile-th tile, of which the others have sent their sums.
        auto collect = [&](int tile, int k) {
            if (!dead && !warp_wait_cluster(&bars.sums[k & 1], (k >> 1) & 1)) dead = true;
            if (!dead && tid == 0) mbar_arrive_expect_tx(&bars.sums[k & 1], 128 * nb * 4);   // for the next tile but one
            const float *const buf = recv + (k & 1) * 128 * R8;
            for (int x = tid; x < ro * nb; x += 32 * IR_ACC) {
                const int b = x / ro, rr = x - b * ro, i = tile * 128 + rank * ro + rr;
                float v = 0.f;
                for (int c = 0; c < cs; ++c) v += buf[(c * R8 + b) * ro + rr];
                if (i < a.n) i4_store<DT>(a, dead ? __int_as_float(0x7fc00000) : v, b0 + b, i);
            }
        };
        scales(tile0, 0, sn);
        int k = 0;
        for (int tile = tile0; tile < tiles; tile += step_t, ++k) {
            float2 tot[H / 2];
#pragma unroll
            for (int x = 0; x < H / 2; ++x) tot[x] = make_float2(0.f, 0.f);
            for (int g0 = 0; g0 < gn; g0 += 4) {
#pragma unroll
                for (int y = 0; y < 4; ++y) sc[y] = sn[y] * 512.f;   // (x's unit is half of xu's, the weights' 2^-10)
                scales(tile, g0 + 4, sn);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int g = g0 + y, st = it % C::STAGES;
                    if (g >= gn) break;
                    wait(&bars.done[st], (it / C::STAGES) & 1);
                    tc_fence_after();
                    uint32_t d[H];
                    if constexpr (H == 8) tmem_ld8u(from + st * NP, d);
                    else tmem_ld16u(from + st * NP, d);
                    tmem_wait_ld(d);
                    tc_fence_before();
                    __syncwarp();
                    if (!dead && lane == 0) mbar_arrive(&bars.dfree[st]);
#pragma unroll
                    for (int x = 0; x < H; x += 4) {
                        const float4 u = *(const float4 *)&xu[g * NP + c0 + x];
                        const float2 s2 = make_float2(sc[y], sc[y]);
                        float2 v0 = make_float2(__uint_as_float(d[x]), __uint_as_float(d[x + 1]));
                        float2 v1 = make_float2(__uint_as_float(d[x + 2]), __uint_as_float(d[x + 3]));
                        v0 = fmul2(v0, make_float2(u.x, u.y));
                        v1 = fmul2(v1, make_float2(u.z, u.w));
                        tot[x / 2] = ffma2(v0, s2, tot[x / 2]);
                        tot[x / 2 + 1] = ffma2(v1, s2, tot[x / 2 + 1]);
                    }
                    ++it;
                }
            }
            const auto value = [&](int x) { return dead ? __int_as_float(0x7fc00000) : x & 1 ? tot[x / 2].y : tot[x / 2].x; };
            if (cs == 1) {
#pragma unroll
                for (int x = 0; x < H; ++x)
                    if (c0 + x < nb && tile * 128 + r < a.n) i4_store<DT>(a, value(x), b0 + c0 + x, tile * 128 + r);
                continue;
            }
            // The last tile's sums have had this tile's time to come. Then this tile's go to the buffer of two tiles ago: whoever
            // has all sums of the last tile knows that all ranks have added up those before, since they send behind the barrier.
            if (k > 0) {
                collect(tile - step_t, k - 1);
                bar_sync(1, 32 * IR_ACC);
            }
            if (!dead) {
                float *const to = recv + (k & 1) * 128 * R8 + rank * R8 * ro + r % ro;
#pragma unroll
                for (int x = 0; x < H; ++x)
                    if (c0 + x < nb) send_to(to + (c0 + x) * ro, value(x), &bars.sums[k & 1], owner);
            }
        }
        if (cs > 1 && k > 0) collect(tile0 + (k - 1) * step_t, k - 1);
    } else if (warp < IR_COPY) {
        // ------------------------------------------------------------------------------------ weights: a thread to a row of W
        const int j = (warp - IR_ACC) >> 2, r = (warp & 3) * 32 + lane;   // the group of a box
        const uint32_t to = tmem + ((uint32_t)(warp & 3) << 21);
        int box = 0, base = 0;   // boxes and groups before
        for (int tile = tile0; tile < tiles; tile += step_t, base += gn)
            for (int pair = 0; pair < pairs; ++pair, ++box) {
                const int slot = box % slots, it = base + 2 * pair + j, st = it % C::STAGES;
                wait(&bars.wfull[slot], (box / slots) & 1);
                uint4 w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) w[c] = *(const uint4 *)(ring + slot * IR_BOX + sw128_off(r, j * 4 + c));
                fence_proxy_async_smem();   // the next copy into the place comes after the loads
                __syncwarp();
                if (!dead && lane == 0) mbar_arrive(&bars.wfree[slot]);
                if (2 * pair + j >= gn) continue;   // (an odd share's last box has one group)
                if (it >= C::STAGES) wait(&bars.done[st], (it / C::STAGES - 1) & 1);   // the place's last products have read it
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int x = 0; x < 4; ++x) i4_word_h2(word4(w[c], x), *(uint32_t(*)[4])(p + 4 * x));
                    if (!dead) tmem_st16(to + st * 64 + c * 16, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (!dead && lane == 0) mbar_arrive(&bars.afull[st]);
            }
    } else if (warp == IR_COPY) {
        // ------------------------------------------------------------------------------------ copies
        while (ask_tile < tiles && !dead) {
            wait(&bars.wfree[asked % slots], (asked / slots - 1) & 1);
            if (!dead) request();
        }
        if (dead)   // nothing may land after the CTA is gone: the last copy into each place
            for (int x = 0; x < slots && x < asked; ++x) warp_wait(&bars.wfull[x], ((asked - 1 - x) / slots) & 1);
    } else {
        // ------------------------------------------------------------------------------------ products
        const uint64_t dx = sw128_desc(smem_u32(frag), 16, 1024);
        int it = 0;
        for (int tile = tile0; tile < tiles && !dead; tile += step_t)
            for (int g = 0; g < gn && !dead; ++g) {
                const int st = it % C::STAGES;
                wait(&bars.afull[st], (it / C::STAGES) & 1);
                if (it >= C::STAGES) wait(&bars.dfree[st], (it / C::STAGES - 1) & 1);
                if (dead) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int t = 0; t < T; ++t)
#pragma unroll
                        for (int s = 0; s < 8; ++s)
                            umma_f16_ts(tsum + st * NP, tmem + st * 64 + s * 8,
                                        dx + (uint32_t)(((g * T + t) * 256 * R8 + (s >> 2) * 128 * R8 + (s & 3) * 32) / 16), ID,
                                        t + s > 0);
                    umma_commit(&bars.done[st]);
                }
                __syncwarp();
                ++it;
            }
        if (dead)
            for (int x = it - 1; x >= 0 && x > it - 1 - C::STAGES; --x) warp_wait(&bars.done[x % C::STAGES], (x / C::STAGES) & 1);
    }
    tc_fence_before();
    // Sums on their way to this CTA have come, but where a wait ran out: those were sent before the barrier.
    if (cs > 1) cl.sync();
    else __syncthreads();
    if (cs > 1 && dead) {
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 100000) __nanosleep(1000);
    }
    if (warp == IR_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, IR_COLS);
    }
}

namespace {

struct RowsPlan {
    int cluster, rows_per, slots;
    size_t bar_at;
};

template <int DT, int NP>
cudaError_t launch_of(const Int4Args &in, const RowsPlan &p, const CUtensorMap &map, int nsm, cudaStream_t s)
{
    Int4Args a = in;
    a.cluster = p.cluster;
    a.rows_per = p.rows_per;
    a.slots = p.slots;
    a.groups = (a.k / I4_GROUP + p.cluster - 1) / p.cluster;
    a.bar_at = (int)p.bar_at;
    const cudaError_t e = allow_smem<k_int4_rows<DT, NP>>(I4_SMEM);
    if (e != cudaSuccess) return e;
    // CTAs stay and go through tiles: as many as the GPU holds at a time
    const int slices = (a.rows + p.rows_per - 1) / p.rows_per, tiles = (a.n + 127) / 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(std::min(tiles, std::max(1, clusters_at_once(nsm, p.cluster) / slices)) * p.cluster), (unsigned)slices);
    cfg.blockDim = dim3(IR_NT);
    cfg.dynamicSmemBytes = std::max(IR_SMEM_MIN, p.bar_at + sizeof(RowsBars));
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_int4_rows<DT, NP>, a, map);
}

template <int DT>
bool launch_dt(const Int4Args &a, int nsm, cudaStream_t s, cudaError_t *e)
{
    const int G = a.k / I4_GROUP, T = DT == DT_F32 ? 2 : 1, tiles = (a.n + 127) / 128;
    // The fastest by an estimate: rounds of tiles, each of its groups and its sums, behind bringing in x. (Up to 32 rows: with 64
    // columns the sums' registers spill, 64 rows of bf16 5120 -> 15360 59.8 us where two slices of 32 take 49.8.)
    RowsPlan p = {};
    double best = 0;
    int np = 0;
    for (int slices = (a.rows + 31) / 32; slices <= (a.rows + 7) / 8; ++slices)
        for (int cs = 1; cs <= 8; cs *= 2) {
            const int per = (a.rows + slices - 1) / slices, r8 = (per + 7) / 8 * 8, cols = per <= 16 ? 16 : 32;
            const int groups = (G + cs - 1) / cs;
            if (cs > G) continue;
            const size_t rest = (size_t)groups * (T * 256 * r8 + 4 * cols) + (cols - r8) * 128 + (cs > 1 ? 2 * 128 * 4 * r8 : 0);
            if (rest + 2 * IR_BOX + sizeof(RowsBars) > I4_SMEM) continue;
            const int slots = std::min<int>(IR_SLOTS, (int)((I4_SMEM - sizeof(RowsBars) - rest) / IR_BOX));
            // (clusters of a slice; more slices than clusters at a time go one after the other)
            const int all = clusters_at_once(nsm, cs), at_once = std::max(1, all / slices);
            const int64_t rounds = (int64_t)((tiles + at_once - 1) / at_once) * ((slices + all - 1) / all);
            const double us = rounds * (groups * IR_GROUP_US + (cs > 1 ? IR_TILE_US : 0.0)) + groups * per * IR_X_US;
            if (p.cluster == 0 || us < best) {
                best = us;
                p = RowsPlan{cs, per, slots, (slots * (size_t)IR_BOX + rest + 7) / 8 * 8};
                np = cols;
            }
        }
    if (p.cluster == 0) return false;
    // W as rows of k / 2 bytes; boxes of 128 rows and 128 bytes, swizzled. What lies past its edges reads as zeros.
    CUtensorMap map;
    if (!encode_bytes(&map, a.w, a.n, a.k / 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B))
        *e = cudaErrorUnknown;
    else
        *e = np == 16 ? launch_of<DT, 16>(a, p, map, nsm, s) : launch_of<DT, 32>(a, p, map, nsm, s);
    return true;
}

}  // namespace

bool launch_int4_rows(const Int4Args &a, int dtype, int nsm, cudaStream_t s, cudaError_t *e)
{
    return dtype == DT_F32    ? launch_dt<DT_F32>(a, nsm, s, e)
           : dtype == DT_BF16 ? launch_dt<DT_BF16>(a, nsm, s, e)
                              : launch_dt<DT_F16>(a, nsm, s, e);
}

}  // namespace pi
