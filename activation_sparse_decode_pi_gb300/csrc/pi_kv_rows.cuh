// pi_kv_rows.cuh -- attention over the paged 8-bit cache for many query rows, on tcgen05 (sm_103a).
//
// For prompt chunks: 128 rows (query token and head of the group) of one sequence and kv head against
// tiles of TOK positions. S = Q K^T and O += P V run on the tensor cores with fp32 accumulators in
// tensor memory; the weights P = 2^(S - m) go back to tensor memory as f16 and are the A operand of
// the second product. Nothing of S or P leaves the SM. The next tile's S is written over no P that a product may
// still read, and a tile's codes are read from their stage before the next copy into it is asked for.
//
// What bounds it: per 128 rows and tile the two products take 2 * 128 * TOK * D / 8192 cycles, the softmax
// about as many issue slots (one exponential and a handful of operations per score), and e4m3 has to
// become f16 in shared memory first, since a tcgen05 product takes operands of one width and 8 bits are
// too few for queries and weights. So a CTA works on NG = 2 tiles of 128 rows at once (head dim 256: one):
// a converted tile serves both, and one's products run under the other's softmax. Each has 8 warps with
// two threads to a row (a half of the tile's positions each: the softmax is latency-bound with fewer),
// whose first warp issues its products; 4 more warps convert codes, which TMA brings a tile ahead,
// into a ring of NB tiles.
// Measured: four chunks of 707..1724 tokens over 2290..6425 positions, 32 heads on 8 of 128, bf16 354 us =
// 918 TFLOP/s of the visible pairs (tensor pipe 41% active: the hand-offs between conversion, products and
// softmax bound it); one prompt of 8191 in a window of 1000 + 70, 32 heads, fp16 282 us.
// Rounding: as in pi_kv_split.cuh: q as f16 scaled per row by a power of two, weights as f16 in
// units of 2^-7 of a reference that trails the running maximum by at most 2^8 (floor 2^-31 of the
// row's largest weight). QT = 2 (fp32 output): a second f16 term of both. QT = 1: 11 bits of the weight, for fp16
// outputs as for bf16: on the windowed prompt the error against 64 bits is 2.7e-4, 2.1e-4 of it the output's rounding;
// a second term would double the second product and halve the tile.
#pragma once

#include "pi_kv_device.cuh"
#include "pi_umma.cuh"

namespace pi {

template <int D, int QT>
struct RowsCfg {
    static constexpr int NG = D == 256 ? 1 : 2;                 // groups of 128 rows
    static constexpr int ROWS = 128 * NG, RT = 2 * ROWS;        // rows, and their threads
    static constexpr int LOADERS = 128, NT = RT + LOADERS;
    static constexpr int TOK = D == 256 || QT == 2 ? 64 : 128;  // positions per tile
    static constexpr int NB = D == 256 && QT == 2 ? 1 : 2;      // tiles of K and of V in shared memory
    static constexpr int Q_BYTES = 128 * D * 2, KV_BYTES = TOK * D * 2;
    static constexpr int STAGE = TOK * D;                       // bytes of the codes of one tile
    static constexpr int DATA = NG * QT * Q_BYTES + 2 * NB * KV_BYTES + 2 * STAGE;
    // Tensor memory, per group: S (TOK columns), O (D) and, where there is room, P (two 16-bit weights to a column).
    // The tensor cores keep products in their order only where these go to one accumulator in one shape. So the next
    // tile's S is not written over weights that P V may still read: P has columns of its own (APART), or S waits until
    // P V is done (head dim 128, 16-bit types).
    static constexpr int TCOLS = 512, PCOLS = QT * TOK / 2;
    static constexpr bool APART = NG * (TOK + D + PCOLS) <= TCOLS;
    static constexpr int GCOLS = TOK + D + (APART ? PCOLS : 0);
};

constexpr float ROWS_TRAIL = 8.f;   // base-2 growth of the maximum that is taken up without rescaling
constexpr float ROWS_UNIT = 7.f;    // weights are kept times 2^7: below 2^15 with the trail

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// 32 columns of this thread's lane, asynchronously
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// 16 columns
__device__ __forceinline__ void tmem_ld16u(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// The loads above have landed; the registers pass through, so that no use of them moves up past the wait.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B: A 128 rows of f16 pairs, one pair per 32-bit column.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            bool accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accum)
        : "memory");
}

// The lowest n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// One tile for the softmax, by runs of 16 positions (each in one page).
struct RowsMeta {
    float ks[8];      // key scale
    float vexp[8];    // ROWS_UNIT + log2(value scale / unit): the value scale rides in the weight's exponent
    float vback[8];   // 2^-vexp
    float unit;       // largest value scale of the tiles so far
    float shrink;     // the last tile's unit over this one's
    uint32_t valid;   // bit per run: its page is present
    int whole;        // every row sees every position of the tile
};

__device__ __forceinline__ float lg2(float x)
{
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int ROWS, int NW>
struct RowsShared {
    uint64_t bar_s[2], bar_p[2], bar_o[2], drain[2], kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], sempty[2];
    RowsMeta meta[4];
    float half[2][ROWS];   // what the two threads of a row tell each other
    int item[4], wsum[NW], nan, last;
    KvSeq seq;
    uint32_t taddr;
};

template <int D, int QT>
constexpr int rows_smem()
{
    using C = RowsCfg<D, QT>;
    constexpr int n = C::DATA + (int)sizeof(RowsShared<C::ROWS, C::NT / 32>);
    static_assert(n <= 227 * 1024, "shared memory");
    return n;
}

template <int D, int QT>
__global__ void __launch_bounds__(RowsCfg<D, QT>::NT, 1) k_kv_rows(const __grid_constant__ KvAttendArgs a,
                                                                    const __grid_constant__ CUtensorMap mk,
                                                                    const __grid_constant__ CUtensorMap mv)
{
    using C = RowsCfg<D, QT>;
    constexpr int TOK = C::TOK, NB = C::NB, NW = C::NT / 32;
    constexpr int NBLK = D / 64, NV = TOK * D / 16 / C::LOADERS;   // 64-column blocks; 16-byte vectors per loader thread
    constexpr int RPY = C::LOADERS / 4;   // rows of a tile that the loaders take at a time
    extern __shared__ __align__(1024) uint8_t dsm[];   // no static shared memory beside it: it starts on its alignment
    uint8_t *const gq = dsm;
    const uint32_t base = smem_u32(dsm);
    if (base & 1023u) {
        if (threadIdx.x == 0) set_status(a.c.status, ST_DEVICE_CHECK);
        return;
    }
    RowsShared<C::ROWS, NW> &sh = *(RowsShared<C::ROWS, NW> *)(dsm + C::DATA);
    auto &bar_s = sh.bar_s, &bar_p = sh.bar_p, &bar_o = sh.bar_o, &kfull = sh.kfull, &kempty = sh.kempty, &vfull = sh.vfull,
         &vempty = sh.vempty, &sfull = sh.sfull, &sempty = sh.sempty;
    auto &meta = sh.meta;
    auto &s_half = sh.half;
    auto &s_item = sh.item;
    auto &wsum = sh.wsum;
    int &s_nan = sh.nan, &s_last = sh.last;
    uint32_t &taddr_s = sh.taddr;
    const uint32_t off_k = C::NG * QT * C::Q_BYTES, off_v = off_k + NB * C::KV_BYTES, off_st = off_v + NB * C::KV_BYTES;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // warp: uniform
    const KvView &c = a.c;
    const int G = c.hq / c.hkv, P = c.page;

    if (tid == 0) {
        s_item[0] = -1;
        s_nan = 0;
    }
    __syncthreads();
    pdl_wait();

    // the blockIdx.x-th item of the call: sequence, kv head, run of ROWS rows (the last rows, which see most, first)
    {
        int before = 0;
        for (int b0 = 0; b0 < a.b.n && before <= (int)blockIdx.x; b0 += C::NT) {
            const int i = b0 + tid;
            int cnt = 0, rts = 0;
            if (i < a.b.n) {
                const KvSeq q = kv_sequence(c, a.b, i, blockIdx.x == 0 && blockIdx.y == 0);
                const long long rows = (long long)q.n * G;
                rts = rows >= a.rows_from ? (int)((rows + C::ROWS - 1) / C::ROWS) : 0;
                cnt = rts * c.hkv;
            }
            int inc = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) wsum[warp] = inc;
            __syncthreads();
            int at = before + inc - cnt;
            for (int w = 0; w < NW; ++w) {
                at += w < warp ? wsum[w] : 0;
                before += wsum[w];
            }
            if (at <= (int)blockIdx.x && (int)blockIdx.x < at + cnt) {
                const int local = (int)blockIdx.x - at;
                s_item[0] = i;
                s_item[1] = rts - 1 - local / c.hkv;
                s_item[2] = local % c.hkv;
                sh.seq = kv_sequence(c, a.b, i, false);
            }
            __syncthreads();
        }
    }
    if (s_item[0] < 0) return;
    const KvSeq sq = sh.seq;
    const int h = s_item[2], row0 = s_item[1] * C::ROWS, rows = min(C::ROWS, sq.n * G - row0), p0 = sq.len - sq.n;
    const int pos_lo = p0 + row0 / G, pos_hi = p0 + (row0 + rows - 1) / G;
    // tiles [0, ns) and [w0, w1) hold what the rows see; this CTA takes its split's share of them
    const int w0 = max(0, pos_lo - a.window + 1) / TOK, w1 = pos_hi < 0 ? w0 : pos_hi / TOK + 1;
    const int ns = pos_hi >= 0 ? min((a.sinks + TOK - 1) / TOK, w0) : 0;
    const int nt_all = ns + max(w1 - w0, 0), splits = gridDim.y;
    const int k0 = (int)((long long)nt_all * blockIdx.y / splits), k1 = (int)((long long)nt_all * (blockIdx.y + 1) / splits);
    const int nt = k1 - k0;
    auto tile_of = [&](int i) { return (k0 + i < ns ? k0 + i : w0 + k0 + i - ns) * TOK; };   // its first position
    auto is_whole = [&](int j0) {
        return j0 + TOK - 1 <= pos_lo && (pos_hi - j0 < a.window || j0 + TOK <= a.sinks);
    };

    const int groups = rows > 128 ? 2 : 1;   // that have rows
    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bar_s[x], 2);   // the product, and what its issuer has seen of the loaders' (the tile's description)
            mbar_init(&bar_p[x], 1);
            mbar_init(&bar_o[x], 1);
            mbar_init(&sh.drain[x], 1);
            mbar_init(&kfull[x], C::LOADERS / 32);
            mbar_init(&vfull[x], C::LOADERS / 32);
            mbar_init(&sfull[x], x == 0 ? 2 : 1);   // keys: their bytes, and the tile's description
            mbar_init(&sempty[x], C::LOADERS / 32);
            mbar_init(&kempty[x], groups);
            mbar_init(&vempty[x], groups);
        }
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&taddr_s, C::TCOLS);
    // A warp whose wait has run out asks for no more copies and issues no more products, waits (again bounded) for those
    // that it has under way, and goes through the CTA's barriers to the end, where the tensor memory is freed.
    bool dead = false;   // the same in all lanes of a warp
    auto wait = [&](uint64_t *bar, uint32_t parity) {   // by the whole warp
        if (!dead && !warp_wait(bar, parity)) {
            dead = true;
            set_status(c.status, ST_TIMEOUT);
        }
    };
    auto wait_alone = [&](uint64_t *bar, uint32_t parity) {   // by one thread, which shares `dead` with its warp afterwards
        if (!dead && !mbar_wait(bar, parity)) {
            dead = true;
            set_status(c.status, ST_TIMEOUT);
        }
    };

    const int grp = warp >> 3, half = (warp >> 2) & 1, row = grp * 128 + (warp & 3) * 32 + lane;   // of a row's thread
    const bool mine = tid < C::RT, on = mine && row < rows;
    const int pos = on ? p0 + (row0 + row) / G : -1;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = taddr_s;
    // Only now: a CTA of the next kernel that shares the SM may take tensor memory before it waits for this one
    // (k_tc does), and the allocation above would then wait for it in turn.
    pdl_launch_dependents();

    if (!mine) {
        // ------------------------------------------------------------ loaders
        // All four warps convert. The first also asks for keys, the second describes the tiles, the third asks for
        // values: page ids are loaded a step before they are looked at, scales another step before they are used.
        const int lt = tid - C::RT, role = warp - C::RT / 32;
        const int page_shift = __ffs(P) - 1, ppt = max(1, TOK >> page_shift);   // pages per tile
        const int box_rows = min(P, KV_TILE), box_shift = __ffs(box_rows) - 1, boxes = TOK >> box_shift;
        const int pshift = __ffs(min(P, TOK)) - 1;   // of a page's positions inside a tile
        constexpr int UNSEEN = -2;
        // Page ids of tile i: lane x < ppt gets that of its x-th page as the table has it, UNSEEN where no row sees it.
        auto pages = [&](int i) {
            const int j0 = tile_of(i) + (lane << page_shift), last = j0 + min(P, TOK) - 1;
            const bool seen = i < nt && lane < ppt && j0 <= pos_hi && (j0 < a.sinks || pos_lo - last < a.window);
            return seen ? c.table[(size_t)sq.row * c.max_pages + (j0 >> page_shift)] : UNSEEN;
        };
        auto clean = [&](int pid) { return (unsigned)pid < (unsigned)c.n_pages ? pid : -1; };
        // Codes of tile i (kv 0: keys, 1: values) into their stage. Absent pages are left out.
        int asked = -1;   // last tile whose codes this warp has asked for
        auto request = [&](int kv, int i, int pid) {
            const int page = __shfl_sync(0xffffffffu, pid, lane < boxes ? (lane << box_shift) >> pshift : 0);
            const bool go = lane < boxes && page >= 0;
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, go));
            if (i > 0) wait(&sempty[kv], (i - 1) & 1);   // the loaders have read the last tile's
            if (dead) return;
            asked = i;
            if (lane == 0) mbar_arrive_expect_tx(&sfull[kv], n * box_rows * D);
            __syncwarp();
            if (go) {
                const int at = (page * c.hkv + h) * P + ((tile_of(i) + (lane << box_shift)) & (P - 1));
                uint8_t *dst = gq + off_st + kv * C::STAGE + (lane << box_shift) * (D < 128 ? D : 128);
#pragma unroll
                for (int x0 = 0; x0 < D; x0 += 128) tma_load_2d(dst + x0 * TOK, kv ? &mv : &mk, x0, at, &sfull[kv]);
            }
            __syncwarp();
        };
        // Scales of a tile's pages, one run of 16 positions to a lane, and what the softmax makes of them.
        auto scales = [&](int pid, float &ks, float &vs) {
            const int page = __shfl_sync(0xffffffffu, pid, lane < TOK / 16 ? (lane * 16) >> pshift : 0);
            const bool run = lane < TOK / 16 && page >= 0;
            ks = run ? a.l.ks[(size_t)page * c.hkv + h] : 0.f;
            vs = run ? a.l.vs[(size_t)page * c.hkv + h] : 0.f;
        };
        float unit = 0.f;
        auto describe = [&](int i, int pid, float ks, float vs) {
            RowsMeta &m = meta[i & 3];
            const bool ok = is_scale(ks) && is_scale(vs);
            if (!ok) {
                set_status(c.status, ST_DEVICE_CHECK);
                ks = vs = 0.f;
            }
            float top = vs;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = fmaxf(unit, __shfl_sync(0xffffffffu, top, 0));
            const int page = __shfl_sync(0xffffffffu, pid, (lane * 16) >> pshift);   // of the lane's run
            const uint32_t there = __ballot_sync(0xffffffffu, ok && page >= 0);
            if (lane < TOK / 16) {
                // below 2^-60 of the largest scale a page adds nothing either way; its weights still count in the sum
                const float b = (vs > 0.f ? fmaxf(lg2(vs) - lg2(top), -60.f) : -60.f) + ROWS_UNIT;
                m.ks[lane] = ks;
                m.vexp[lane] = b;
                m.vback[lane] = ex2(-b);
            }
            if (lane == 0) {
                constexpr uint32_t all = (1u << (TOK / 16)) - 1u;
                m.unit = top;
                m.shrink = top > unit ? unit / top : 1.f;
                m.valid = there & all;
                m.whole = is_whole(tile_of(i)) && (there & all) == all;
            }
            unit = top;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfull[0]);
        };
        // This thread's vectors of a tile: rows RPY y + tr, 64-column blocks b. Eight lanes hold four chunks of two
        // rows, odd rows a block off, so that reads of the stage and writes of the operand hit every bank once.
        const int tr = lt / 4, ch = lt % 4, odd = NBLK > 1 ? tr & 1 : 0;
        auto fetch = [&](int kv, int i, uint4 (&r)[NV]) {
            wait(&sfull[kv], i & 1);
            if (dead) return;
            const uint8_t *st = gq + off_st + kv * C::STAGE;
#pragma unroll
            for (int y = 0; y < TOK / RPY; ++y)
#pragma unroll
                for (int b = 0; b < NBLK; ++b) {
                    const int bb = b ^ odd;
                    const int off = D == 64 ? tr * 64 + ((ch ^ ((tr >> 1) & 3)) << 4)
                                            : (bb >> 1) * TOK * 128 + tr * 128 + ((((bb & 1) * 4 + ch) ^ (tr & 7)) << 4);
                    r[y * NBLK + b] = *(const uint4 *)(st + off + y * RPY * (D < 128 ? D : 128));
                }
            fence_proxy_async_smem();   // the next copy into the stage comes after these loads
            __syncwarp();
            if (lane == 0) mbar_arrive(&sempty[kv]);
            if (meta[i & 3].whole) return;
            // positions that no row sees and absent pages: zeros. A NaN among values that not every row sees: 0 too,
            // and the rows that see it learn of it at the end.
            const uint32_t there = meta[i & 3].valid;
            const int j0 = tile_of(i);
            const bool part = !is_whole(j0);
#pragma unroll
            for (int y = 0; y < TOK / RPY; ++y) {
                const int tok = y * RPY + tr, j = j0 + tok;
                const bool live =
                    ((there >> (tok >> 4)) & 1u) && j <= pos_hi && (j < a.sinks || pos_lo - j < a.window);
#pragma unroll
                for (int b = 0; b < NBLK; ++b) {
                    uint4 &v = r[y * NBLK + b];
                    if (!live) v = make_uint4(0, 0, 0, 0);
                    else if (kv && part && (e4m3_any_nan(v.x) | e4m3_any_nan(v.y) | e4m3_any_nan(v.z) | e4m3_any_nan(v.w))) {
                        v = make_uint4(e4m3_no_nan(v.x), e4m3_no_nan(v.y), e4m3_no_nan(v.z), e4m3_no_nan(v.w));
                        s_nan = 1;
                    }
                }
            }
        };
        const uint32_t o_lo = sw128_off(tr, ch * 2), o_hi = sw128_off(tr, ch * 2 + 1);
        auto convert = [&](uint32_t at, const uint4 (&r)[NV], uint64_t *full) {
#pragma unroll
            for (int b = 0; b < NBLK; ++b) {
                uint8_t *const lo = gq + at + (b ^ odd) * (TOK * 128) + o_lo, *const hi = lo + (int)(o_hi - o_lo);
#pragma unroll
                for (int y = 0; y < TOK / RPY; ++y) {
                    const uint4 v = r[y * NBLK + b];
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t f[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) e4m3x4_f16x4(w[e], f[2 * e], f[2 * e + 1]);
                    *(uint4 *)(lo + y * RPY * 128) = make_uint4(f[0], f[1], f[2], f[3]);
                    *(uint4 *)(hi + y * RPY * 128) = make_uint4(f[4], f[5], f[6], f[7]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
        };
        uint4 r[NV];
        int pid1 = -1, raw2 = UNSEEN;   // pages of tiles i + 1 (clean) and i + 2
        float ks1 = 0.f, vs1 = 0.f;
#pragma unroll 1
        for (int i = -3; i < nt; ++i) {
            int pid2 = -1, raw3 = UNSEEN;
            float ks2 = 0.f, vs2 = 0.f;
            if (role < 3) {
                pid2 = clean(raw2);
                if (role == 1) {
                    if (pid2 < 0 && raw2 != UNSEEN) set_status(c.status, ST_DEVICE_CHECK);   // seen, but absent
                    scales(pid2, ks2, vs2);
                }
                raw3 = pages(i + 3);
            }
            const bool next = i >= -1 && i + 1 < nt;
            const int b = i & (NB - 1);
            if (i >= 0) fetch(0, i, r);
            if (dead) break;
            // (arrivals for the next tile's keys: only after this tile's phase, which fetch has waited for)
            if (role == 0 && next) request(0, i + 1, pid1);
            if (role == 1 && next) describe(i + 1, pid1, ks1, vs1);
            if (i >= 0) {
                if (i >= NB) wait(&kempty[b], (i / NB - 1) & 1);   // the product that read the tile's place before
                if (dead) break;
                convert(off_k + b * C::KV_BYTES, r, &kfull[b]);
                fetch(1, i, r);
                if (dead) break;
            }
            if (role == 2 && next) request(1, i + 1, pid1);
            if (i >= 0) {
                if (i >= NB) wait(&vempty[b], (i / NB - 1) & 1);
                if (dead) break;
                convert(off_v + b * C::KV_BYTES, r, &vfull[b]);
            }
            pid1 = pid2;
            raw2 = raw3;
            ks1 = ks2;
            vs1 = vs2;
        }
        if (dead && asked >= 0) warp_wait(&sfull[role >> 1], asked & 1);
    }

    // ---------------------------------------------------------------- softmax
    float m = -INFINITY, l = 0.f, unit = 0.f;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + grp * C::GCOLS, to = ts + TOK, tp = C::APART ? to + D : ts;
    if (mine && grp < groups) {
        // ------------------------------------------------------------ queries: half a row to a thread
        float qf;
        {
            constexpr int QV = QT == 2 ? D / 8 : D / 16;   // 16-byte vectors (QT 2: fp32)
            uint4 raw[QV];
            const int64_t at = ((int64_t)sq.start + (row0 + row) / G) * a.ldq + (int64_t)(h * G + (row0 + row) % G) * D +
                               half * (D / 2);
            const uint4 *from = (const uint4 *)((const uint8_t *)a.q + at * (QT == 2 ? 4 : 2));
#pragma unroll
            for (int x = 0; x < QV; ++x) raw[x] = on ? from[x] : make_uint4(0, 0, 0, 0);
            auto eight = [&](int x, float (&f)[8]) {   // elements 8 x ... of the half
                if constexpr (QT == 2) {
                    float u[4], v[4];
                    unpack<DT_F32>(raw[2 * x], u);
                    unpack<DT_F32>(raw[2 * x + 1], v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = u[e], f[4 + e] = v[e];
                } else if (a.dtype == DT_BF16) {
                    unpack<DT_BF16>(raw[x], f);
                } else {
                    unpack<DT_F16>(raw[x], f);
                }
            };
            float top = 0.f;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                float f[8];
                eight(x, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_abs(f[e]));
            }
            s_half[half][row] = top;
            bar_sync(2 + grp, 256);
            top = fmaxf(top, s_half[half ^ 1][row]);
            const int ex = top > 0.f ? min(max(ilogbf(top), -118), 127) : 0;
            // the sign of the scale goes into q, so that a larger product is a larger score
            const float mul = a.scale_log2 < 0.f ? -exp2i(7 - ex) : exp2i(7 - ex);
            qf = fabsf(a.scale_log2) * exp2i(ex - 7);
            uint8_t *const dst = gq + (uint32_t)(grp * QT) * C::Q_BYTES;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                float f[8];
                uint32_t hi[4], lo[4];
                eight(x, f);
#pragma unroll
                for (int e = 0; e < 4; ++e) split_pair(f[2 * e] * mul, f[2 * e + 1] * mul, hi[e], lo[e]);
                const int ch = half * (D / 16) + x;
                const uint32_t off = (uint32_t)(ch / 8) * 16384u + sw128_off(row & 127, ch % 8);
                *(uint4 *)(dst + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if constexpr (QT == 2) *(uint4 *)(dst + C::Q_BYTES + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async_smem();
            bar_sync(2 + grp, 256);
        }
        constexpr uint32_t ID_S = f16_idesc(0, 0, 0, 128, TOK), ID_O = f16_idesc(0, 0, 1, 128, D);
        // One thread of the group's first warp issues its products. Descriptors differ in their address only (bits 0-13,
        // in 16 bytes), and everything here is uniform over the warp, so that each product is one instruction and an add.
        const uint64_t dq = sw128_desc(base + (uint32_t)(grp * QT) * C::Q_BYTES, 16u, 1024u);
        const uint64_t dk = sw128_desc(base + off_k, 16u, 1024u), dv = sw128_desc(base + off_v, TOK * 128u, 1024u);
        auto issue_s = [&](int i) {   // S = Q K^T of tile i
            const int b = i & (NB - 1);
            wait_alone(&kfull[b], (i / NB) & 1);
            if constexpr (!C::APART) {   // the last tile's P V has read the weights
                if (i > 0) wait_alone(&bar_p[grp], (i - 1) & 1);
                tc_fence_after();
            }
            if (dead) return;
            const uint64_t k1 = dk + (uint32_t)(b * C::KV_BYTES / 16);
#pragma unroll
            for (int term = QT - 1; term >= 0; --term)   // (second terms first: sums are cut off, small ones lose less)
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_f16(ts, dq + (uint32_t)((term * C::Q_BYTES + x * 16384 + j * 32) / 16),
                                 k1 + (uint32_t)((x * TOK * 128 + j * 32) / 16), ID_S, QT - 1 - term + x + j > 0);
            umma_commit(&bar_s[grp]);
            umma_commit(&kempty[b]);
            mbar_arrive(&bar_s[grp]);
        };
        auto issue_o = [&](int i) {   // O += P V
            const int b = i & (NB - 1);
            wait_alone(&vfull[b], (i / NB) & 1);
            if (dead) return;
            const uint64_t v1 = dv + (uint32_t)(b * C::KV_BYTES / 16);
#pragma unroll
            for (int term = 0; term < QT; ++term)
#pragma unroll
                for (int j = 0; j < TOK / 16; ++j)
                    umma_f16_ts(to, tp + term * (TOK / 2) + j * 8, v1 + (uint32_t)(j * 2048 / 16), ID_O,
                                i > 0 || term + j > 0);
            if constexpr (!C::APART) umma_commit(&bar_p[grp]);
            umma_commit(&vempty[b]);
            if (i + 1 == nt) umma_commit(&bar_o[grp]);
        };
        const bool issues = (warp & 7) == 0;
        if (nt > 0 && issues && elect_one()) issue_s(0);
        dead = __any_sync(0xffffffffu, dead);
        constexpr int HC = TOK / 2;   // positions of the tile that this thread takes
        const uint32_t my_s = ts + lane_base + half * HC, my_p = tp + lane_base + half * (HC / 2);
        for (int i = 0; i < nt; ++i) {
            wait(&bar_s[grp], i & 1);
            tc_fence_after();
            const RowsMeta &mt = meta[i & 3];
            uint32_t r[HC];
#pragma unroll
            for (int x = 0; x < HC; x += 32) tmem_ld32(my_s + x, r + x);
            tmem_wait_ld(r);
            if (!mt.whole) {   // what the row does not see: -infinity
                const int j0 = tile_of(i) + half * HC;
#pragma unroll
                for (int x = 0; x < HC; x += 32) {
                    const int j = j0 + x;
                    uint32_t see = low_bits(pos - j + 1);
                    see &= ~low_bits(pos - a.window + 1 - j) | low_bits(a.sinks - j);
                    const uint32_t there = mt.valid >> ((half * HC + x) / 16);
                    see &= (there & 1u ? 0xffffu : 0u) | (there & 2u ? 0xffff0000u : 0u);
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[x + e] = (see >> e) & 1u ? r[x + e] : 0xff800000u;
                }
            }
            // From product to base-2 score, by runs of 16. Never 0, so that -infinity stays what it is.
            float factor[HC / 16], top = -INFINITY;
#pragma unroll
            for (int x = 0; x < HC / 16; ++x) {
                factor[x] = fmaxf(qf * mt.ks[half * (HC / 16) + x], 1e-37f);
                float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 16; ++e) t[e & 3] = fmaxf(t[e & 3], __uint_as_float(r[x * 16 + e]));
                top = fmaxf(top, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * factor[x]);
            }
            s_half[half][row] = top;
            tc_fence_before();
            bar_sync(2 + grp, 256);   // also: every score of the group's tile has been read
            tc_fence_after();
            top = fmaxf(top, s_half[half ^ 1][row]);
            // the reference is raised when the maximum has outrun it; O follows it and the unit of the values
            float shrink = mt.shrink;
            if (top > m + ROWS_TRAIL || (m == -INFINITY && top > m)) {
                const float down = ex2(m - top);
                shrink *= down;
                l *= down;
                m = top;
            }
            unit = mt.unit;
            if (i > 0 && __any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll 1
                for (int x = half * (D / 2); x < (half + 1) * (D / 2); x += 16) {
                    uint32_t o[16];
                    tmem_ld16u(to + lane_base + x, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * shrink);
                    tmem_st16(to + lane_base + x, o);
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            uint32_t plo[QT == 2 ? HC / 2 : 1];
#pragma unroll
            for (int x = 0; x < HC / 16; ++x) {
                const float f = factor[x], off = mt.vexp[half * (HC / 16) + x] - ref;
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = x * 16; e < x * 16 + 16; e += 2) {
                    float2 w = ffma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), make_float2(f, f),
                                     make_float2(off, off));
                    w.x = ex2(w.x);
                    w.y = ex2(w.y);
                    sum = fadd2(sum, w);
                    if constexpr (QT == 2) split_pair(w.x, w.y, r[e / 2], plo[e / 2]);
                    else r[e / 2] = pack_f16(w.x, w.y);
                }
                l = fmaf(sum.x + sum.y, mt.vback[half * (HC / 16) + x], l);
                // Weights: first terms in columns [0, TOK / 2) of P, second ones behind.
                if (x & 1) {
                    tmem_st16(my_p + (x / 2) * 16, r + (x / 2) * 16);
                    if constexpr (QT == 2) tmem_st16(my_p + TOK / 2 + (x / 2) * 16, plo + (x / 2) * 16);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            bar_sync(2 + grp, 256);
            if (issues && elect_one()) {
                tc_fence_after();
                issue_o(i);
                if (i + 1 < nt) issue_s(i + 1);
            }
            dead = __any_sync(0xffffffffu, dead);
        }
        if (nt > 0) wait(&bar_o[grp], 0);
        if (dead && issues) {
            if (elect_one()) {
                umma_commit(&sh.drain[grp]);
                mbar_wait(&sh.drain[grp], 0);
            }
            __syncwarp();
        }
        tc_fence_after();

        // ------------------------------------------------------------ output
        s_half[half][row] = l;
        bar_sync(2 + grp, 256);
        l += s_half[half ^ 1][row];
        // (the unit, which may be as small as an append's 2^-120, is multiplied in by itself: its quotient would lose bits)
        const float back = exp2i(-(int)ROWS_UNIT), norm = splits > 1 ? back : l == 0.f ? 0.f : back / l;
        const int64_t at = ((int64_t)blockIdx.x * splits + blockIdx.y) * C::ROWS + row;
        const int64_t at_out = ((int64_t)sq.start + (row0 + row) / G) * a.ldo + (int64_t)(h * G + (row0 + row) % G) * D;
#pragma unroll 1
        for (int x = half * (D / 2); x < (half + 1) * (D / 2); x += 32) {
            uint32_t o[32];
            if (nt > 0) {
                tmem_ld32(to + lane_base + x, o);
                tmem_wait_ld(o);
            }
            if (on) {
                float f[32];   // l = 0: nothing seen (a NaN sum stays: it is not equal to 0)
#pragma unroll
                for (int e = 0; e < 32; ++e) f[e] = nt == 0 || l == 0.f ? 0.f : __uint_as_float(o[e]) * norm * unit;
                if (splits > 1) store_f32<32>(a.rows_part + at * D + x, f);
                else store_out<32>(a, at_out + x, f);
            }
            __syncwarp();   // the next load of tensor memory takes the whole warp, lanes past the last row too
        }
        if (splits == 1 && on && half == 0 && a.lse)
            a.lse[((int64_t)sq.start + (row0 + row) / G) * c.hq + h * G + (row0 + row) % G] = row_lse(m, l);
        if (splits > 1 && on && half == 0) {
            a.rows_ml[at * 2] = m;
            a.rows_ml[at * 2 + 1] = l;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TCOLS);
    }
    const int4 f4 = make_int4(sq.row, sq.len, sq.start, sq.n);
    if (splits > 1) {
        if (tid == 0) {   // bit 16 of the ticket: a part met a NaN value
            const uint32_t before = ticket_acq_rel(&a.rows_tickets[blockIdx.x], s_nan ? 0x10001u : 1u);
            s_last = (before & 0xffffu) == (uint32_t)splits - 1;
            s_nan |= before >> 16;
        }
        __syncthreads();
        if (!s_last) return;
        const int64_t u0 = (int64_t)blockIdx.x * splits;
        for (int x = tid; x < rows * (D / 4); x += C::NT) {
            const int r = x / (D / 4), d = (x % (D / 4)) * 4;
            float M = -INFINITY, S = 0.f;
            for (int y = 0; y < splits; ++y) M = fmaxf(M, __ldcg(&a.rows_ml[((u0 + y) * C::ROWS + r) * 2]));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int y = 0; y < splits; ++y) {
                const float my = __ldcg(&a.rows_ml[((u0 + y) * C::ROWS + r) * 2]);
                const float ly = __ldcg(&a.rows_ml[((u0 + y) * C::ROWS + r) * 2 + 1]);
                const float w = my == -INFINITY ? (ly != 0.f ? 1.f : 0.f) : ex2(my - M);
                const float4 v = __ldcg((const float4 *)&a.rows_part[((u0 + y) * C::ROWS + r) * D + d]);
                S += w * ly;
                o.x += v.x * w, o.y += v.y * w, o.z += v.z * w, o.w += v.w * w;
            }
            store_row(a, f4, h, G, D, row0 + r, d, o, M, S);
        }
        if (tid == 0) a.rows_tickets[blockIdx.x] = 0;
    }
    if (!s_nan) return;
    // NaN values among positions that not every row sees: they were left out above; here each row that
    // sees one gets it (rare, so straight from the pool).
    __syncthreads();
    if (!on || half) return;
    for (int x = 0; x < nt_all; ++x) {
        const int j0 = (x < ns ? x : w0 + x - ns) * TOK;
        if (is_whole(j0)) continue;
        for (int j = j0; j < j0 + TOK && j <= pos; ++j) {
            if (pos - j >= a.window && j >= a.sinks) continue;
            const int page = c.table[(size_t)sq.row * c.max_pages + j / P];
            if (page < 0 || page >= c.n_pages) continue;
            const size_t block = (size_t)page * c.hkv + h;
            if (!is_scale(a.l.ks[block]) || !is_scale(a.l.vs[block])) continue;
            const uint32_t *v = (const uint32_t *)(a.l.v + (block * P + (j & (P - 1))) * D);
            for (int w = 0; w < D / 4; ++w)
                if (e4m3_any_nan(v[w]))
                    for (int b = 0; b < 4; ++b)
                        if (((v[w] >> (8 * b)) & 0x7fu) == 0x7fu) store_nan(a, f4, h, G, D, row0 + row, 4 * w + b);
        }
    }
}

template <int D, int QT>
cudaError_t rows_setup()
{
    return cudaFuncSetAttribute(k_kv_rows<D, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, rows_smem<D, QT>());
}

template <int D, int QT>
cudaError_t rows_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, unsigned items,
                        unsigned splits, cudaStream_t s)
{
    Launch L;
    L.grid = dim3(items, splits);
    L.block = dim3(RowsCfg<D, QT>::NT);
    L.smem = rows_smem<D, QT>();
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    return launch_ex(L, k_kv_rows<D, QT>, a, mk, mv);
}

}  // namespace pi
