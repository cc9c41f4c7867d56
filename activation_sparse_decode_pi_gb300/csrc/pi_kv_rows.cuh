// pi_kv_rows.cuh -- attention over the paged 8-bit cache for many query rows, on tcgen05 (sm_103a).
//
// For prompt chunks: 128 rows (query token and head of the group) of one sequence and kv head against
// tiles of TOK positions. S = Q K^T and O += P V run on the tensor cores with fp32 accumulators in
// tensor memory; the weights P = 2^(S - m) go back to tensor memory as f16 and are the A operand of
// the second product. Nothing of S or P leaves the SM.
//
// What bounds it: per 128 rows and tile the two products take 2 * 128 * TOK * D / 8192 cycles, the softmax
// about as many issue slots (one exponential and a handful of operations per score), and e4m3 has to
// become f16 in shared memory first, since a tcgen05 product takes operands of one width and 8 bits are
// too few for queries and weights. So a CTA works on NG = 2 tiles of 128 rows at once (head dim 256: one):
// a converted tile serves both, and one's products run under the other's softmax. Each has 4 warps
// with a row per thread, whose first thread issues its products; 4 more warps load codes (16-byte
// loads, a tile ahead in registers) and convert them into a ring of NB tiles.
// Rounding: as in pi_kv_split.cuh: q as f16 scaled per row by a power of two, weights as f16 in
// units of 2^-7 of a reference that trails the running maximum by at most 2^8 (floor 2^-31 of the
// row's largest weight). QT = 2 (fp32 output): a second f16 term of both.
#pragma once

#include "pi_kv_device.cuh"
#include "pi_umma.cuh"

namespace pi {

template <int D, int QT>
struct RowsCfg {
    static constexpr int NG = D == 256 ? 1 : 2;                 // groups of 128 rows
    static constexpr int ROWS = 128 * NG, NT = ROWS + 128;      // threads: a row each, and the loaders
    static constexpr int TOK = D == 256 || QT == 2 ? 64 : 128;  // positions per tile
    static constexpr int NB = D == 256 && QT == 2 ? 1 : 2;      // tiles of K and of V in shared memory
    static constexpr int Q_BYTES = 128 * D * 2, KV_BYTES = TOK * D * 2;
    static constexpr int SMEM = 1024 + NG * QT * Q_BYTES + 2 * NB * KV_BYTES;
    static constexpr int TCOLS = 512;                           // per group: S (TOK columns) and O (D columns)
};

constexpr float ROWS_TRAIL = 8.f;   // base-2 growth of the maximum that is taken up without rescaling
constexpr float ROWS_UNIT = 7.f;    // weights are kept times 2^7: below 2^15 with the trail

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
__device__ __forceinline__ uint32_t low_bits(long long n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << (int)n) - 1u;
}

// Pages of one tile for the softmax: scale factors and which are there.
struct RowsMeta {
    float ks[8];      // key scale
    float vexp[8];    // ROWS_UNIT + log2(value scale / unit): the value scale rides in the weight's exponent
    float vback[8];   // 2^-vexp
    float unit;       // largest value scale of the tiles so far
    float shrink;     // the last tile's unit over this one's
    uint32_t valid;   // bit per page: present
    int whole;        // every row sees every position of the tile
};

template <int D, int QT>
__global__ void __launch_bounds__(RowsCfg<D, QT>::NT, 1) k_kv_rows(const __grid_constant__ KvAttendArgs a)
{
    using C = RowsCfg<D, QT>;
    constexpr int TOK = C::TOK, NB = C::NB, NW = C::NT / 32;
    constexpr int NBLK = D / 64, NV = TOK * D / 16 / 128;   // 64-column blocks; 16-byte vectors per loader thread
    extern __shared__ uint8_t dsm[];
    __shared__ uint64_t bar_s[2], bar_o[2], kfull[2], kempty[2], vfull[2], vempty[2];
    __shared__ uint32_t taddr_s;
    __shared__ RowsMeta meta[4];
    __shared__ int s_item[4], wsum[NW], s_nan, s_last;
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    uint8_t *const gq = dsm + (base - smem_u32(dsm));
    const uint32_t off_k = C::NG * QT * C::Q_BYTES, off_v = off_k + NB * C::KV_BYTES;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KvView &c = a.c;
    const int G = c.hq / c.hkv, P = c.page;

    if (tid == 0) {
        s_item[0] = -1;
        s_nan = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

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
            }
            __syncthreads();
        }
    }
    if (s_item[0] < 0) return;
    const KvSeq sq = kv_sequence(c, a.b, s_item[0], false);
    const int h = s_item[2], row0 = s_item[1] * C::ROWS, rows = min(C::ROWS, sq.n * G - row0), p0 = sq.len - sq.n;
    const int pos_lo = p0 + row0 / G, pos_hi = p0 + (row0 + rows - 1) / G;
    // tiles [0, ns) and [w0, w1) hold what the rows see; this CTA takes its split's share of them
    const long long low = a.window > 0 ? max(0ll, (long long)pos_lo - a.window + 1) : 0ll;
    const int w0 = (int)(low / TOK), w1 = pos_hi < 0 ? w0 : pos_hi / TOK + 1;
    const int ns = a.window > 0 && pos_hi >= 0 ? (int)min(((long long)a.sinks + TOK - 1) / TOK, (long long)w0) : 0;
    const int nt_all = ns + max(w1 - w0, 0), splits = gridDim.y;
    const int k0 = (int)((long long)nt_all * blockIdx.y / splits), k1 = (int)((long long)nt_all * (blockIdx.y + 1) / splits);
    const int nt = k1 - k0;
    auto tile_of = [&](int i) { return (k0 + i < ns ? k0 + i : w0 + k0 + i - ns) * TOK; };   // its first position
    auto is_whole = [&](int j0) {
        return j0 + TOK - 1 <= pos_lo && (a.window <= 0 || (long long)pos_hi - j0 < a.window || j0 + TOK <= a.sinks);
    };

    const int groups = rows > 128 ? 2 : 1;   // that have rows
    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bar_s[x], 2);   // the product, and what its issuer has seen of the loaders' (the tile's description)
            mbar_init(&bar_o[x], 1);
            mbar_init(&kfull[x], 4);
            mbar_init(&vfull[x], 4);
            mbar_init(&kempty[x], groups);
            mbar_init(&vempty[x], groups);
        }
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&taddr_s, C::TCOLS);
    bool dead = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity)) {
            dead = true;
            set_status(c.status, ST_TIMEOUT);
        }
    };

    // ---------------------------------------------------------------- queries: a row per thread
    float qf = 0.f;
    const bool on = tid < rows;
    const int grp = warp >> 2;   // of a row's thread
    const int pos = on ? p0 + (row0 + tid) / G : -1;
    if (tid < C::ROWS) {
        const int64_t at = on ? ((int64_t)sq.start + (row0 + tid) / G) * a.ldq + (int64_t)(h * G + (row0 + tid) % G) * D : 0;
        float top = 0.f;
        if (on) {
#pragma unroll 4
            for (int x = 0; x < D / 16; ++x) {
                float f[16];
                load16(a.q, a.dtype, at + x * 16, f);
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, finite_abs(f[e]));
            }
        }
        const int ex = top > 0.f ? min(max(ilogbf(top), -118), 127) : 0;
        // the sign of the scale goes into q, so that a larger product is a larger score
        const float mul = a.scale_log2 < 0.f ? -exp2i(7 - ex) : exp2i(7 - ex);
        qf = fabsf(a.scale_log2) * exp2i(ex - 7);
#pragma unroll 2
        for (int x = 0; x < D / 16; ++x) {
            float f[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = 0.f;
            if (on) load16(a.q, a.dtype, at + x * 16, f);
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) split_pair(f[2 * e] * mul, f[2 * e + 1] * mul, hi[e], lo[e]);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t off = (uint32_t)(grp * QT) * C::Q_BYTES + (uint32_t)(x / 4) * 16384u + sw128_off(tid & 127, (x % 4) * 2 + hf);
                *(uint4 *)(gq + off) = make_uint4(hi[4 * hf], hi[4 * hf + 1], hi[4 * hf + 2], hi[4 * hf + 3]);
                if constexpr (QT == 2)
                    *(uint4 *)(gq + C::Q_BYTES + off) = make_uint4(lo[4 * hf], lo[4 * hf + 1], lo[4 * hf + 2], lo[4 * hf + 3]);
            }
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = taddr_s;

    if (tid >= C::ROWS) {
        // ------------------------------------------------------------ loaders
        const int lt = tid - C::ROWS;
        const int ppt = P >= TOK ? 1 : TOK / P;   // pages per tile
        float unit = 0.f;
        // page ids of tile i: lane x < ppt holds that of its x-th page (-1: no row sees it, or it is absent)
        auto pages = [&](int i) {
            int page = -1;
            const int j0 = tile_of(i) + lane * P;
            if (lane < ppt && j0 <= pos_hi) {
                const int end = j0 + min(P, TOK);
                if (a.window <= 0 || j0 < a.sinks || (long long)pos_lo - (end - 1) < a.window) {
                    page = c.table[(size_t)sq.row * c.max_pages + j0 / P];
                    if (page < 0 || page >= c.n_pages) {
                        set_status(c.status, ST_DEVICE_CHECK);
                        page = -1;
                    }
                }
            }
            return page;
        };
        // This thread's vectors of a tile: x = 0, 1, ...: 64-column block x % NBLK of row 32 (x / NBLK) + tr. Eight
        // lanes hold four chunks of two rows, whose places in the swizzled atoms fall into different banks.
        const int tr = lt / 4, ch = lt % 4, pshift = __ffs(min(P, TOK)) - 1;
        auto fetch = [&](const uint8_t *pool, int i, int pid, uint4 (&r)[NV]) {
            const int j0 = tile_of(i);
            const bool whole = is_whole(j0);
            const uint8_t *from = pool + (size_t)((j0 & (P - 1)) * D + ch * 16);
#pragma unroll
            for (int y = 0; y < TOK / 32; ++y) {
                const int tok = y * 32 + tr;
                const int page = __shfl_sync(0xffffffffu, pid, tok >> pshift);
                bool live = page >= 0;
                if (!whole) {
                    const int j = j0 + tok;
                    live = live && j <= pos_hi && (a.window <= 0 || j < a.sinks || (long long)pos_lo - j < a.window);
                }
                const uint8_t *row = from + (size_t)(unsigned)(page * c.hkv + h) * (unsigned)(P * D) +
                                     (tok & ((1 << pshift) - 1)) * D;
#pragma unroll
                for (int b = 0; b < NBLK; ++b)
                    r[y * NBLK + b] = live ? ld_codes((const uint4 *)(row + b * 64)) : make_uint4(0, 0, 0, 0);
            }
        };
        const uint32_t o_lo = sw128_off(tr, ch * 2), o_hi = sw128_off(tr, ch * 2 + 1);
        auto convert = [&](uint32_t at, const uint4 (&r)[NV]) {
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                const uint32_t w[4] = {r[x].x, r[x].y, r[x].z, r[x].w};
                uint32_t f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) e4m3x4_f16x4(w[e], f[2 * e], f[2 * e + 1]);
                uint8_t *dst = gq + at + (x % NBLK) * (TOK * 128) + (x / NBLK) * 32 * 128;
                *(uint4 *)(dst + o_lo) = make_uint4(f[0], f[1], f[2], f[3]);
                *(uint4 *)(dst + o_hi) = make_uint4(f[4], f[5], f[6], f[7]);
            }
        };
        // A NaN value in a tile that not every row sees in full: 0 here, and the rows that see it learn of it at the end.
        auto strip_nan = [&](int i, uint4 (&r)[NV]) {
            if (is_whole(tile_of(i))) return;
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                uint32_t *w = &r[x].x;
                for (int e = 0; e < 4; ++e)
                    if (e4m3_any_nan(w[e])) {
                        for (int b = 0; b < 32; b += 8)
                            if (((w[e] >> b) & 0x7fu) == 0x7fu) w[e] &= ~(0xffu << b);
                        s_nan = 1;
                    }
            }
        };
        // Scales of the pages of a tile (lanes as in pages()), and what the softmax makes of them.
        auto scales = [&](int pid, float &ks, float &vs) {
            ks = pid >= 0 ? a.l.ks[(size_t)pid * c.hkv + h] : 0.f;
            vs = pid >= 0 ? a.l.vs[(size_t)pid * c.hkv + h] : 0.f;
        };
        auto describe = [&](int i, int pid, float ks, float vs) {
            RowsMeta &m = meta[i & 3];
            if (warp != C::ROWS / 32) return;
            float top = vs;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = fmaxf(unit, __shfl_sync(0xffffffffu, top, 0));
            const uint32_t there = __ballot_sync(0xffffffffu, pid >= 0);
            if (lane < ppt) {
                // below 2^-60 of the largest scale a page adds nothing either way; its weights still count in the sum
                const float b = (vs > 0.f ? fmaxf(log2f(vs / top), -60.f) : -60.f) + ROWS_UNIT;
                m.ks[lane] = ks;
                m.vexp[lane] = b;
                m.vback[lane] = ex2(-b);
            }
            if (lane == 0) {
                m.unit = top;
                m.shrink = top > unit ? unit / top : 1.f;
                m.valid = there;
                m.whole = is_whole(tile_of(i)) && there == (1u << ppt) - 1u;
            }
            unit = top;
        };
        auto ready = [&](uint64_t *bar) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // Codes and scales are asked for a tile ahead, page ids two.
        uint4 kr[NV], vr[NV];
        int pid0 = -1, pid1 = nt > 0 ? pages(0) : -1;
        float ks0 = 0.f, vs0 = 0.f;
#pragma unroll 1
        for (int i = -1; i < nt; ++i) {
            const int pid2 = i + 2 < nt ? pages(i + 2) : -1, b = i & (NB - 1);
            if (i >= 0) {
                if (i >= NB) wait(&kempty[b], (i / NB - 1) & 1);
                describe(i, pid0, ks0, vs0);
                convert(off_k + b * C::KV_BYTES, kr);
                ready(&kfull[b]);
            }
            if (i + 1 < nt) {
                scales(pid1, ks0, vs0);
                fetch(a.l.k, i + 1, pid1, kr);
            }
            if (i >= 0) {
                strip_nan(i, vr);
                if (i >= NB) wait(&vempty[b], (i / NB - 1) & 1);
                convert(off_v + b * C::KV_BYTES, vr);
                ready(&vfull[b]);
            }
            if (i + 1 < nt) fetch(a.l.v, i + 1, pid1, vr);
            pid0 = pid1;
            pid1 = pid2;
        }
    }

    // ---------------------------------------------------------------- softmax
    float m = -INFINITY, l = 0.f, unit = 0.f;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + grp * (TOK + D), to = ts + TOK;
    if (grp < groups && tid < C::ROWS) {
        constexpr uint32_t ID_S = f16_idesc(0, 0, 0, 128, TOK), ID_O = f16_idesc(0, 0, 1, 128, D);
        auto issue_s = [&](int i) {   // S = Q K^T of tile i
            const int b = i & (NB - 1);
            wait(&kfull[b], (i / NB) & 1);
            const uint32_t q0 = base + (uint32_t)(grp * QT) * C::Q_BYTES, k0s = base + off_k + b * C::KV_BYTES;
#pragma unroll
            for (int term = 0; term < QT; ++term)
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_f16(ts, sw128_desc(q0 + term * C::Q_BYTES + x * 16384u + j * 32u, 16u, 1024u),
                                 sw128_desc(k0s + x * (TOK * 128u) + j * 32u, 16u, 1024u), ID_S, term + x + j > 0);
            umma_commit(&bar_s[grp]);
            umma_commit(&kempty[b]);
            mbar_arrive(&bar_s[grp]);
        };
        auto issue_o = [&](int i) {   // O += P V
            const int b = i & (NB - 1);
            wait(&vfull[b], (i / NB) & 1);
            const uint32_t v0s = base + off_v + b * C::KV_BYTES;
#pragma unroll
            for (int term = 0; term < QT; ++term)
#pragma unroll
                for (int j = 0; j < TOK / 16; ++j)
                    umma_f16_ts(to, ts + term * (TOK / 2) + j * 8, sw128_desc(v0s + j * 2048u, TOK * 128u, 1024u), ID_O,
                                i > 0 || term + j > 0);
            umma_commit(&vempty[b]);
            if (i + 1 == nt) umma_commit(&bar_o[grp]);
        };
        if (nt > 0 && (tid & 127) == 0) issue_s(0);
        __syncwarp();
        const int pshift = __ffs(P) - 1;
        // A page's factor from product to base-2 score. Never 0, so that -infinity stays what it is.
        auto factor = [&](const RowsMeta &mt, int pg) { return fmaxf(qf * mt.ks[pg], 1e-37f); };
        for (int i = 0; i < nt; ++i) {
            wait(&bar_s[grp], i & 1);
            tc_fence_after();
            const RowsMeta &mt = meta[i & 3];
            const int j0 = tile_of(i);
            // scores to factors of the row's largest; what a row does not see becomes -infinity in place
            float top = -INFINITY;
            auto take = [&](const uint32_t *r, int t0) {   // 16 positions: one page
                float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 16; ++e) t[e & 3] = fmaxf(t[e & 3], __uint_as_float(r[e]));
                const float t4 = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                if (t4 > -INFINITY) top = fmaxf(top, t4 * factor(mt, P >= TOK ? 0 : t0 >> pshift));
            };
            if (mt.whole) {
#pragma unroll 1
                for (int ch = 0; ch < TOK; ch += 64) {
                    uint32_t r[64];
                    tmem_ld32(ts + lane_base + ch, r);
                    tmem_ld32(ts + lane_base + ch + 32, r + 32);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int g16 = 0; g16 < 64; g16 += 16) take(r + g16, ch + g16);
                }
            } else {
#pragma unroll 1
                for (int ch = 0; ch < TOK; ch += 32) {
                    uint32_t r[32];
                    tmem_ld32(ts + lane_base + ch, r);
                    const int j = j0 + ch;
                    uint32_t see = low_bits(pos - j + 1);
                    if (a.window > 0) see &= ~low_bits((long long)pos - a.window + 1 - j) | low_bits((long long)a.sinks - j);
                    const uint32_t v0 = mt.valid >> (P >= TOK ? 0 : ch >> pshift) & 1u;
                    const uint32_t v1 = mt.valid >> (P >= TOK ? 0 : (ch + 16) >> pshift) & 1u;
                    see &= (v0 ? 0xffffu : 0u) | (v1 ? 0xffff0000u : 0u);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = (see >> e) & 1u ? r[e] : 0xff800000u;
                    take(r, ch);
                    take(r + 16, ch + 16);
                    tmem_st16(ts + lane_base + ch, r);
                    tmem_st16(ts + lane_base + ch + 16, r + 16);
                }
                tmem_wait_st();
            }
            // the reference is raised when the maximum has outrun it; O follows it and the unit of the values
            float shrink = 1.f;
            if (top > m + ROWS_TRAIL || (m == -INFINITY && top > m)) {
                shrink = ex2(m - top);
                m = top;
                l *= shrink;
            }
            shrink *= mt.shrink;
            unit = mt.unit;
            if (i > 0 && __any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t r[32];
                    tmem_ld32(to + lane_base + ch * 32, r);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * shrink);
                    tmem_st16(to + lane_base + ch * 32, r);
                    tmem_st16(to + lane_base + ch * 32 + 16, r + 16);
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 1
            for (int ch = 0; ch < TOK; ch += 64) {
                uint32_t r[64], plo[QT == 2 ? 32 : 1];
                tmem_ld32(ts + lane_base + ch, r);
                tmem_ld32(ts + lane_base + ch + 32, r + 32);
                tmem_wait_ld(r);
#pragma unroll
                for (int g16 = 0; g16 < 64; g16 += 16) {
                    const int pg = P >= TOK ? 0 : (ch + g16) >> pshift;
                    const float f = factor(mt, pg), off = mt.vexp[pg] - ref;
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = g16; e < g16 + 16; e += 2) {
                        float2 x = ffma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])),
                                         make_float2(f, f), make_float2(off, off));
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        sum = fadd2(sum, x);
                        if constexpr (QT == 2) split_pair(x.x, x.y, r[e / 2], plo[e / 2]);
                        else r[e / 2] = pack_f16(x.x, x.y);
                    }
                    l = fmaf(sum.x + sum.y, mt.vback[pg], l);
                }
                // the weights take the place of scores already read, their second terms (TOK 64) that of the rest
                tmem_st16(ts + lane_base + ch / 2, r);
                tmem_st16(ts + lane_base + ch / 2 + 16, r + 16);
                if constexpr (QT == 2) {
                    tmem_st16(ts + lane_base + 32, plo);
                    tmem_st16(ts + lane_base + 48, plo + 16);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            bar_sync(2 + grp, 128);
            if ((tid & 127) == 0) {
                tc_fence_after();
                issue_o(i);
                if (i + 1 < nt) issue_s(i + 1);
            }
            __syncwarp();
        }
        if (nt > 0) wait(&bar_o[grp], 0);
        tc_fence_after();

        // ------------------------------------------------------------ output
        const float back = unit * exp2i(-(int)ROWS_UNIT);
        const int64_t unit_id = (int64_t)blockIdx.x * splits + blockIdx.y;
        const int4 f4 = make_int4(sq.row, sq.len, sq.start, sq.n);
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t r[32];
            if (nt > 0) {
                tmem_ld32(to + lane_base + ch * 32, r);
                tmem_wait_ld(r);
            }
            if (!on) continue;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                if (nt > 0)
                    o = make_float4(__uint_as_float(r[e]) * back, __uint_as_float(r[e + 1]) * back,
                                    __uint_as_float(r[e + 2]) * back, __uint_as_float(r[e + 3]) * back);
                if (splits > 1) *(float4 *)&a.rows_part[(unit_id * C::ROWS + tid) * D + ch * 32 + e] = o;
                else store_row(a, f4, h, G, D, row0 + tid, ch * 32 + e, o, m, l);
            }
        }
        if (splits > 1 && on) {
            a.rows_ml[(unit_id * C::ROWS + tid) * 2] = m;
            a.rows_ml[(unit_id * C::ROWS + tid) * 2 + 1] = l;
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
    if (!on) return;
    for (int x = 0; x < nt_all; ++x) {
        const int j0 = (x < ns ? x : w0 + x - ns) * TOK;
        if (is_whole(j0)) continue;
        for (int j = j0; j < j0 + TOK && j <= pos; ++j) {
            if (a.window > 0 && pos - j >= a.window && j >= a.sinks) continue;
            const int page = c.table[(size_t)sq.row * c.max_pages + j / P];
            if (page < 0 || page >= c.n_pages) continue;
            const uint32_t *v = (const uint32_t *)(a.l.v + (((size_t)page * c.hkv + h) * P + (j & (P - 1))) * D);
            for (int w = 0; w < D / 4; ++w)
                if (e4m3_any_nan(v[w]))
                    for (int b = 0; b < 4; ++b)
                        if (((v[w] >> (8 * b)) & 0x7fu) == 0x7fu) store_nan(a, f4, h, G, D, row0 + tid, 4 * w + b);
        }
    }
}

template <int D, int QT>
cudaError_t rows_setup()
{
    return cudaFuncSetAttribute(k_kv_rows<D, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsCfg<D, QT>::SMEM);
}

template <int D, int QT>
cudaError_t rows_launch(const KvAttendArgs &a, unsigned items, unsigned splits, cudaStream_t s)
{
    Launch L;
    L.grid = dim3(items, splits);
    L.block = dim3(RowsCfg<D, QT>::NT);
    L.smem = RowsCfg<D, QT>::SMEM;
    L.stream = s;
    L.pdl = true;
    L.nsm = 0;
    return launch_ex(L, k_kv_rows<D, QT>, a);
}

}  // namespace pi
