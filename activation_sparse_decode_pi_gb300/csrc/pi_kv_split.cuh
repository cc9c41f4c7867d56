// pi_kv_split.cuh -- attention over the paged 8-bit cache, the cache split over the whole GPU (sm_103a).
//
// For the queries of one tile (R rows: a query token and one head of its group, all reading one kv
// head) and the keys j that they see,
//   s_j = scale * ks * (q . c_j),   out = sum_j e^{s_j} vs v_j / sum_j e^{s_j}
// with e4m3 codes c_j, v_j and block scales ks, vs. The kernel streams 64-position tiles of the cache
// once and keeps a running maximum and sum (base 2) and numerators per warp.
//
// What bounds it: at one query token per sequence the bytes of the cache (2 dim flops per byte and
// query head), so everything else has to hide under the loads:
//  - one producer warp keeps a ring of K and V tiles in flight with TMA (swizzled, so that the
//    fragment reads are free of bank conflicts); consumer warps take the tiles in turn;
//  - the products run on mma.sync m16n8k16 (f16 in, fp32 out) with the cache as the 16-row operand (16
//    positions of K, 16 columns of V) and the queries as the 8 columns, so that a decode step's few rows
//    waste little of it. An e4m3 code is exact in f16, two codes convert in one instruction, and the
//    fragments are read straight from the tile's rows because the contraction may run over dim in any
//    order that q and k share, and the output's rows may stand for its columns in any order;
//  - all (sequence, kv head, row tile) items are laid end to end and cut into equal runs of tiles, one
//    per CTA, so ragged lengths and one long sequence fill the GPU alike. An item cut over CTAs is
//    joined by the last of them to finish, in the order of its parts (the same bits every time).
// Measured (one token a sequence, 8 kv heads of 128 for 64 or 32 heads, bf16): 128 sequences of 129..16383
// positions 332 us = 6.6 TB/s, 64 windows of 4096 + 4 positions 96 us, one sequence of 131067 56 us (start and
// join ~15 us). fp32, 16 sequences of 1..8191, 40 heads: 151 us = 4.6 TB/s, bound by the consumer warps, whose
// second terms double the products. Many items of 1 to 5 tiles (85 sequences, 40 heads, fp32): 158 us at a floor of
// 22 us. (146 us before a slot's loads were fenced off from its next copy; of that the joins were some 35, left out
// to time the rest; two result slots to every warp, up to 8 items between their first product and their join, gained
// nothing there and cost 5% on 128 x 300..1000.)
// Rounding: q is scaled by a power of two per row so that its largest value lies in [128, 256) and cut
// to f16, weights are held as f16 in units of 2^-14 (floor 2^-38). T = 2: both keep a second f16 term
// (22 bits, fp32 accuracy). T = 1 (bf16 output): 11 bits of the weight meet the output's 8.
#pragma once

#include "pi_kv_device.cuh"
#include "pi_umma.cuh"

namespace pi {

// What an item costs besides its tiles, in tiles (ragged 16 x 8k, 40 heads, fp32, each tile's products added
// straight to the running sums: 139 us at 4, 136 at 8, 185 without).
constexpr int SPLIT_ITEM = 8;

// QN: runs of 8 rows per tile; T: 16-bit terms.
template <int D, int QN, int T>
struct SplitCfg {
    static constexpr bool WIDE = QN == 2 || D == 256;    // accumulators that leave no more than 8 warps on an SM
    static constexpr int NW = QN == 2 && D == 256 ? 4 : 7;   // consumer warps (and one producer)
    // Where there is room, 4 more warps join the consumers' results of an item while these go on to the next one: two
    // to each of the two buffers, so that short items do not queue for one join, and all four to a cut item (85
    // sequences of 1..300, 40 heads, fp32, before loads were fenced: 146 us, 153 with four to each; one of 131067:
    // 56 us, 62 with two).
    static constexpr bool FLOW = !WIDE;
    static constexpr int R = 8 * QN;                     // rows per tile
    static constexpr int SLOT = KV_TILE * D;             // bytes of one K or V tile
    static constexpr int JT = FLOW ? 64 : NW * 32;       // threads that join an item
    static constexpr int NT = (NW + 1) * 32 + (FLOW ? 2 * JT : 0);
    static constexpr int NM = FLOW ? 2 : 1;              // buffers of the warps' results
    static constexpr int MERGE = NW * R * (D + 4) * 4;   // bytes of one: numerators of every warp
    static constexpr int STEPS = D / 16;                 // 16-wide steps of the score's contraction
    // query fragments in shared memory where they and the accumulators are too many for the registers
    static constexpr bool QS = STEPS * 2 * T * QN + D / 16 * QN * 4 > 160;
    static constexpr int QB = QS ? STEPS * QN * T * 32 * 8 : 0;
    static constexpr bool FRESH = T == 2 && D / 16 * QN <= 8;
    // ^ a tile's products in sums of their own, where registers allow: adding to a large sum inside the
    // product loses low bits. 16 x 8k, 40 heads, fp32: error 5.6e-7 in 162 us, without 1.4e-6 in 136 us
    // (both before items were stepped through without searching: 151 us now).
    static constexpr int MAX_SLOTS = 24;
};

struct SplitMeta {   // of one ring slot
    float sc[4];     // block scales of the tile's pages
    uint32_t valid;  // bit per page: present
    uint32_t round;  // times the slot was filled before
    uint32_t pad[2];
};

struct Seg {
    int i, h, rt, k0, k1, nt;
    long long first;   // step of the item's first tile
    // the step after the last of its tiles that the CTA takes (or would)
    __device__ __forceinline__ long long after() const { return first + k1; }
};

template <int D, int QN, int T>
__global__ void __launch_bounds__(SplitCfg<D, QN, T>::NT, 1)
    k_kv_split(const __grid_constant__ KvAttendArgs a, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, int slots)
{
    using C = SplitCfg<D, QN, T>;
    constexpr int NW = C::NW, R = C::R, NJ = D / 16, NCH = D / 64;   // output row tiles, 16-byte key chunks per lane
    constexpr int QC = 2 * QN;                                       // rows (columns of the products) a lane holds
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float *merge = (float *)(ring + (size_t)slots * C::SLOT);
    uint2 *qfrag = (uint2 *)((uint8_t *)merge + C::NM * C::MERGE);   // [step][run of rows][term][lane]
    float *ml = (float *)((uint8_t *)qfrag + C::QB);   // per buffer: [NW][R][2] of the warps, [R][2] joined
    SplitMeta *meta = (SplitMeta *)(ml + C::NM * (NW + 1) * R * 2);
    uint64_t *full = (uint64_t *)(meta + slots), *empty = full + slots;
    long long *prefix = (long long *)(empty + slots);                      // [n + 1] tiles before sequence i
    int4 *info = (int4 *)((uintptr_t)(prefix + a.b.n + 2) & ~(uintptr_t)15);   // [n] row, length, start, new tokens
    __shared__ long long wtot[C::NT / 32];
    __shared__ uint64_t jfull[2], jempty[2];   // results of a segment: written, joined
    __shared__ int s_last[2], s_dead;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KvView &c = a.c;
    const int G = c.hq / c.hkv;
    if (tid == 0) {
        for (int s = 0; s < slots; ++s) {
            meta[s].round = 0xffffffffu;
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&jfull[x], NW);
            mbar_init(&jempty[x], 1);
        }
        fence_mbar_init();
        s_dead = 0;
        prefetch_tensormap(&mk);
        prefetch_tensormap(&mv);
    }
    pdl_wait();
    pdl_launch_dependents();

    // tiles of every sequence, and their running sum
    auto view = [&](int L, int nq, int &w0, int &ns, int &nt) {   // tiles [0, ns) and [w0, ...) are read
        w0 = max(0, L - nq - a.window + 1) / KV_TILE;
        const int w1 = max((L + KV_TILE - 1) / KV_TILE, w0 + 1);
        ns = min((a.sinks + KV_TILE - 1) / KV_TILE, w0);
        nt = ns + w1 - w0;
    };
    long long run = 0;
    for (int base = 0; base < a.b.n; base += C::NT) {
        const int i = base + tid;
        long long w = 0;
        if (i < a.b.n) {
            KvSeq q = kv_sequence(c, a.b, i, blockIdx.x == 0);
            if ((long long)q.n * G >= a.rows_from) q.n = 0;   // the rows kernel's
            info[i] = make_int4(q.row, q.len, q.start, q.n);
            int w0, ns, nt;
            view(q.len, q.n, w0, ns, nt);
            w = (((long long)q.n * G + R - 1) / R) * (nt + SPLIT_ITEM) * c.hkv;
        }
        long long inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) wtot[warp] = inc;
        __syncthreads();
        long long before = run, all = 0;
        for (int k = 0; k < C::NT / 32; ++k) {
            before += k < warp ? wtot[k] : 0;
            all += wtot[k];
        }
        if (i < a.b.n) prefix[i] = before + inc - w;
        run += all;
        __syncthreads();
    }
    if (tid == 0) prefix[a.b.n] = run;
    __syncthreads();
    const long long total = run;
    // A CTA's share: equal shares over the grid, but a tile at least for every consumer warp. Shares are counted in
    // steps: an item is SPLIT_ITEM steps of its own, and then a step for each tile.
    const long long quota = max((total + gridDim.x - 1) / gridDim.x, (long long)(NW + SPLIT_ITEM));
    const long long t0 = quota * blockIdx.x, t1 = min(total, t0 + quota);
    if (t0 >= t1) return;

    auto segment = [&](long long t) {   // the item that step t belongs to, and its tiles up to step t1
        int lo = 0, hi = a.b.n;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= t) lo = mid;
            else hi = mid;
        }
        Seg s;
        s.i = lo;
        const int4 f = info[lo];
        int w0, ns;
        view(f.y, f.w, w0, ns, s.nt);
        const long long local = t - prefix[lo], item = local / (s.nt + SPLIT_ITEM);
        const int rts = (int)(((long long)f.w * G + R - 1) / R);
        s.h = (int)(item / rts);
        s.rt = (int)(item % rts);
        s.first = prefix[lo] + item * (s.nt + SPLIT_ITEM) + SPLIT_ITEM;
        s.k0 = (int)max(t - s.first, 0ll);
        s.k1 = (int)min((long long)s.nt, max(t1 - s.first, 0ll));   // (none: the share ends before the first tile)
        return s;
    };
    auto following = [&](const Seg &p) {   // the next item, where p goes to the end of its own and ends before t1
        Seg s = p;
        const long long t = p.after();
        s.first = t + SPLIT_ITEM;
        if ((long long)++s.rt * R >= (long long)info[s.i].w * G) {
            s.rt = 0;
            if (++s.h == c.hkv) {
                s.h = 0;
                do ++s.i;
                while (prefix[s.i + 1] <= t);   // (sequences without rows; prefix[n] >= t1 > t)
                const int4 f = info[s.i];
                int w0, ns;
                view(f.y, f.w, w0, ns, s.nt);
            }
        }
        s.k0 = 0;
        s.k1 = (int)min((long long)s.nt, max(t1 - s.first, 0ll));
        return s;
    };
    const int P = c.page, box_rows = min(P, KV_TILE), np = KV_TILE / box_rows;   // pages (boxes) per tile

    if (warp == NW) {
        // ------------------------------------------------------------ producer
        // Runs of up to `per` tiles of a segment, whose pages the lanes look up at once (lane: tile lane / np, its page
        // lane % np). Page ids are loaded two runs before the copies are issued, scales one.
        struct Run {
            int h, k, k1, w0, ns, row, len, low, page;   // low: first position in the windows
            float ks, vs;
        };
        const int per = 32 / np;
        long long at = t0;   // next segment
        Seg g;
        Run seg{0, 0, 0, 0, 0, 0, 0, 0, -1, 0.f, 0.f};
        auto next = [&]() {   // the next run and its page ids; k >= k1 when there is none
            if (seg.k >= seg.k1 && at < t1) {
                g = at == t0 ? segment(at) : following(g);
                const int4 f = info[g.i];
                int nt;
                view(f.y, f.w, seg.w0, seg.ns, nt);
                seg.h = g.h, seg.k = g.k0, seg.k1 = g.k1, seg.row = f.x, seg.len = f.y;
                seg.low = f.y - f.w - a.window + 1;
                at = g.k0 < g.k1 ? g.after() : t1;
            }
            Run r = seg;
            r.k1 = min(seg.k1, seg.k + per);
            seg.k = r.k1;
            const int k = r.k + lane / np, pos = (k < r.ns ? k : r.w0 + k - r.ns) * KV_TILE + (lane % np) * box_rows;
            const bool seen = k < r.k1 && lane < per * np && pos < r.len && (pos < a.sinks || pos + box_rows > r.low);
            r.page = seen ? c.table[(size_t)r.row * c.max_pages + pos / P] : -2;
            return r;
        };
        auto scales = [&](Run &r) {
            if (r.page != -2 && (unsigned)r.page >= (unsigned)c.n_pages) set_status(c.status, ST_DEVICE_CHECK);
            if ((unsigned)r.page >= (unsigned)c.n_pages) r.page = -1;
            r.ks = r.page >= 0 ? a.l.ks[(size_t)r.page * c.hkv + r.h] : 0.f;
            r.vs = r.page >= 0 ? a.l.vs[(size_t)r.page * c.hkv + r.h] : 0.f;
        };
        uint32_t n = 0;   // tiles issued
        bool dead = false;
        Run r0 = next();
        scales(r0);
        Run r1 = next();
        while (r0.k < r0.k1 && !dead) {
            const Run r2 = next();
            scales(r1);
            if (!is_scale(r0.ks) || !is_scale(r0.vs)) {   // (looked at no earlier: they were loaded a run ahead)
                set_status(c.status, ST_DEVICE_CHECK);
                r0.page = -1;
                r0.ks = r0.vs = 0.f;
            }
            // Four ring slots at a time, a lane to each: keys and values of two tiles.
            const uint32_t there = __ballot_sync(0xffffffffu, r0.page >= 0);
            const int count = r0.k1 - r0.k;
            for (int x = 0; x < count; x += 2) {
                const int y = x + ((lane >> 1) & 1), kv = lane & 1;
                const bool act = lane < 4 && y < count;
                const uint32_t u = 2 * (n + y) + kv, slot = u % slots, round = u / slots;
                if (act && round > 0 && !mbar_wait(&empty[slot], (round - 1) & 1)) dead = true;
                if (*(volatile int *)&s_dead) dead = true;
                dead = __any_sync(0xffffffffu, dead);
                if (dead) {
                    n += x;
                    break;
                }
                const uint32_t valid = (there >> ((y * np) & 31)) & ((1u << np) - 1u);
                if (act) {
                    meta[slot].valid = valid;
                    *(volatile uint32_t *)&meta[slot].round = round;
                }
                int pg[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int from = (y * np + p) & 31;
                    pg[p] = __shfl_sync(0xffffffffu, r0.page, from);
                    const float k1 = __shfl_sync(0xffffffffu, r0.ks, from), v1 = __shfl_sync(0xffffffffu, r0.vs, from);
                    if (act && p < np) meta[slot].sc[p] = kv ? v1 : k1;
                }
                if (act) {
                    mbar_arrive_expect_tx(&full[slot], __popc(valid) * box_rows * D);
                    const int k = r0.k + y, tile = k < r0.ns ? k : r0.w0 + k - r0.ns;
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        if (p < np && ((valid >> p) & 1u)) {
                            const int row = (pg[p] * c.hkv + r0.h) * P + ((tile * KV_TILE + p * box_rows) & (P - 1));
                            uint8_t *dst = ring + (size_t)slot * C::SLOT + p * box_rows * (D < 128 ? D : 128);
#pragma unroll
                            for (int x0 = 0; x0 < D; x0 += 128)
                                tma_load_2d(dst + x0 * KV_TILE, kv ? &mv : &mk, x0, row, &full[slot]);
                        }
                }
                __syncwarp();
            }
            if (!dead) n += count;
            r0 = r1;
            r1 = r2;
        }
        if (dead && lane == 0) {   // nothing may land after the CTA is gone: the last copies of every slot (bounded)
            *(volatile int *)&s_dead = 1;
            set_status(c.status, ST_TIMEOUT);
            const uint32_t u = 2 * n;
            for (uint32_t s = 0; s < (uint32_t)slots && s < u; ++s) {
                const uint32_t last = (u - 1 - s) / slots;   // last round begun in slot s
                mbar_wait(&full[s], last & 1);
            }
        }
        return;
    }

    // Joins a segment (whose first tile is the CTA's n-th): the results of the warps that had tiles of it, in the
    // order of their tiles, by the `threads` threads `me`, which meet at barrier `bar`.
    auto join = [&](const Seg &sg, uint32_t n, int buf, int me, int threads, int bar) {
        auto sync = [&]() {
            __syncwarp();   // (a warp's lanes come from loops of different lengths)
            bar_sync(bar, threads);
        };
        float *const mg = merge + buf * (C::MERGE / 4), *const mm = ml + buf * ((NW + 1) * R * 2);
        float *const sums = mm + NW * R * 2;
        const int4 f = info[sg.i];
        const int row0 = sg.rt * R, rows = min(R, f.w * G - row0), count = sg.k1 - sg.k0, turn = n % NW;
        const bool cut = sg.k0 > 0 || sg.k1 < sg.nt;
        int ca = 0, cb = 0;   // the item's CTAs
        if (cut) ca = (int)(sg.first / quota), cb = (int)((sg.first + sg.nt - 1) / quota);
        const int part = (int)blockIdx.x == ca ? 2 * ca + 1 : 2 * (int)blockIdx.x;
        // per row: the warps' weights against the common maximum (in place of their own), the maximum and the sum
        const int np_w = min(count, NW);
        if (me < rows) {
            float M = -INFINITY, S = 0.f;
            for (int y = 0, w = turn; y < np_w; ++y, w = w + 1 == NW ? 0 : w + 1) M = fmaxf(M, mm[(w * R + me) * 2]);
            for (int y = 0, w = turn; y < np_w; ++y, w = w + 1 == NW ? 0 : w + 1) {
                const float mw = mm[(w * R + me) * 2], lw = mm[(w * R + me) * 2 + 1];
                const float f2 = mw == -INFINITY ? (lw != 0.f ? 1.f : 0.f) : ex2(mw - M);
                S += lw * f2;
                mm[(w * R + me) * 2] = f2;
            }
            sums[me * 2] = M;
            sums[me * 2 + 1] = S;
        }
        sync();
        for (int x = me; x < rows * (D / 4); x += threads) {
            const int r = x / (D / 4), d = (x % (D / 4)) * 4;
            const float M = sums[r * 2], S = sums[r * 2 + 1];
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            int w = turn;
#pragma unroll
            for (int y = 0; y < NW; ++y) {
                if (y < np_w) {
                    const float f2 = mm[(w * R + r) * 2];
                    const float4 v = *(const float4 *)&mg[(w * R + r) * (D + 4) + d];
                    o.x += v.x * f2, o.y += v.y * f2, o.z += v.z * f2, o.w += v.w * f2;
                }
                w = w + 1 == NW ? 0 : w + 1;
            }
            if (cut) {
                *(float4 *)&a.part[((size_t)part * R + r) * D + d] = o;
                if (d == 0) {
                    a.part_ml[((size_t)part * R + r) * 2] = M;
                    a.part_ml[((size_t)part * R + r) * 2 + 1] = S;
                }
            } else {
                store_row(a, f, sg.h, G, D, row0 + r, d, o, M, S);
            }
        }
        if (!cut) return;
        sync();
        if (me == 0) s_last[buf] = ticket_acq_rel(&a.tickets[ca], 1u) == (uint32_t)(cb - ca);
        sync();
        if (!s_last[buf]) return;
        float *wt = mg;   // [parts][R] weights
        const int parts = cb - ca + 1;
        for (int r = me / 32; r < rows; r += threads / 32) {
            float M = -INFINITY;
            for (int x = lane; x < parts; x += 32) {
                const int sl = x == 0 ? 2 * ca + 1 : 2 * (ca + x);
                M = fmaxf(M, __ldcg(&a.part_ml[((size_t)sl * R + r) * 2]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            float S = 0.f;
            for (int x = lane; x < parts; x += 32) {
                const int sl = x == 0 ? 2 * ca + 1 : 2 * (ca + x);
                const float mx = __ldcg(&a.part_ml[((size_t)sl * R + r) * 2]);
                const float sx = __ldcg(&a.part_ml[((size_t)sl * R + r) * 2 + 1]);
                const float w = mx == -INFINITY ? (sx != 0.f ? 1.f : 0.f) : ex2(mx - M);
                wt[x * R + r] = w;
                S += w * sx;
            }
            S = warp_sum(S);
            if (lane == 0) {
                sums[r * 2] = M;
                sums[r * 2 + 1] = S;
            }
        }
        sync();
        for (int x = me; x < rows * (D / 4); x += threads) {
            const int r = x / (D / 4), d = (x % (D / 4)) * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int y = 0; y < parts; ++y) {
                const int sl = y == 0 ? 2 * ca + 1 : 2 * (ca + y);
                const float4 v = __ldcg((const float4 *)&a.part[((size_t)sl * R + r) * D + d]);
                const float w = wt[y * R + r];
                o.x += v.x * w, o.y += v.y * w, o.z += v.z * w, o.w += v.w * w;
            }
            store_row(a, f, sg.h, G, D, row0 + r, d, o, sums[r * 2], sums[r * 2 + 1]);
        }
        if (me == 0) a.tickets[ca] = 0;
        sync();
    };

    if (C::FLOW && warp > NW) {
        // ------------------------------------------------------------ joiners
        const int own = (warp - NW - 1) / 2;   // buffer of this pair of warps
        uint32_t n = 0;
        int number = 0;
        bool dead = false;
        Seg sg;
        for (long long t = t0; t < t1; ++number) {
            sg = t == t0 ? segment(t) : following(sg);
            if (sg.k0 >= sg.k1) break;
            // A cut item is the first or the last of the share, and on the way to the call's end: every joiner's. (The
            // pair of the other buffer has seen the segment before, so it cannot take an older phase for this one's.)
            const bool all = sg.k0 > 0 || sg.k1 < sg.nt;
            const int b = number & 1;
            if (all || b == own) {
                if (!dead && !warp_wait(&jfull[b], (number >> 1) & 1)) {
                    dead = true;
                    set_status(c.status, ST_TIMEOUT);
                }
                const int me = tid - (NW + 1) * 32 - (all ? 0 : own * C::JT);
                const int threads = all ? 2 * C::JT : C::JT, bar = all ? 4 : 2 + own;
                join(sg, n, b, me, threads, bar);
                bar_sync(bar, threads);
                if (me == 0) mbar_arrive(&jempty[b]);
            }
            n += sg.k1 - sg.k0;
            t = sg.after();
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int g = lane >> 2, q = lane & 3;
    // byte offsets of this lane's key chunk 0/1 and value chunks of even/odd tokens inside a tile
    int koff[2], voff[2];
    if (D == 64) {
        koff[0] = koff[1] = g * 64 + ((q ^ ((g >> 1) & 3)) << 4);
        for (int e = 0; e < 2; ++e) voff[e] = (2 * q + e) * 64 + (((g >> 1) ^ q) << 4) + (g & 1) * 8;
    } else {
        for (int e = 0; e < 2; ++e) {
            koff[e] = g * 128 + (((2 * q + e) ^ g) << 4);
            voff[e] = (2 * q + e) * 128 + ((g ^ (2 * q + e)) << 4);
        }
    }
    constexpr int ROWB = D < 128 ? D : 128;   // bytes of a tile row (per 128-column half)
    const int page_shift = __ffs(box_rows) - 1;
    uint32_t n0 = 0;
    bool dead = false;
    float inv = 0.f;   // 1 / unit of the item
    // A warp may come to a slot while an earlier filling is on its way (most do where the ring has fewer slots than
    // the warps' tiles), and parity tells a phase from its neighbours only. So the producer's count is read first: it
    // reaches `round` after phase round - 1 has completed, and phase round + 1 cannot complete before this warp has
    // released the slot, so a parity read after it is that of `round` or of the phase under way.
    auto filled = [&](uint32_t slot, uint32_t round) {
        return *(volatile uint32_t *)&meta[slot].round == round && mbar_try_wait(&full[slot], round & 1);
    };
    auto wait_full = [&](uint32_t slot, uint32_t round) {
        if (dead) return;
        bool ok = filled(slot, round);
        if (!ok) {
            const unsigned long long since = globaltimer_ns();
            while (!(ok = filled(slot, round)))
                if (globaltimer_ns() - since > WAIT_LIMIT_NS) break;
        }
        if (!__all_sync(0xffffffffu, ok)) {   // (the warp leaves as one, as from warp_wait)
            dead = true;
            *(volatile int *)&s_dead = 1;
            set_status(c.status, ST_TIMEOUT);
        }
    };

    int number = -1;   // of the segment
    Seg sg;
    for (long long t = t0; t < t1;) {
        sg = t == t0 ? segment(t) : following(sg);
        const int count = sg.k1 - sg.k0;
        if (count <= 0) break;
        // this warp's first tile of the segment: the warps take the CTA's tiles in turn
        const int kw0 = sg.k0 + (int)((warp + NW - n0 % NW) % NW);
        ++number;
        const int buf = C::FLOW ? number & 1 : 0;
        auto buffer_free = [&]() {   // the results of the segment before the last have left it
            if (C::FLOW && number > 1 && !dead && !warp_wait(&jempty[buf], ((number >> 1) - 1) & 1)) {
                dead = true;
                *(volatile int *)&s_dead = 1;
                set_status(c.status, ST_TIMEOUT);
            }
        };
        if (C::FLOW && kw0 >= sg.k1) {   // no tile of it is this warp's
            buffer_free();   // (every lane has seen that phase: one left behind could take a later one for it)
            if (lane == 0) mbar_arrive(&jfull[buf]);
            n0 += count;
            t = sg.after();
            continue;
        }
        const int4 f = info[sg.i];
        const int L = f.y, nq = f.w, p0 = L - nq;
        int w0, ns, nt_all;
        view(L, nq, w0, ns, nt_all);
        const int row0 = sg.rt * R, rows = min(R, nq * G - row0);   // rows of this tile
        const int pos_lo = p0 + row0 / G, pos_hi = p0 + (row0 + rows - 1) / G;
        // query fragments: this lane's row(s) of each run, elements in the order of the keys' bytes
        uint32_t qa[C::QS ? 1 : C::STEPS][QN][T][2];
        float qs[QN];   // factor from product to base-2 score of row g of each run
#pragma unroll
        for (int rr = 0; rr < QN; ++rr) {
            const int r = g + 8 * rr;
            const bool on = r < rows;
            const int64_t at = on ? ((int64_t)f.z + (row0 + r) / G) * a.ldq +
                                        (int64_t)(sg.h * G + (row0 + r) % G) * D
                                  : 0;
            float x[NCH][16];
            float top = 0.f;
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) {
                const int d0 = D == 64 ? q * 16 : (ch >> 1) * 128 + (2 * q + (ch & 1)) * 16;
                if (on) load16(a.q, a.dtype, at + d0, x[ch]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (!on) x[ch][e] = 0.f;
                    top = fmaxf(top, finite_abs(x[ch][e]));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = top > 0.f ? min(max(ilogbf(top), -118), 127) : 0;   // 2^ex <= top < 2^(ex + 1)
            const float mul = exp2i(7 - ex);
            qs[rr] = a.scale_log2 * exp2i(ex - 7);
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        split_pair(x[ch][st * 4 + 2 * e] * mul, x[ch][st * 4 + 2 * e + 1] * mul, hi[e], lo[e]);
                    const int k = ch * 4 + st;
                    if constexpr (C::QS) {
                        if (k % NW != warp) continue;   // the warps share one copy
                        qfrag[((k * QN + rr) * T) * 32 + lane] = make_uint2(hi[0], hi[1]);
                        if constexpr (T == 2) qfrag[((k * QN + rr) * T + 1) * 32 + lane] = make_uint2(lo[0], lo[1]);
                    } else {
                        qa[k][rr][0][0] = hi[0], qa[k][rr][0][1] = hi[1];
                        if constexpr (T == 2) qa[k][rr][T - 1][0] = lo[0], qa[k][rr][T - 1][1] = lo[1];
                    }
                }
        }
        if constexpr (C::QS) bar_sync(1, NW * 32);
        // of this lane's rows 8 rr + 2 q + e: position, and factor from product to base-2 score
        int pos[QC];
        float qf[QC], m[QC], l[QC], acc[QN][NJ][4], unit = 0.f;
        inv = 0.f;
#pragma unroll
        for (int x = 0; x < QC; ++x) {
            const int r = 8 * (x >> 1) + 2 * q + (x & 1);
            pos[x] = r < rows ? p0 + (row0 + r) / G : -1;
            qf[x] = __shfl_sync(0xffffffffu, qs[x >> 1], (2 * q + (x & 1)) * 4);
            m[x] = -INFINITY;
            l[x] = 0.f;
        }
#pragma unroll
        for (int rr = 0; rr < QN; ++rr)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[rr][j][e] = 0.f;

        for (int k = kw0; k < sg.k1; k += NW) {
            const uint32_t u = 2 * (n0 + (k - sg.k0));
            const int tile = k < ns ? k : w0 + k - ns, j0 = tile * KV_TILE;
            // ---- scores: s[rr][t][2 h + e] of position 16 t + 8 h + g and row 8 rr + 2 q + e
            const uint32_t ks_slot = u % slots;
            wait_full(ks_slot, u / slots);
            const uint8_t *kt = ring + (size_t)ks_slot * C::SLOT;
            const uint32_t valid = meta[ks_slot].valid;
            const bool whole = valid == (1u << np) - 1u && j0 + KV_TILE - 1 <= pos_lo &&
                               (pos_hi - j0 < a.window || j0 + KV_TILE <= a.sinks);
            // (T 2: second terms in sums of their own. The tensor cores cut sums off, each time by up to a unit of the
            // sum's last place, so every product added to a large sum costs.)
            float s[QN][4][4], s2[T == 2 ? QN : 1][4][4];
#pragma unroll
            for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[rr][t][e] = 0.f;
                        if constexpr (T == 2) s2[rr][t][e] = 0.f;
                    }
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) {
#pragma unroll
                for (int t2 = 0; t2 < 4; t2 += 2) {   // two runs of 16 positions at a time
                    uint4 kw[2][2];
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            kw[t][h] = *(const uint4 *)(kt + (ch >> 1) * KV_TILE * 128 +
                                                        ((t2 + t) * 16 + h * 8) * ROWB + koff[ch & 1]);
#pragma unroll
                    for (int st = 0; st < 4; ++st) {
                        uint32_t qb[QN][T][2];
#pragma unroll
                        for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                            for (int x = 0; x < T; ++x) {
                                if constexpr (C::QS) {
                                    const uint2 v = qfrag[(((ch * 4 + st) * QN + rr) * T + x) * 32 + lane];
                                    qb[rr][x][0] = v.x, qb[rr][x][1] = v.y;
                                } else {
                                    qb[rr][x][0] = qa[ch * 4 + st][rr][x][0], qb[rr][x][1] = qa[ch * 4 + st][rr][x][1];
                                }
                            }
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            uint32_t ka[4];   // rows g and g + 8, columns 0-1 and 2-3 of this lane's four
                            e4m3x4_f16x4(word4(kw[t][0], st), ka[0], ka[2]);
                            e4m3x4_f16x4(word4(kw[t][1], st), ka[1], ka[3]);
#pragma unroll
                            for (int rr = 0; rr < QN; ++rr) {
                                mma_f16(s[rr][t2 + t], ka, qb[rr][0][0], qb[rr][0][1]);
                                if constexpr (T == 2) mma_f16(s2[rr][t2 + t], ka, qb[rr][T - 1][0], qb[rr][T - 1][1]);
                            }
                        }
                    }
                }
            }
            float sc[4];   // of the four runs of 16 positions
            auto run_scales = [&](uint32_t slot) {
                if (np == 1) {
                    sc[0] = sc[1] = sc[2] = sc[3] = meta[slot].sc[0];
                } else {
                    const float4 v = *(const float4 *)meta[slot].sc;
                    sc[0] = v.x, sc[1] = np == 2 ? v.x : v.y, sc[2] = np == 2 ? v.y : v.z, sc[3] = np == 2 ? v.y : v.w;
                }
            };
            run_scales(ks_slot);
            // Every lane has read its keys and their scales, and the slot's next copy (by TMA, past the order of ordinary
            // loads) comes after that.
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[ks_slot]);
            // ---- to base-2 logits; what a row does not see is -infinity
            float top[QC];
#pragma unroll
            for (int x = 0; x < QC; ++x) top[x] = -INFINITY;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = s[rr][t][e];
                        if constexpr (T == 2) v += s2[rr][t][e];
                        s[rr][t][e] = v * (qf[2 * rr + (e & 1)] * sc[t]);
                    }
            if (!whole) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = j0 + t * 16 + (e >> 1) * 8 + g, p = pos[2 * rr + (e & 1)];
                            const bool see = j <= p && ((valid >> ((t * 16) >> page_shift)) & 1u) &&
                                             (p - j < a.window || j < a.sinks);
                            if (!see) s[rr][t][e] = -INFINITY;
                        }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top[2 * rr + (e & 1)] = fmaxf(top[2 * rr + (e & 1)], s[rr][t][e]);
            // ---- running maximum
            float corr[QC];
            bool grew = false;
#pragma unroll
            for (int x = 0; x < QC; ++x) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], o));
                const float mn = fmaxf(m[x], top[x]);
                corr[x] = mn > m[x] ? ex2(m[x] - mn) : 1.f;   // m = -infinity: 0
                grew |= mn > m[x];
                m[x] = mn;
            }
            // ---- values
            const uint32_t vs_slot = (u + 1) % slots;
            wait_full(vs_slot, (u + 1) / slots);
            uint8_t *vt = ring + (size_t)vs_slot * C::SLOT;
            run_scales(vs_slot);
            const float vmax = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
            // numerators are kept in units of the largest value scale so far
            float shrink = 1.f;
            if (vmax > unit) {
                // (an append gives zeros the scale 2^-120: the unit's reciprocal has to be finite, and 2^14 stays out of it)
                const float up = fmaxf(vmax, 0x1p-126f);
                shrink = unit / up;
                unit = up;
                inv = 1.f / unit;
            }
            if (__any_sync(0xffffffffu, grew) || shrink != 1.f) {
#pragma unroll
                for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[rr][j][e] *= corr[2 * rr + (e & 1)] * shrink;
            }
            // FRESH: a tile's products in sums of their own, which are then added with rounding (see above)
            float sum[C::FRESH ? QN : 1][NJ][4];
            if constexpr (C::FRESH) {
#pragma unroll
                for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[rr][j][e] = 0.f;
            }
#pragma unroll
            for (int x = 0; x < QC; ++x) l[x] *= corr[x];
            if (!whole) {
                // values of positions that no row of the tile sees (stale, absent, past the end) must not
                // meet a zero weight: 0 * NaN. Others that are NaN poison only the rows that see them.
                auto dead_token = [&](int j) {
                    if (!((valid >> ((j - j0) >> page_shift)) & 1u) || j > pos_hi) return true;
                    return j >= a.sinks && pos_lo - j >= a.window;
                };
                bool nan = false;
                for (int x = lane; x < C::SLOT / 16; x += 32) {
                    uint4 *p = (uint4 *)vt + x;
                    const int tok = (x * 16 / ROWB) & (KV_TILE - 1);
                    if (dead_token(j0 + tok)) *p = make_uint4(0, 0, 0, 0);
                    else nan |= e4m3_any_nan(p->x) | e4m3_any_nan(p->y) | e4m3_any_nan(p->z) | e4m3_any_nan(p->w);
                }
                __syncwarp();
                if (__any_sync(0xffffffffu, nan)) {
                    for (int tok = 0; tok < KV_TILE; ++tok)
                        for (int j = 0; j < NJ; ++j)
                            for (int h = 0; h < 2; ++h) {
                                if ((vt[tile_byte<D>(tok, out_col<D>(j, g, h))] & 0x7f) != 0x7f) continue;
                                const int at = j0 + tok;
#pragma unroll
                                for (int x = 0; x < QC; ++x)
                                    if (at <= pos[x] && (pos[x] - at < a.window || at < a.sinks))
                                        poison(acc[x >> 1], j, 2 * h + (x & 1));
                            }
                    __syncwarp();
                    for (int x = lane; x < C::SLOT; x += 32)
                        if ((vt[x] & 0x7f) == 0x7f) vt[x] = 0;
                }
                __syncwarp();
            }
            // ---- weights, and their products with the values, 16 positions at a time
            float ref[QC];
#pragma unroll
            for (int x = 0; x < QC; ++x) ref[x] = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t pb[QN][T][2];   // positions 2 q, 2 q + 1 (and 8 on) of row g: the scores' fragment transposed
                const float vs = sc[t] * inv * 16384.f;
#pragma unroll
                for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float e0 = ex2(s[rr][t][2 * h] - ref[2 * rr]);
                        const float e1 = ex2(s[rr][t][2 * h + 1] - ref[2 * rr + 1]);
                        l[2 * rr] += e0;
                        l[2 * rr + 1] += e1;
                        if constexpr (T == 2) {
                            uint32_t hi, lo;
                            split_pair(e0 * vs, e1 * vs, hi, lo);
                            pb[rr][0][h] = transpose8(hi);
                            pb[rr][T - 1][h] = transpose8(lo);
                        } else {
                            pb[rr][0][h] = transpose8(pack_f16(e0 * vs, e1 * vs));
                        }
                    }
#pragma unroll
                for (int hf = 0; hf < (D + 127) / 128; ++hf) {
                    uint32_t vw[2][2][4];   // [position half][even / odd position][words]
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint8_t *p = vt + hf * KV_TILE * 128 + (t * 16 + h * 8) * ROWB + voff[e];
                            if constexpr (D == 64) {
                                const uint2 v = *(const uint2 *)p;
                                vw[h][e][0] = v.x, vw[h][e][1] = v.y;
                            } else {
                                const uint4 v = *(const uint4 *)p;
                                vw[h][e][0] = v.x, vw[h][e][1] = v.y, vw[h][e][2] = v.z, vw[h][e][3] = v.w;
                            }
                        }
#pragma unroll
                    for (int w = 0; w < (D == 64 ? 2 : 4); ++w)
#pragma unroll
                        for (int b2 = 0; b2 < 2; ++b2) {   // columns 2 b2 and 2 b2 + 1 of the word
                            uint32_t va[4];
                            e4m3x4_f16x4(__byte_perm(vw[0][0][w], vw[0][1][w], b2 ? 0x7362 : 0x5140), va[0], va[1]);
                            e4m3x4_f16x4(__byte_perm(vw[1][0][w], vw[1][1][w], b2 ? 0x7362 : 0x5140), va[2], va[3]);
                            const int j = hf * 8 + w * 2 + b2;
#pragma unroll
                            for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                                for (int x = 0; x < T; ++x) {
                                    if constexpr (C::FRESH) mma_f16(sum[rr][j], va, pb[rr][x][0], pb[rr][x][1]);
                                    else mma_f16(acc[rr][j], va, pb[rr][x][0], pb[rr][x][1]);
                                }
                        }
                }
            }
            if constexpr (C::FRESH) {
#pragma unroll
                for (int rr = 0; rr < QN; ++rr)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[rr][j][e] += sum[rr][j][e];
            }
            fence_proxy_async_smem();   // the slot's next copy comes after the loads (and what was cleared)
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[vs_slot]);
        }
        // ---- the warp's results, for the join
        buffer_free();
        float *const mg = merge + buf * (C::MERGE / 4), *const mm = ml + buf * ((NW + 1) * R * 2);
#pragma unroll
        for (int x = 0; x < QC; ++x) {
            const int r = 8 * (x >> 1) + 2 * q + (x & 1);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], o);
            if (r >= rows) continue;
            if (g == 0) {
                mm[(warp * R + r) * 2] = m[x];
                mm[(warp * R + r) * 2 + 1] = l[x];
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                *(float2 *)&mg[(warp * R + r) * (D + 4) + out_col<D>(j, g, 0)] =
                    make_float2(acc[x >> 1][j][x & 1] * 0x1p-14f * unit, acc[x >> 1][j][2 + (x & 1)] * 0x1p-14f * unit);
        }
        if constexpr (C::FLOW) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&jfull[buf]);
        } else {
            bar_sync(1, NW * 32);
            join(sg, n0, 0, tid, C::JT, 2);
            bar_sync(1, NW * 32);
        }
        n0 += count;
        t = sg.after();
    }
}

// Ring slots (and so shared memory) for a call of n sequences: what is left beside the rest.
struct SplitPlan {
    int slots;
    size_t smem;
};
template <int D, int QN, int T>
SplitPlan split_plan(int n)
{
    using C = SplitCfg<D, QN, T>;
    SplitPlan p;
    const size_t fixed = 1024 + C::NM * (C::MERGE + (C::NW + 1) * C::R * 8) + C::QB + (size_t)(n + 2) * 8 + 32 +
                         (size_t)n * 16;
    const size_t avail = 227 * 1024 - 256 - fixed;   // 256: static shared memory
    p.slots = (int)(avail / (C::SLOT + sizeof(SplitMeta) + 16));
    if (p.slots > C::MAX_SLOTS) p.slots = C::MAX_SLOTS;
    p.smem = fixed + (size_t)p.slots * (C::SLOT + sizeof(SplitMeta) + 16);
    return p;
}

template <int D, int QN, int T>
cudaError_t split_setup()
{
    return cudaFuncSetAttribute(k_kv_split<D, QN, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 256);
}

template <int D, int QN, int T>
cudaError_t split_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int grid, cudaStream_t s)
{
    const SplitPlan p = split_plan<D, QN, T>(a.b.n);
    Launch L;
    L.grid = dim3(grid);
    L.block = dim3(SplitCfg<D, QN, T>::NT);
    L.smem = p.smem;
    L.stream = s;
    L.pdl = true;
    L.nsm = grid;
    return launch_ex(L, k_kv_split<D, QN, T>, a, mk, mv, p.slots);
}

}  // namespace pi
