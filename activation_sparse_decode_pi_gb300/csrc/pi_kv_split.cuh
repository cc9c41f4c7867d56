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
//  - the products run on mma.sync m16n8k16 (f16 in, fp32 out): an e4m3 code is exact in f16, two codes
//    convert in one instruction, and the fragments are read straight from the tile's rows because the
//    contraction may run over dim in any order that q and k share. A tcgen05 product would need
//    128 rows; a decode step has 1 to 16;
//  - all (sequence, kv head, row tile) items are laid end to end and cut into equal runs of tiles, one
//    per CTA, so ragged lengths and one long sequence fill the GPU alike. An item cut over CTAs is
//    joined by the last of them to finish, in the order of its parts (the same bits every time).
// Rounding: q is scaled by a power of two per row so that its largest value lies in [128, 256) and cut
// to f16, weights are held as f16 in units of 2^-14 (floor 2^-38). TWO: both keep a second f16 term
// (22 bits, fp32 accuracy; rows 8-15 of the mma hold the second terms of rows 0-7, at no extra cost).
// Without it (bf16 output, more than 8 rows) 11 bits of the weight meet the output's 8.
#pragma once

#include "pi_kv_device.cuh"
#include "pi_umma.cuh"

namespace pi {

template <int D, bool TWO>
struct SplitCfg {
    static constexpr int NW = D == 256 ? 4 : 7;          // consumer warps (8 warps in all: 255 registers each)
    static constexpr int R = TWO ? 8 : 16;               // rows per tile
    static constexpr int SLOT = KV_TILE * D;             // bytes of one K or V tile
    static constexpr int NT = (NW + 1) * 32;
    static constexpr int MERGE = NW * R * (D + 4) * 4;   // bytes: numerators of every warp
    static constexpr int QB = D == 256 ? 16 * 512 : 0;   // bytes: query fragments (D 256 has no registers left)
    static constexpr int MAX_SLOTS = 24;
};

struct SplitMeta {   // of one ring slot
    float sc[4];     // block scales of the tile's pages
    uint32_t valid;  // bit per page: present
    uint32_t pad[3];
};

struct Seg {
    int i, h, rt, k0, k1, nt;
};

template <int D, bool TWO>
__global__ void __launch_bounds__(SplitCfg<D, TWO>::NT, 1)
    k_kv_split(const __grid_constant__ KvAttendArgs a, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, int slots)
{
    using C = SplitCfg<D, TWO>;
    constexpr int NW = C::NW, R = C::R, NJ = D / 8, NCH = D / 64;   // output n-tiles, 16-byte key chunks per lane
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float *merge = (float *)(ring + (size_t)slots * C::SLOT);
    uint4 *qfrag = (uint4 *)((uint8_t *)merge + C::MERGE);
    float *ml = (float *)((uint8_t *)qfrag + C::QB);                       // [NW][R][2]
    SplitMeta *meta = (SplitMeta *)(ml + NW * R * 2);
    uint64_t *full = (uint64_t *)(meta + slots), *empty = full + slots;
    long long *prefix = (long long *)(empty + slots);                      // [n + 1] tiles before sequence i
    int4 *info = (int4 *)((uintptr_t)(prefix + a.b.n + 2) & ~(uintptr_t)15);   // [n] row, length, start, new tokens
    __shared__ long long wtot[NW + 1];
    __shared__ int s_last, s_dead;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KvView &c = a.c;
    const int G = c.hq / c.hkv;
    if (tid == 0) {
        for (int s = 0; s < slots; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
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
            w = (((long long)q.n * G + R - 1) / R) * nt * c.hkv;
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
        for (int k = 0; k <= NW; ++k) {
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
    // A CTA's share: equal shares over the grid, but a tile at least for every consumer warp.
    const long long quota = max((total + gridDim.x - 1) / gridDim.x, (long long)NW);
    const long long t0 = quota * blockIdx.x, t1 = min(total, t0 + quota);
    if (t0 >= t1) return;

    auto segment = [&](long long t) {   // the item that tile t belongs to, and its tiles up to t1
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
        const long long local = t - prefix[lo], item = local / s.nt;
        const int rts = (int)(((long long)f.w * G + R - 1) / R);
        s.h = (int)(item / rts);
        s.rt = (int)(item % rts);
        s.k0 = (int)(local % s.nt);
        s.k1 = (int)min((long long)s.nt, s.k0 + (t1 - t));
        return s;
    };
    const int P = c.page, box_rows = min(P, KV_TILE), np = KV_TILE / box_rows;   // pages (boxes) per tile

    if (warp == NW) {
        // ------------------------------------------------------------ producer
        uint32_t n = 0;   // tiles issued
        bool dead = false;
        for (long long t = t0; t < t1 && !dead;) {
            const Seg g = segment(t);
            const int4 f = info[g.i];
            int w0, ns, nt;
            view(f.y, f.w, w0, ns, nt);
            const int per = 32 / np;   // tiles whose pages the lanes look up at once
            for (int kb = g.k0; kb < g.k1 && !dead; kb += per) {
                const int k = kb + lane / np, sub = lane % np;
                const int tile = k < ns ? k : w0 + k - ns;
                const int pos = tile * KV_TILE + sub * box_rows;
                int page = -1;
                float ks = 0.f, vs = 0.f;
                const int low = f.y - f.w - a.window + 1;   // first position in the windows
                const bool seen = pos < f.y && (pos < a.sinks || pos + box_rows > low);
                if (k < g.k1 && lane < per * np && seen) {
                    page = c.table[(size_t)f.x * c.max_pages + pos / P];
                    if (page < 0 || page >= c.n_pages) {
                        set_status(c.status, ST_DEVICE_CHECK);
                        page = -1;
                    } else {
                        ks = a.l.ks[(size_t)page * c.hkv + g.h];
                        vs = a.l.vs[(size_t)page * c.hkv + g.h];
                    }
                }
                const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
                for (int x = 0; x < per && kb + x < g.k1; ++x, ++n) {
                    const uint32_t valid = (there >> (x * np)) & ((1u << np) - 1u);
                    const uint32_t bytes = __popc(valid) * box_rows * D;
                    const bool mine = lane / np == x && lane < per * np;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t u = 2 * n + kv, slot = u % slots, round = u / slots;
                        if (round > 0 && !dead && !mbar_wait(&empty[slot], (round - 1) & 1)) dead = true;
                        if (*(volatile int *)&s_dead) dead = true;
                        dead = __any_sync(0xffffffffu, dead);
                        if (dead) break;
                        if (mine) {
                            meta[slot].sc[sub] = kv ? vs : ks;
                            if (sub == 0) meta[slot].valid = valid;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
                        __syncwarp();
                        if (mine && page >= 0) {
                            const int row = (page * c.hkv + g.h) * P + (P > KV_TILE ? (pos & (P - 1)) : 0);
                            uint8_t *dst = ring + (size_t)slot * C::SLOT + sub * box_rows * (D < 128 ? D : 128);
#pragma unroll
                            for (int x0 = 0; x0 < D; x0 += 128)
                                tma_load_2d(dst + x0 * KV_TILE, kv ? &mv : &mk, x0, row, &full[slot]);
                        }
                    }
                    if (dead) break;
                }
            }
            t += g.k1 - g.k0;
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
    auto wait_full = [&](uint32_t slot, uint32_t round) {
        if (!dead && !mbar_wait(&full[slot], round & 1)) {
            dead = true;
            *(volatile int *)&s_dead = 1;
            set_status(c.status, ST_TIMEOUT);
        }
    };

    for (long long t = t0; t < t1;) {
        const Seg sg = segment(t);
        const int4 f = info[sg.i];
        const int L = f.y, nq = f.w, p0 = L - nq;
        int w0, ns, nt_all;
        view(L, nq, w0, ns, nt_all);
        const int row0 = sg.rt * R, rows = min(R, nq * G - row0);   // rows of this tile
        const int pos_lo = p0 + row0 / G, pos_hi = p0 + (row0 + rows - 1) / G;
        int pos[TWO ? 1 : 2];
        float qf[TWO ? 1 : 2];
        uint32_t qa[D == 256 ? 1 : NCH * 4][4];
        // query fragments: this lane's row(s), elements koff-ordered like the keys
#pragma unroll
        for (int rr = 0; rr < (TWO ? 1 : 2); ++rr) {
            const int r = g + 8 * rr;
            const bool on = r < rows;
            pos[rr] = on ? p0 + (row0 + r) / G : -1;
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
            qf[rr] = a.scale_log2 * exp2i(ex - 7);
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        split_pair(x[ch][st * 4 + 2 * e] * mul, x[ch][st * 4 + 2 * e + 1] * mul, hi[e], lo[e]);
                    uint32_t *dst;
                    if constexpr (D == 256) dst = (uint32_t *)&qfrag[(ch * 4 + st) * 32 + lane];
                    else dst = qa[ch * 4 + st];
                    if constexpr (D == 256) {
                        if ((ch * 4 + st) % NW != warp) continue;   // the warps share one copy
                    }
                    if constexpr (TWO) {
                        dst[0] = hi[0];
                        dst[1] = lo[0];
                        dst[2] = hi[1];
                        dst[3] = lo[1];
                    } else {
                        dst[rr] = hi[0];
                        dst[2 + rr] = hi[1];
                    }
                }
        }
        if constexpr (D == 256) bar_sync(1, NW * 32);

        float m[TWO ? 1 : 2], l[TWO ? 1 : 2], acc[NJ][4], unit = 0.f;
#pragma unroll
        for (int rr = 0; rr < (TWO ? 1 : 2); ++rr) {
            m[rr] = -INFINITY;
            l[rr] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

        for (int k = sg.k0 + warp; k < sg.k1; k += NW) {
            const uint32_t u = 2 * (n0 + (k - sg.k0));
            const int tile = k < ns ? k : w0 + k - ns, j0 = tile * KV_TILE;
            // ---- scores
            const uint32_t ks_slot = u % slots;
            wait_full(ks_slot, u / slots);
            const uint8_t *kt = ring + (size_t)ks_slot * C::SLOT;
            const uint32_t valid = meta[ks_slot].valid;
            const bool whole = valid == (1u << np) - 1u && j0 + KV_TILE - 1 <= pos_lo &&
                               (pos_hi - j0 < a.window || j0 + KV_TILE <= a.sinks);
            float s[8][4];
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) {
#pragma unroll
                for (int h4 = 0; h4 < 2; ++h4) {
                    uint4 kw[4];
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
                        kw[nt] = *(const uint4 *)(kt + (ch >> 1) * KV_TILE * 128 + (h4 * 4 + nt) * 8 * ROWB +
                                                  koff[ch & 1]);
#pragma unroll
                    for (int st = 0; st < 4; ++st) {
                        uint32_t af[4];
                        if constexpr (D == 256) {
                            const uint4 v = qfrag[(ch * 4 + st) * 32 + lane];
                            af[0] = v.x, af[1] = v.y, af[2] = v.z, af[3] = v.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) af[e] = qa[ch * 4 + st][e];
                        }
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt) {
                            const uint32_t w = st == 0 ? kw[nt].x : st == 1 ? kw[nt].y : st == 2 ? kw[nt].z : kw[nt].w;
                            mma_f16(s[h4 * 4 + nt], af, e4m3x2_f16x2((uint16_t)w), e4m3x2_f16x2((uint16_t)(w >> 16)));
                        }
                    }
                }
            }
            float sc[4];
            if (np == 1) {
                sc[0] = meta[ks_slot].sc[0];
            } else {
                const float4 v = *(const float4 *)meta[ks_slot].sc;
                sc[0] = v.x, sc[1] = v.y, sc[2] = v.z, sc[3] = v.w;
            }
            auto pick = [&](const float (&v)[4], int nt) {   // of the page that n-tile nt lies in
                const int p = (nt * 8) >> page_shift;
                return np == 1 ? v[0] : p == 0 ? v[0] : p == 1 ? v[1] : p == 2 ? v[2] : v[3];
            };
            // ---- to base-2 logits; what a row does not see is -infinity
            float top[TWO ? 1 : 2];
#pragma unroll
            for (int rr = 0; rr < (TWO ? 1 : 2); ++rr) top[rr] = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float ks = pick(sc, nt);
#pragma unroll
                for (int rr = 0; rr < (TWO ? 1 : 2); ++rr)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = TWO ? s[nt][e] + s[nt][2 + e] : s[nt][2 * rr + e];
                        v *= qf[rr] * ks;
                        if (!whole) {
                            const int j = j0 + nt * 8 + 2 * q + e;
                            const bool see = j <= pos[rr] && ((valid >> ((nt * 8) >> page_shift)) & 1u) &&
                                             (pos[rr] - j < a.window || j < a.sinks);
                            v = see ? v : -INFINITY;
                        }
                        s[nt][2 * rr + e] = v;
                        top[rr] = fmaxf(top[rr], v);
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[ks_slot]);   // every lane has read its keys and their scales
            // ---- running maximum
            float corr[TWO ? 1 : 2];
            bool grew = false;
#pragma unroll
            for (int rr = 0; rr < (TWO ? 1 : 2); ++rr) {
                top[rr] = fmaxf(top[rr], __shfl_xor_sync(0xffffffffu, top[rr], 1));
                top[rr] = fmaxf(top[rr], __shfl_xor_sync(0xffffffffu, top[rr], 2));
                const float mn = fmaxf(m[rr], top[rr]);
                corr[rr] = mn > m[rr] ? ex2(m[rr] - mn) : 1.f;   // m = -infinity: 0
                grew |= mn > m[rr];
                m[rr] = mn;
            }
            // ---- values
            const uint32_t vs_slot = (u + 1) % slots;
            wait_full(vs_slot, (u + 1) / slots);
            uint8_t *vt = ring + (size_t)vs_slot * C::SLOT;
            if (np == 1) {
                sc[0] = meta[vs_slot].sc[0];
            } else {
                const float4 v = *(const float4 *)meta[vs_slot].sc;
                sc[0] = v.x, sc[1] = v.y, sc[2] = v.z, sc[3] = v.w;
            }
            float vmax = sc[0];
            for (int p = 1; p < np; ++p) vmax = fmaxf(vmax, p == 1 ? sc[1] : p == 2 ? sc[2] : sc[3]);
            // numerators are kept in units of the largest value scale so far
            float shrink = 1.f;
            if (vmax > unit) {
                shrink = unit / vmax;
                unit = vmax;
            }
            const float inv = unit > 0.f ? 16384.f / unit : 0.f;
            if (__any_sync(0xffffffffu, grew) || shrink != 1.f) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] *= corr[TWO ? 0 : e >> 1] * shrink;
            }
#pragma unroll
            for (int rr = 0; rr < (TWO ? 1 : 2); ++rr) l[rr] *= corr[rr];
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
                        for (int jj = 0; jj < NJ; ++jj)
                            for (int e = 0; e < 2; ++e) {
                                const int d = out_col<D>(jj, 2 * q + e);
                                if ((vt[tile_byte<D>(tok, d)] & 0x7f) != 0x7f) continue;
                                for (int rr = 0; rr < (TWO ? 1 : 2); ++rr) {
                                    const int j = j0 + tok;
                                    if (j <= pos[rr] && (pos[rr] - j < a.window || j < a.sinks))
                                        poison(acc, jj, 2 * rr + e);
                                }
                            }
                    __syncwarp();
                    for (int x = lane; x < C::SLOT; x += 32)
                        if ((vt[x] & 0x7f) == 0x7f) vt[x] = 0;
                }
                fence_proxy_async_smem();   // the slot's next copy comes after these stores
                __syncwarp();
            }
            // ---- weights and their products with the values, 16 positions at a time
#pragma unroll
            for (int st = 0; st < 4; ++st) {
                uint32_t pf[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int nt = 2 * st + h;
                    const float vs = pick(sc, nt) * inv;
#pragma unroll
                    for (int rr = 0; rr < (TWO ? 1 : 2); ++rr) {
                        const float ref = m[rr] == -INFINITY ? 0.f : m[rr];
                        const float e0 = ex2(s[nt][2 * rr] - ref), e1 = ex2(s[nt][2 * rr + 1] - ref);
                        l[rr] += e0 + e1;
                        if constexpr (TWO) split_pair(e0 * vs, e1 * vs, pf[2 * h], pf[2 * h + 1]);
                        else pf[2 * h + rr] = pack_f16(e0 * vs, e1 * vs);
                    }
                }
#pragma unroll
                for (int hf = 0; hf < (D + 127) / 128; ++hf) {
                    uint32_t vw[2][2][4];   // [token half][even / odd token][words]
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint8_t *p = vt + hf * KV_TILE * 128 + (st * 16 + h * 8) * ROWB + voff[e];
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
                        for (int b2 = 0; b2 < 2; ++b2) {   // bytes 2 b2 and 2 b2 + 1 of the word
                            const uint32_t p0w = __byte_perm(vw[0][0][w], vw[0][1][w], b2 ? 0x7362 : 0x5140);
                            const uint32_t p1w = __byte_perm(vw[1][0][w], vw[1][1][w], b2 ? 0x7362 : 0x5140);
                            const int j = hf * 16 + w * 4 + b2 * 2;
                            mma_f16(acc[j], pf, e4m3x2_f16x2((uint16_t)p0w), e4m3x2_f16x2((uint16_t)p1w));
                            mma_f16(acc[j + 1], pf, e4m3x2_f16x2((uint16_t)(p0w >> 16)),
                                    e4m3x2_f16x2((uint16_t)(p1w >> 16)));
                        }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[vs_slot]);
        }
        n0 += sg.k1 - sg.k0;

        // ---- join the warps
        const float back = unit * (1.f / 16384.f);
#pragma unroll
        for (int rr = 0; rr < (TWO ? 1 : 2); ++rr) {
            const int r = g + 8 * rr;
            l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 1);
            l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 2);
            if (q == 0) {
                ml[(warp * R + r) * 2] = m[rr];
                ml[(warp * R + r) * 2 + 1] = l[rr];
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    merge[(warp * R + r) * (D + 4) + out_col<D>(j, 2 * q + e)] =
                        (TWO ? acc[j][e] + acc[j][2 + e] : acc[j][2 * rr + e]) * back;
        }
        bar_sync(1, NW * 32);
        const bool cut = sg.k0 > 0 || sg.k1 < sg.nt;
        const long long item0 = t - sg.k0;                                 // first tile of the item
        const int ca = (int)(item0 / quota), cb = (int)((item0 + sg.nt - 1) / quota);
        const int part = (int)blockIdx.x == ca ? 2 * ca + 1 : 2 * (int)blockIdx.x;
        for (int x = tid; x < R * D / 4; x += NW * 32) {
            const int r = x / (D / 4), d = (x % (D / 4)) * 4;
            float M = -INFINITY, S = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[(w * R + r) * 2]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float mw = ml[(w * R + r) * 2], f2 = mw == -INFINITY ? (ml[(w * R + r) * 2 + 1] != 0.f ? 1.f : 0.f) : ex2(mw - M);
                const float4 v = *(const float4 *)&merge[(w * R + r) * (D + 4) + d];
                S += ml[(w * R + r) * 2 + 1] * f2;
                o.x += v.x * f2, o.y += v.y * f2, o.z += v.z * f2, o.w += v.w * f2;
            }
            if (r >= rows) continue;
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
        bar_sync(1, NW * 32);
        if (cut) {
            if (tid == 0) {
                const uint32_t before = ticket_acq_rel(&a.tickets[ca], 1u);
                s_last = before == (uint32_t)(cb - ca);
            }
            bar_sync(1, NW * 32);
            if (s_last) {
                float *wt = merge;   // [parts][R] weights, then [R][2] maximum and sum
                const int parts = cb - ca + 1;
                for (int r = warp; r < rows; r += NW) {
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
                        ml[r * 2] = M;
                        ml[r * 2 + 1] = S;
                    }
                }
                bar_sync(1, NW * 32);
                for (int x = tid; x < rows * (D / 4); x += NW * 32) {
                    const int r = x / (D / 4), d = (x % (D / 4)) * 4;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int y = 0; y < parts; ++y) {
                        const int sl = y == 0 ? 2 * ca + 1 : 2 * (ca + y);
                        const float4 v = __ldcg((const float4 *)&a.part[((size_t)sl * R + r) * D + d]);
                        const float w = wt[y * R + r];
                        o.x += v.x * w, o.y += v.y * w, o.z += v.z * w, o.w += v.w * w;
                    }
                    store_row(a, f, sg.h, G, D, row0 + r, d, o, ml[r * 2], ml[r * 2 + 1]);
                }
                if (tid == 0) a.tickets[ca] = 0;
                bar_sync(1, NW * 32);
            }
        }
        t += sg.k1 - sg.k0;
    }
}

// Ring slots (and so shared memory) for a call of n sequences: what is left beside the rest.
struct SplitPlan {
    int slots;
    size_t smem;
};
template <int D, bool TWO>
SplitPlan split_plan(int n)
{
    using C = SplitCfg<D, TWO>;
    SplitPlan p;
    const size_t fixed = 1024 + C::MERGE + C::QB + C::NW * C::R * 8 + (size_t)(n + 2) * 8 + 32 + (size_t)n * 16;
    const size_t avail = 227 * 1024 - 256 - fixed;   // 256: static shared memory
    p.slots = (int)(avail / (C::SLOT + sizeof(SplitMeta) + 16));
    if (p.slots > C::MAX_SLOTS) p.slots = C::MAX_SLOTS;
    p.smem = fixed + (size_t)p.slots * (C::SLOT + sizeof(SplitMeta) + 16);
    return p;
}

template <int D, bool TWO>
cudaError_t split_setup()
{
    return cudaFuncSetAttribute(k_kv_split<D, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 256);
}

template <int D, bool TWO>
cudaError_t split_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int grid, cudaStream_t s)
{
    const SplitPlan p = split_plan<D, TWO>(a.b.n);
    Launch L;
    L.grid = dim3(grid);
    L.block = dim3(SplitCfg<D, TWO>::NT);
    L.smem = p.smem;
    L.stream = s;
    L.pdl = true;
    L.nsm = grid;
    return launch_ex(L, k_kv_split<D, TWO>, a, mk, mv, p.slots);
}

}  // namespace pi
