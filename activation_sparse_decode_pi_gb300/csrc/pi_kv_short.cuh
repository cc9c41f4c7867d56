// pi_kv_short.cuh -- attention of few rows over what lies behind a shared prefix (sm_103a).
//
// The second pass of pi_kv_attend_shared: for each sequence and kv head a tile of up to 8 rows (query token and head of the
// group) and the positions behind the prefix, often some hundred, then the join with what the first pass left of the rows.
// And the first pass where a prefix has few rows, which all see all of it.
// There are many such items and little in each, so what counts is how many are under way and what one costs from end to
// end: a CTA has four warps that share nothing until an item's end, four CTAs to an SM. A warp takes 16 of a tile's 64
// positions: it asks for their codes by TMA, three tiles ahead, into boxes of its own, and keeps its own maximum, sum and
// numerators; the products are pi_kv_split.cuh's (the cache as the 16-row operand on mma.sync m16n8k16, codes to f16 two
// at a time, queries in T terms), and so are their units and rounding; weights have two terms in every type. The items are laid end to end and cut into equal
// shares. An item of up to two shares belongs to the CTA with its first step; a longer one is cut over CTAs and joined by
// the last of them, in the order of its parts.
// Measured: 64 sequences of 1..716 positions behind a prefix, 64 heads on 8 of 128, bf16, with the join of the prefix's 9
// parts 29 us; 72 of 4..331, 40 heads, fp16 68 us = 2.3 TB/s. An item takes about 15 us from end to end (search 1.5,
// queries and page lookups 2, first codes and the prefix's parts 3..5, 0.8 a tile, join 2), bound by latency and, with many
// items, by issue slots; one or two warps to an item took as long or longer (the latter's whole call, with an earlier first
// pass: 251 and 247 us, 242 with four).
#pragma once

#include "pi_kv_device.cuh"
#include "pi_umma.cuh"

namespace pi {

constexpr int SHORT_ITEM = 8;    // what an item costs besides its tiles, in tiles (4: 89 us instead of 84 on 64 x 1..700 positions)
constexpr int SHORT_SHARE = 2;   // steps of a share at least

template <int D, int T>
struct ShortCfg {
    static constexpr int NW = 4, NT = NW * 32, R = 8, CTAS = SHORT_CTAS;
    static constexpr int SLOTS = 3, BOX = 16 * D;   // places of a warp for 16 positions' keys and values; bytes of either
    static constexpr int RING = NW * SLOTS * 2 * BOX;
    static_assert(RING >= NW * R * (D + 4) * 4, "the warps' results take the boxes' place");
    static constexpr int SMEM = RING + (NW + 1) * R * 8 + NW * SLOTS * 8;   // and 28 bytes a sequence
};

template <int D, int T>
__global__ void __launch_bounds__(ShortCfg<D, T>::NT, ShortCfg<D, T>::CTAS)
    k_kv_short(const __grid_constant__ KvAttendArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    using C = ShortCfg<D, T>;
    constexpr int NW = C::NW, NT = C::NT, R = C::R, NJ = D / 16, NCH = D / 64;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *const smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float *const merge = (float *)smem, *const ml = (float *)(smem + C::RING), *const sums = ml + NW * R * 2;
    int4 *const info = (int4 *)(smem + C::SMEM);                                  // [n] row, length, start, new tokens
    long long *const prefix = (long long *)(info + a.b.n);                        // [n + 1] steps before sequence i
    int *const skips = (int *)(prefix + a.b.n + 1);                               // [n]
    __shared__ long long wtot[NW];
    __shared__ int s_last;
    __shared__ float s_pw[R][16], s_pm[R], s_ps[R];   // weights of what the first pass left of a row; its maximum and sum
    static_assert(NT == R * 16, "a thread to a row's part");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const KvView &c = a.c;
    const int G = c.hq / c.hkv, P = c.page;
    const bool flat = a.pass == 1;   // every row sees the whole length
    uint8_t *const ring = smem + warp * C::SLOTS * 2 * C::BOX;
    uint64_t *const full = (uint64_t *)(sums + R * 2) + warp * C::SLOTS;
    if (lane == 0) {
        for (int x = 0; x < C::SLOTS; ++x) mbar_init(&full[x], 1);
        fence_mbar_init();
    }
    __syncwarp();
    if (tid == 0) {
        prefetch_tensormap(&mk);
        prefetch_tensormap(&mv);
    }
    pdl_wait();
    pdl_launch_dependents();
    uint32_t asked = 0, taken = 0;   // boxes of the warp
    bool dead = false;
    long long run = 0;
    for (int base = 0; base < a.b.n; base += NT) {
        const int i = base + tid;
        long long w = 0;
        if (i < a.b.n) {
            KvSeq s = kv_sequence<true>(c, a.b, i, blockIdx.x == 0);
            if ((long long)s.n * G >= a.rows_from) s.n = 0;   // the rows kernel's
            info[i] = make_int4(s.row, s.len, s.start, s.n);
            skips[i] = s.skip;
            w = (((long long)s.n * G + R - 1) / R) * (max(0, (s.len - s.skip + KV_TILE - 1) / KV_TILE) + SHORT_ITEM) * c.hkv;
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
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            before += k < warp ? wtot[k] : 0;
            all += wtot[k];
        }
        if (i < a.b.n) prefix[i] = before + inc - w;
        run += all;
        __syncthreads();
    }
    if (tid == 0) prefix[a.b.n] = run;
    __syncthreads();
    const long long quota = max((run + gridDim.x - 1) / gridDim.x, (long long)SHORT_SHARE);
    const bool small = run < (1ll << 31);   // steps are 32-bit numbers: the divisions cost less
    const long long t0 = quota * blockIdx.x, t1 = min(run, t0 + quota);

    for (long long t = t0; t < t1;) {
        // the item that step t belongs to, and its tiles up to step t1
        int i = 0;
        for (int hi = a.b.n; hi - i > 1;) {
            const int mid = (i + hi) >> 1;
            if (prefix[mid] <= t) i = mid;
            else hi = mid;
        }
        const int4 f = info[i];
        const int L = f.y, nq = f.w, tile0 = skips[i] / KV_TILE, nt = max(0, (L + KV_TILE - 1) / KV_TILE - tile0);
        const long long local = t - prefix[i], item = small ? (long long)((uint32_t)local / (uint32_t)(nt + SHORT_ITEM)) : local / (nt + SHORT_ITEM);
        const int rts = (int)(((long long)nq * G + R - 1) / R), h = small ? (int)((uint32_t)item / (uint32_t)rts) : (int)(item / rts);
        const int row0 = (int)(item - (long long)h * rts) * R;
        const long long first = prefix[i] + item * (nt + SHORT_ITEM) + SHORT_ITEM;   // step of the item's first tile
        const bool whole_item = nt == 0 || nt + SHORT_ITEM <= 2 * quota;   // (without positions there is nothing to cut)
        int k0 = 0, k1 = nt;
        if (whole_item) {
            t = first + nt;
            if (first - SHORT_ITEM < t0) continue;   // the CTA's before
        } else {
            k0 = (int)max(t - first, 0ll);
            k1 = (int)min((long long)nt, max(t1 - first, 0ll));
            t = first + nt < t1 ? first + nt : t1;
            if (k0 >= k1) continue;   // (the share ends before the item's first tile)
        }
        const int p0 = L - nq, rows = min(R, nq * G - row0);
        const int pos_lo = flat ? L - 1 : p0 + row0 / G, pos_hi = flat ? L - 1 : p0 + (row0 + rows - 1) / G;

        // ---------------------------------------------------------------- pages of up to 32 tiles, one to a lane
        int pid = -2;
        float ks = 0.f, vs = 0.f;
        auto look_up = [&](int k) {   // of tiles k ... k + 31: this warp's 16 positions
            const int pos = (tile0 + k + lane) * KV_TILE + warp * 16;
            pid = k + lane < k1 && pos <= pos_hi ? c.table[(size_t)f.x * c.max_pages + pos / P] : -2;
        };
        auto look_up_scales = [&]() {
            bool bad = pid != -2 && (unsigned)pid >= (unsigned)c.n_pages;
            if (bad) pid = -1;
            ks = pid >= 0 ? a.l.ks[(size_t)pid * c.hkv + h] : 0.f;
            vs = pid >= 0 ? a.l.vs[(size_t)pid * c.hkv + h] : 0.f;
            if (!is_scale(ks) || !is_scale(vs)) {
                bad = true;
                pid = -1;
                ks = vs = 0.f;
            }
            if (bad) set_status(c.status, ST_DEVICE_CHECK);
        };
        look_up(k0);

        // ---------------------------------------------------------------- queries, in the order of the keys' bytes
        uint32_t qa[D / 16][T][2];
        float qs;   // factor from product to base-2 score of row g
        {
            const bool on = g < rows;
            const int64_t at = on ? ((int64_t)f.z + (row0 + g) / G) * a.ldq + (int64_t)(h * G + (row0 + g) % G) * D : 0;
            float x[NCH][16], top = 0.f;
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) {
                if (on) load16(a.q, a.dtype, at + (D == 64 ? q * 16 : (2 * q + ch) * 16), x[ch]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (!on) x[ch][e] = 0.f;
                    top = fmaxf(top, finite_abs(x[ch][e]));
                }
            }
            look_up_scales();
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = top > 0.f ? min(max(ilogbf(top), -118), 127) : 0;
            const float mul = exp2i(7 - ex);
            qs = a.scale_log2 * exp2i(ex - 7);
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int st = 0; st < 4; ++st)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t hi, lo;
                        split_pair(x[ch][st * 4 + 2 * e] * mul, x[ch][st * 4 + 2 * e + 1] * mul, hi, lo);
                        qa[ch * 4 + st][0][e] = hi;
                        if constexpr (T == 2) qa[ch * 4 + st][T - 1][e] = lo;
                    }
        }
        // of this lane's rows 2 q + e: position, factor, maximum, sum; numerators of columns out_col(j, g, h)
        int pos[2];
        float qf[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[NJ][4], unit = 0.f, inv = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            pos[e] = 2 * q + e >= rows ? -1 : flat ? L - 1 : p0 + (row0 + 2 * q + e) / G;
            qf[e] = __shfl_sync(0xffffffffu, qs, (2 * q + e) * 4);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;

        // What the first pass has left of this thread's outputs, under the first tiles' way.
        constexpr int PER = R * (D / 4) / NT;   // float4 of outputs to a thread
        const bool cut = k0 > 0 || k1 < nt, join = skips[i] > 0;
        float4 prior[PER];
        // A box's codes into a place: the next tile that is there, in order. kb: the first of the 32 looked up.
        int kb = k0, ka_next = k0;
        auto ask = [&]() {   // by the whole warp
            while (ka_next < k1) {
                if (ka_next - kb >= 32) return;   // (after the tiles that are looked up now)
                const int page = __shfl_sync(0xffffffffu, pid, ka_next - kb), at = (tile0 + ka_next) * KV_TILE + warp * 16;
                ++ka_next;
                if (page < 0) continue;   // absent, or no row sees any of it
                const int slot = asked % C::SLOTS;
                if (lane == 0) {
                    const int row = (page * c.hkv + h) * P + (at & (P - 1));
                    mbar_arrive_expect_tx(&full[slot], 2 * C::BOX);
                    tma_load_2d(ring + slot * 2 * C::BOX, &mk, 0, row, &full[slot]);
                    tma_load_2d(ring + slot * 2 * C::BOX + C::BOX, &mv, 0, row, &full[slot]);
                }
                ++asked;
                return;
            }
        };
        if (!dead)
            for (int x = 0; x < C::SLOTS; ++x) ask();
        // The first pass's parts of the item's rows, joined: their weights, a part to a thread, then the numerators of this
        // thread's outputs.
        auto prior_rows = [&]() {
            const int64_t all = (int64_t)a.b.n_tokens * c.hq;
            auto row_of = [&](int r) { return ((int64_t)f.z + (row0 + r) / G) * c.hq + h * G + (row0 + r) % G; };
            {
                const int r = tid / 16, x = tid % 16;
                float2 p = make_float2(-INFINITY, 0.f);
                if (r < rows && x < a.parts) p = __ldcg((const float2 *)a.prior_ml + row_of(r) + x * all);
                float M = p.x;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                const float w = part_weight(p.x, p.y, M);
                float S = w * p.y;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
                s_pw[r][x] = w;
                if (x == 0) s_pm[r] = M, s_ps[r] = S;
            }
            __syncthreads();
            const float *num[PER];
            const float *pw[PER];
#pragma unroll
            for (int y = 0; y < PER; ++y) {
                const int x = tid + y * NT, r = min(x / (D / 4), rows - 1), d = (x % (D / 4)) * 4;
                num[y] = a.prior + row_of(r) * D + d;
                pw[y] = s_pw[r];
                prior[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll 4
            for (int z = 0; z < a.parts; ++z)
#pragma unroll
                for (int y = 0; y < PER; ++y) {
                    const float4 v = __ldcg((const float4 *)(num[y] + z * all * D));
                    const float w = pw[y][z];
                    float4 &o = prior[y];
                    if (w != 0.f) o.x += v.x * w, o.y += v.y * w, o.z += v.z * w, o.w += v.w * w;   // (an empty part has none)
                }
        };
        auto add_prior = [&](int y, int r, float4 &o, float &M, float &S) {
            const float top = fmaxf(M, s_pm[r]), w0 = part_weight(M, S, top), w1 = part_weight(s_pm[r], s_ps[r], top);
            o = make_float4(o.x * w0 + prior[y].x * w1, o.y * w0 + prior[y].y * w1, o.z * w0 + prior[y].z * w1,
                            o.w * w0 + prior[y].w * w1);
            S = S * w0 + s_ps[r] * w1;
            M = top;
        };
        if (join && !cut) prior_rows();
        for (int k = k0; k < k1; ++k) {
            if (k - kb == 32) {
                kb = k;
                look_up(kb);
                look_up_scales();
                if (!dead)
                    while (asked - taken < (uint32_t)C::SLOTS && ka_next < k1 && ka_next - kb < 32) ask();
            }
            const int page = __shfl_sync(0xffffffffu, pid, k - kb), j0 = (tile0 + k) * KV_TILE + warp * 16;
            const float sk = __shfl_sync(0xffffffffu, ks, k - kb), sv = __shfl_sync(0xffffffffu, vs, k - kb);
            if (page < 0 || dead) continue;
            const int slot = taken % C::SLOTS;
            if (!warp_wait(&full[slot], taken / C::SLOTS & 1)) {
                dead = true;
                set_status(c.status, ST_TIMEOUT);
                continue;
            }
            ++taken;
            const uint8_t *const kt = ring + slot * 2 * C::BOX, *const vt = kt + C::BOX;
            uint4 kc[NCH][2], vc[2][2];   // keys of rows g and g + 8, values of tokens 2 q + e (+ 8)
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    kc[ch][x] = *(const uint4 *)(kt + (D == 64 ? (x * 8 + g) * 64 + ((q ^ ((g >> 1) & 3)) << 4)
                                                               : (x * 8 + g) * 128 + (((2 * q + ch) ^ g) << 4)));
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if constexpr (D == 64) {
                        const uint2 v = *(const uint2 *)(vt + (x * 8 + 2 * q + e) * 64 + (((g >> 1) ^ q) << 4) + (g & 1) * 8);
                        vc[x][e] = make_uint4(v.x, v.y, 0, 0);
                    } else {
                        vc[x][e] = *(const uint4 *)(vt + (x * 8 + 2 * q + e) * 128 + ((g ^ (2 * q + e)) << 4));
                    }
                }
            fence_proxy_async_smem();   // the next copy into the place comes after these loads
            __syncwarp();
            ask();
            // ---- scores: s[2 x + e] of position 8 x + g and row 2 q + e
            float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                    uint32_t ka[4];
                    e4m3x4_f16x4(word4(kc[ch][0], st), ka[0], ka[2]);
                    e4m3x4_f16x4(word4(kc[ch][1], st), ka[1], ka[3]);
                    mma_f16(s, ka, qa[ch * 4 + st][0][0], qa[ch * 4 + st][0][1]);
                    if constexpr (T == 2) mma_f16(s2, ka, qa[ch * 4 + st][T - 1][0], qa[ch * 4 + st][T - 1][1]);
                }
            const bool whole = j0 + 15 <= pos_lo;
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = s[2 * x + e];
                    if constexpr (T == 2) v += s2[2 * x + e];
                    v *= qf[e] * sk;
                    if (!whole && j0 + x * 8 + g > pos[e]) v = -INFINITY;
                    s[2 * x + e] = v;
                    top[e] = fmaxf(top[e], v);
                }
            // ---- running maximum, and the unit of the values
            float corr[2], shrink = 1.f;
            bool grew = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
                const float mn = fmaxf(m[e], top[e]);
                corr[e] = mn > m[e] ? ex2(m[e] - mn) : 1.f;   // m = -infinity: 0
                grew |= mn > m[e];
                m[e] = mn;
                l[e] *= corr[e];
            }
            if (sv > unit) {   // (an append gives zeros the scale 2^-120: the unit's reciprocal has to be finite)
                const float up = fmaxf(sv, 0x1p-126f);
                shrink = unit / up;
                unit = up;
                inv = 1.f / unit;
            }
            if (__any_sync(0xffffffffu, grew) || shrink != 1.f) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] *= corr[e & 1] * shrink;
            }
            if (!whole) {
                // Values that no row of the tile sees must not meet a zero weight (0 * NaN), and a NaN that some rows see
                // is for them alone: both become 0 here, the latter after the rows that see it have it.
                uint32_t nan[2][2] = {};   // bit per byte of each token's words
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t *const w = (uint32_t *)&vc[x][e];
                        if (j0 + x * 8 + 2 * q + e > pos_hi) {
#pragma unroll
                            for (int y = 0; y < 4; ++y) w[y] = 0;
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const uint32_t b = ((w[y] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                            nan[x][e] |= ((b >> 7 & 1u) | (b >> 14 & 2u) | (b >> 21 & 4u) | (b >> 28 & 8u)) << (4 * y);
                            w[y] = e4m3_no_nan(w[y]);
                        }
                    }
                if (__any_sync(0xffffffffu, nan[0][0] | nan[0][1] | nan[1][0] | nan[1][1]))
                    for (int from = 0; from < 4; ++from)   // the lanes with this lane's columns
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t bits = __shfl_sync(0xffffffffu, nan[x][e], g * 4 + from);
                                const int at = j0 + x * 8 + 2 * from + e;
#pragma unroll
                                for (int j = 0; j < NJ; ++j)
#pragma unroll
                                    for (int y = 0; y < 4; ++y)   // column 2 j + (y >> 1) of the lane's, row 2 q + (y & 1)
                                        if ((bits >> (2 * j + (y >> 1)) & 1u) && at <= pos[y & 1]) acc[j][y] = __int_as_float(0x7fc00000);
                            }
            }
            // ---- weights, and their products with the values
            const float scale = sv * inv * 16384.f;
            uint32_t pb[2][2];   // two terms of a weight in every type
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float e0 = ex2(s[2 * x] - (m[0] == -INFINITY ? 0.f : m[0])), e1 = ex2(s[2 * x + 1] - (m[1] == -INFINITY ? 0.f : m[1]));
                l[0] += e0;
                l[1] += e1;
                uint32_t hi, lo;
                split_pair(e0 * scale, e1 * scale, hi, lo);
                pb[0][x] = transpose8(hi);
                pb[1][x] = transpose8(lo);
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
#pragma unroll
                for (int b2 = 0; b2 < 2; ++b2) {   // columns 2 b2 and 2 b2 + 1 of the word
                    uint32_t va[4];
                    e4m3x4_f16x4(__byte_perm(word4(vc[0][0], w), word4(vc[0][1], w), b2 ? 0x7362 : 0x5140), va[0], va[1]);
                    e4m3x4_f16x4(__byte_perm(word4(vc[1][0], w), word4(vc[1][1], w), b2 ? 0x7362 : 0x5140), va[2], va[3]);
                    const int j = w * 2 + b2;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};   // added with rounding
                    mma_f16(sum, va, pb[1][0], pb[1][1]);
                    mma_f16(sum, va, pb[0][0], pb[0][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] += sum[e];
                }
        }
        // ---------------------------------------------------------------- the warps' results, joined
        __syncthreads();   // all boxes have been read: the results take their place
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * q + e;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], o);
            if (g == 0) {
                ml[(warp * R + r) * 2] = m[e];
                ml[(warp * R + r) * 2 + 1] = l[e];
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                *(float2 *)&merge[(warp * R + r) * (D + 4) + out_col<D>(j, g, 0)] =
                    make_float2(acc[j][e] * 0x1p-14f * unit, acc[j][2 + e] * 0x1p-14f * unit);
        }
        __syncthreads();
        int ca = 0, cb = 0;   // the item's CTAs
        if (cut) ca = (int)(first / quota), cb = (int)((first + nt - 1) / quota);
        const int part = (int)blockIdx.x == ca ? 2 * ca + 1 : 2 * (int)blockIdx.x;
        if (tid < rows) {
            float M = -INFINITY, S = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[(w * R + tid) * 2]);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f2 = part_weight(ml[(w * R + tid) * 2], ml[(w * R + tid) * 2 + 1], M);
                S += ml[(w * R + tid) * 2 + 1] * f2;
                ml[(w * R + tid) * 2] = f2;
            }
            sums[tid * 2] = M;
            sums[tid * 2 + 1] = S;
        }
        __syncthreads();
#pragma unroll
        for (int y = 0; y < PER; ++y) {
            const int x = tid + y * NT, r = x / (D / 4), d = (x % (D / 4)) * 4;
            if (r >= rows) break;
            float M = sums[r * 2], S = sums[r * 2 + 1];
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f2 = ml[(w * R + r) * 2];
                const float4 v = *(const float4 *)&merge[(w * R + r) * (D + 4) + d];
                o.x += v.x * f2, o.y += v.y * f2, o.z += v.z * f2, o.w += v.w * f2;
            }
            if (cut) {
                *(float4 *)&a.part[((size_t)part * R + r) * D + d] = o;
                if (d == 0) *(float2 *)&a.part_ml[((size_t)part * R + r) * 2] = make_float2(M, S);
                continue;
            }
            if (join) add_prior(y, r, o, M, S);
            store_row<true>(a, f, h, G, D, row0 + r, d, o, M, S);
        }
        fence_proxy_async_smem();   // (the next item's boxes come after these loads)
        __syncthreads();
        if (!cut) continue;
        if (tid == 0) s_last = ticket_acq_rel(&a.tickets[ca], 1u) == (uint32_t)(cb - ca);
        __syncthreads();
        if (!s_last) continue;
        auto slot = [&](int y) { return y == ca ? 2 * ca + 1 : 2 * y; };
        if (join) prior_rows();
#pragma unroll
        for (int y = 0; y < PER; ++y) {
            const int x = tid + y * NT, r = x / (D / 4), d = (x % (D / 4)) * 4;
            if (r >= rows) break;
            float M = -INFINITY, S = 0.f;
            for (int z = ca; z <= cb; ++z) M = fmaxf(M, __ldcg(&a.part_ml[((size_t)slot(z) * R + r) * 2]));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int z = ca; z <= cb; ++z) {
                const float2 p = __ldcg((const float2 *)&a.part_ml[((size_t)slot(z) * R + r) * 2]);
                const float4 v = __ldcg((const float4 *)&a.part[((size_t)slot(z) * R + r) * D + d]);
                const float w = part_weight(p.x, p.y, M);
                S += w * p.y;
                o.x += v.x * w, o.y += v.y * w, o.z += v.z * w, o.w += v.w * w;
            }
            if (join) add_prior(y, r, o, M, S);
            store_row<true>(a, f, h, G, D, row0 + r, d, o, M, S);
        }
        if (tid == 0) a.tickets[ca] = 0;
        __syncthreads();
    }
    if (dead)   // nothing may land after the CTA is gone: the last copies into each place (bounded)
        for (uint32_t x = 0; x < (uint32_t)C::SLOTS && x < asked; ++x) warp_wait(&full[x], (asked - 1 - x) / C::SLOTS & 1);
}

template <int D, int T>
cudaError_t short_setup()
{
    return cudaFuncSetAttribute(k_kv_short<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ShortCfg<D, T>::SMEM + 28 * PI_KV_MAX_CALL_SEQS + 8 + 1024);
}

template <int D, int T>
cudaError_t short_launch(const KvAttendArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int nsm, cudaStream_t s)
{
    Launch L;
    L.grid = dim3((unsigned)(ShortCfg<D, T>::CTAS * nsm));
    L.block = dim3(ShortCfg<D, T>::NT);
    L.smem = ShortCfg<D, T>::SMEM + 28 * (size_t)a.b.n + 8 + 1024;
    L.stream = s;
    L.pdl = true;
    L.nsm = nsm;
    return launch_ex(L, k_kv_short<D, T>, a, mk, mv);
}

}  // namespace pi
