"""Attention over the paged 8-bit cache where hand-offs between warps, tiles and kernels count: against a plain form in
64 bits on the same codes, every (token, head) row by its own error.

Tolerances (relative L2 error of a row). Output: bf16 rounds by at most 2^-8 of a value, fp16 by 2^-11 (and by 2^-25 where
it is a subnormal: rows whose weight lies on values of zero are that small). Weights of 16-bit
types are f16: 2^-11 / sqrt(3) of each on average, and over the 64 or more columns of a row that is 2.8e-4 of it; four
times that for rows that fall badly. fp32: terms of 22 bits, but the tensor cores cut sums off by up to 2^-23 of them at
every addition: 32 additions into a score of up to 10 (3.8e-5), and one for each 8 positions into an output.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROW_TOL = {"f32": 3.8e-5, "bf16": 2.0 ** -8 + 1.2e-3, "f16": 2.0 ** -11 + 1.2e-3}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def P():
    import activation_sparse_decode_pi_gb300 as P

    return P


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), device="cuda").to(dtype)


def starts(new):
    return dev(np.concatenate([[0], np.cumsum(new)]))


class Filled:
    """A cache whose pages were filled with random codes and scales, in shuffled order."""

    def __init__(self, P, lens, *, hq, hkv, dim, page, seed=0, spread=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        cols = [-(-n // page) for n in lens]
        n_pages = sum(cols) + 3
        self.lens, self.hq, self.hkv, self.dim, self.page = lens, hq, hkv, dim, page

        def pool():
            x = torch.randn((n_pages, hkv, page, dim), generator=g, device="cuda").mul_(64).clamp_(-448, 448)
            s = torch.exp2(torch.randint(-7, -6 + spread, (n_pages, hkv), generator=g, device="cuda").float())
            return x.to(torch.float8_e4m3fn), s
        self.k, self.ks = pool()
        self.v, self.vs = pool()
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(lens), max(cols)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, c in enumerate(cols):
            self.table[i, :c] = order[at:at + c]
            at += c
        ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        ref[order[:at].long()] = 1
        self.g = g
        self.cache = P.KVCache([dict(k=self.k, v=self.v, k_scale=self.ks, v_scale=self.vs)], self.table, dev(lens), ref,
                               n_heads=hq)

    def queries(self, new, kind):
        return torch.randn((int(sum(new)), self.hq, self.dim), generator=self.g, device="cuda").to(TYPES[kind])

    def attend(self, new, q, **kw):
        return self.cache.attend(0, dev(range(len(self.lens))), starts(new), q, **kw)

    def exact(self, new, q, window=0, sinks=0, by_column=False):
        """(out, lse) in fp64 from the definition, a sequence and kv head at a time. by_column: a NaN value is in the sums
        of the rows that see it only (in products it meets weights of zero, too)."""
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.full(q.shape[:2], -torch.inf, dtype=torch.float64, device="cuda")
        G, row = self.hq // self.hkv, 0
        for i, (total, m) in enumerate(zip(self.lens, new)):
            if m == 0:
                continue
            j = torch.arange(total, device="cuda")
            page = self.table[i].long()[j // self.page]
            pos = torch.arange(total - m, total, device="cuda")[:, None]
            see = j[None] <= pos
            if window > 0:
                see &= (pos - j[None] < window) | (j[None] < sinks)
            see &= page[None] >= 0
            keep = see.any(0)                                    # (0 * NaN: what nothing sees is not summed)
            j, page, see = j[keep], page[keep], see[:, keep]
            for h in range(self.hkv):
                k, v = ((x.view(torch.uint8)[page, h, j % self.page].view(torch.float8_e4m3fn).double()
                         * s[page, h].double()[:, None]) for x, s in ((self.k, self.ks), (self.v, self.vs)))
                x = q[row:row + m, h * G:(h + 1) * G].double()
                x = torch.einsum("tgd,kd->tgk", x, k) * self.dim ** -0.5
                x = x.masked_fill(~see[:, None], -torch.inf)
                lse[row:row + m, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300))
                z = p.sum(-1, keepdim=True)
                o = torch.einsum("tgk,kd->tgd", p, v.nan_to_num() if by_column else v) / torch.where(z == 0, 1.0, z)
                if by_column:
                    o[((see.double() @ v.isnan().double()) > 0)[:, None].expand_as(o)] = torch.nan
                out[row:row + m, h * G:(h + 1) * G] = o
            row += m
        return out, lse

    def check(self, new, kind, window=0, sinks=0, repeat=0):
        q = self.queries(new, kind)
        lse = torch.empty(q.shape[:2], device="cuda")
        got = self.attend(new, q, lse=lse, window=window, sinks=sinks)
        want, want_lse = self.exact(new, q, window, sinks)
        below = 2.0 ** -25 * self.dim ** 0.5 if kind == "f16" else 0.0
        err = ((got.double() - want).norm(dim=-1) - below) / want.norm(dim=-1).clamp(min=1e-300)
        assert self.cache.status() == 0
        bad = torch.nonzero(~(err <= ROW_TOL[kind] + max(self.lens) / 8 * 2.0 ** -23))
        assert bad.numel() == 0, (len(bad), err.max().item(), bad[:8].tolist())
        assert torch.allclose(lse.double(), want_lse, rtol=1e-5, atol=5e-5)
        outs = [self.attend(new, q, window=window, sinks=sinks) for _ in range(repeat)]
        assert self.cache.status() == 0
        assert all(torch.equal(o, got) for o in outs)


# ------------------------------------------------------------------------------------------------ few rows

@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("group", [1, 16])
def test_few_rows_ring_shorter_than_the_warps_tiles(P, kind, group):
    """Head dim 256: the ring has 8 to 10 slots, fewer than two for each consumer warp, so that warps wait for a slot's
    next filling while an earlier one is on its way. Many short items and some long ones, call after call."""
    lens = [3 + 37 * i % 700 for i in range(70)] + [9001]
    f = Filled(P, lens, hq=4 * group, hkv=4, dim=256, page=32)
    f.check([1] * len(lens), kind, repeat=100)


# ------------------------------------------------------------------------------------------------ prompts

LONG = [1750, 903, 37, 1290]
CHUNKS = [1700, 903, 30, 260]
PROMPTS = [   # group, kv heads, dim, page
    (1, 24, 64, 16), (5, 4, 64, 64), (2, 8, 64, 128), (1, 24, 128, 32), (4, 8, 128, 16), (8, 3, 128, 128),
    (1, 16, 256, 32), (3, 5, 256, 128), (16, 2, 128, 64), (16, 1, 256, 64),
]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group,hkv,dim,page", PROMPTS)
def test_prompt_rows_one_by_one(P, group, hkv, dim, page, kind):
    """Ragged prompts of many tiles and several waves of CTAs, whole and under windows: every row, and 50 calls bit for
    bit."""
    f = Filled(P, LONG, hq=group * hkv, hkv=hkv, dim=dim, page=page)
    f.check(CHUNKS, kind, repeat=50)
    f.check([700, 1, 37, 1290], kind, window=333, sinks=70, repeat=10)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 64), (256, 16)])
def test_short_prompt_over_a_long_cache(P, dim, page, kind):
    """Few items: each one's cache is split over CTAs, and the last of them joins the parts."""
    f = Filled(P, [6007, 129], hq=6, hkv=2, dim=dim, page=page)
    f.check([61, 129], kind, repeat=50)
    f.check([150, 0], kind, window=3000, sinks=200, repeat=10)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompts_that_end_inside_a_warp(P, dim, kind):
    """Every count of rows in the last warp: its lanes past the end take part in the loads of the results."""
    new = [34 + i for i in range(33)] + [129, 257, 287]
    f = Filled(P, [n + 7 * i % 50 for i, n in enumerate(new)], hq=2, hkv=2, dim=dim, page=16)
    f.check(new, kind, repeat=10)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_weights_are_not_written_over(P, dim, kind):
    """Hundreds of tiles in a row for each CTA: the next tile's scores never reach weights that are still being read."""
    f = Filled(P, [12000, 11000], hq=32, hkv=32, dim=dim, page=64)
    f.check([256, 513], kind, repeat=100)


def test_prompt_attention_right_before_the_tensor_core_ffn(P):
    """The predictor's kernel starts while the attention's last CTAs run, and takes tensor memory before it waits."""
    from workload import WORKLOADS, make_layer, scaled

    w = scaled(WORKLOADS["relullama7b_d4096_f11008_bf16_L32"], d=1024, f=2752, r=128, n_layers=1)
    ffn = P.SparseFFN.from_workload(w, [P.apply_hot_first(make_layer(w, 0, 0, device="cuda"))[0]], max_batch=64)
    u = torch.randn(64, 1024, device="cuda")
    idx, count = ffn.predict(0, u)
    for dim in (64, 128, 256):
        f = Filled(P, [900, 700], hq=8, hkv=8, dim=dim, page=64)
        q = f.queries([800, 700], "f16")
        want = f.attend([800, 700], q)
        for _ in range(30):
            got = f.attend([800, 700], q)
            idx2, count2 = ffn.predict(0, u)
            n = int(count)
            assert torch.equal(got, want) and int(count2) == n and torch.equal(idx2[:n], idx[:n])
        assert f.cache.status() == 0
    assert ffn.status() == 0
    ffn.close()


# ------------------------------------------------------------------------------------------------ refusals

def test_row_strides_whose_extent_passes_64_bits(P):
    """2^30 rows of 2^34 (or 2^40) fp32 elements: their extent is 0 modulo 2^64. (The one sequence has no new token, so
    that nothing is read even if the call is taken.)"""
    f = Filled(P, [40], hq=2, hkv=2, dim=64, page=16)
    seqs, start = dev([0]), dev([0, 0])
    q = torch.zeros((1, 2, 64), device="cuda")
    for ld in (1 << 34, 1 << 40):
        for n in ((1 << 30) - 1, 1 << 30):
            for a, b in ((ld, 128), (128, ld), (ld, ld)):
                with pytest.raises(P.PiError) as e:
                    P.pi_kv_attend(f.cache.h, 0, seqs, start, 1, n, q, a, q, b, None, P.PI_F32, 0.1)
                assert e.value.code == P.PI_ERR_INVALID_ARG
            with pytest.raises(P.PiError) as e:
                P.pi_kv_append(f.cache.h, 0, seqs, start, 1, n, q, q, ld, P.PI_F32)
            assert e.value.code == P.PI_ERR_INVALID_ARG
    assert f.cache.status() == 0


# ------------------------------------------------------------------------------------------------ streams

def test_results_belong_to_the_stream_of_the_call(P):
    """Memory freed on one stream (whose work may still use it) is not handed to a call on another, given as a torch
    stream or as a handle."""
    f = Filled(P, [300], hq=8, hkv=8, dim=64, page=16)
    q = f.queries([300], "f32")
    want = f.attend([300], q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        freed = torch.empty_like(q)
        at = freed.data_ptr()
        del freed                                                # the current stream's next block of this size
        out = f.attend([300], q, stream=stream)
        assert out.data_ptr() != at
        side.synchronize()
        assert torch.equal(out, want)
        del out
        assert f.cache.compact(stream=stream).data_ptr() != torch.empty(1, dtype=torch.int32, device="cuda").data_ptr()
    with torch.cuda.stream(side):                                # the default stream's handle is 0
        freed = torch.empty_like(q)
        at = freed.data_ptr()
        del freed
        out = f.attend([300], q, stream=0)
        assert out.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(out, want) and f.cache.status() == 0


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_codes_are_read_before_the_next_copy_lands(P, dim, page, kind):
    """Short parts of a split cache, where the next tile's copy follows at once on the loads of the last."""
    f = Filled(P, [6007], hq=6, hkv=2, dim=dim, page=page)
    f.check([61], kind, repeat=200)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 1), (64, 16), (128, 1), (128, 16), (256, 1), (256, 16)])
def test_few_rows_codes_are_read_before_the_next_copy_lands(P, dim, group, kind):
    """Single tokens over caches of many rounds of the ring, call after call bit for bit."""
    f = Filled(P, [9000 + 501 * i for i in range(12)], hq=4 * group, hkv=4, dim=dim, page=64)
    f.check([1] * 12, kind, repeat=200)


# ------------------------------------------------------------------------------------------------ values of any size

SIZES = [(64, 16, 1), (64, 64, 12), (128, 32, 3), (128, 64, 16), (256, 16, 1), (256, 128, 9)]   # dim, page, group


def zero_positions(f, seq, p0, p1):
    """Values of zero at positions [p0, p1) of a sequence, whole pages of them as an append leaves them."""
    for c in range(p0 // f.page, p1 // f.page):
        f.v.view(torch.uint8)[f.table[seq, c].long()] = 0
        f.vs[f.table[seq, c].long()] = 2.0 ** -120


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,page,group", SIZES)
def test_a_cache_of_zero_values(P, dim, page, group, kind):
    """Every value zero, appended as such: outputs of zero, and the logs of the sums as ever."""
    lens = [300, 64, 1100]
    f = Filled(P, lens, hq=2 * group, hkv=2, dim=dim, page=page)
    x = torch.randn((sum(lens), 2, dim), device="cuda")
    f.cache.append(0, dev(range(3)), starts(lens), x, torch.zeros_like(x))
    assert (f.vs[f.table[0, 0].long()] == 2.0 ** -120).all()
    for new in ([1, 1, 1], [2, 1, 1], [300, 64, 1100]):
        f.check(new, kind)
        f.check(new, kind, window=100, sinks=3)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,page,group", SIZES)
def test_tiles_of_zero_values_among_others(P, dim, page, group, kind):
    """64, 128 and 512 zero positions before, between and behind others."""
    lens = [3000, 704, 1024, 1536]
    f = Filled(P, lens, hq=2 * group, hkv=2, dim=dim, page=page)
    for seq, p0, p1 in ((0, 0, 128), (0, 1024, 1536), (1, 0, 640), (2, 512, 1024), (3, 256, 384), (3, 1024, 1152)):
        zero_positions(f, seq, p0, p1)
    for new in ([1, 1, 1, 1], [3, 0, 2, 1], [700, 600, 1024, 90]):
        f.check(new, kind)
        f.check(new, kind, window=900, sinks=130)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim,page,group", SIZES)
@pytest.mark.parametrize("low", [-120, -115, -113])
def test_values_of_the_smallest_scales(P, dim, page, group, kind, low):
    f = Filled(P, [900, 517], hq=2 * group, hkv=2, dim=dim, page=page)
    f.vs.fill_(2.0 ** low)
    f.vs[f.table[0, 3:5].long()] = 2.0 ** -120
    for new in ([1, 1], [2, 1], [850, 517]):
        f.check(new, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim,page,group", SIZES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -1.0])
def test_pages_whose_scale_is_no_scale(P, dim, page, group, kind, bad):
    """A page in view with a scale that is not a number >= 0: left out and flagged like an absent one, by every kernel."""
    f = Filled(P, [900, 517], hq=2 * group, hkv=2, dim=dim, page=page)
    whole = f.table.clone()
    f.ks[f.table[0, 2].long(), 0] = bad
    f.vs[f.table[0, 4].long(), 1] = bad
    f.vs[f.table[1, 1].long(), 0] = bad
    left = {0: [(0, 2), (1, 1)], 1: [(0, 4)]}                    # kv head: (sequence, column) left out
    for new in ([1, 1], [2, 1], [700, 517]):
        q = f.queries(new, kind)
        got = f.attend(new, q).double()
        assert f.cache.status() == P.PI_ERR_DEVICE_CHECK
        for h, gone in left.items():
            for i, c in gone:
                f.table[i, c] = -1
            want, _ = f.exact(new, q)
            f.table.copy_(whole)
            a, b = got[:, h * group:(h + 1) * group], want[:, h * group:(h + 1) * group]
            err = (a - b).norm(dim=-1) / b.norm(dim=-1).clamp(min=1e-300)
            assert (err <= ROW_TOL[kind] + 900 / 8 * 2.0 ** -23).all(), (h, new, err.max().item())
    f.check([1, 0], kind, window=1)                              # out of view: not looked at


def test_lengths_out_of_range_are_left_alone(P):
    """A sequence whose length its row cannot have: skipped and flagged by every call, its pages and length untouched."""
    f = Filled(P, [100, 200], hq=4, hkv=2, dim=64, page=16)
    c = f.cache
    q = f.queries([1, 1], "f32")
    want = f.attend([0, 1], q[1:])                               # (cut alike, so the same bits)
    assert c.status() == 0
    x = torch.randn((2, 2, 64), device="cuda")
    for bad in (-1, f.table.shape[1] * 16 + 1, -2 ** 31, 2 ** 31 - 1):
        c.length[0] = bad
        table, ref, k = f.table.clone(), c.ref.clone(), f.k.view(torch.uint8).clone()
        c.reserve(dev([0]), dev([0, 1]))
        assert c.status() == P.PI_ERR_DEVICE_CHECK
        assert int(c.length[0]) == bad and torch.equal(f.table, table) and torch.equal(c.ref, ref)
        out = torch.full_like(q, 7.0)
        f.attend([1, 1], q, out=out)
        assert c.status() == P.PI_ERR_DEVICE_CHECK
        assert (out[0] == 7).all() and torch.equal(out[1], want[0])
        c.append(0, dev([0]), dev([0, 2]), x, x)
        assert c.status() == P.PI_ERR_DEVICE_CHECK and torch.equal(f.k.view(torch.uint8), k)


def test_scales_of_the_scores_at_the_ends_of_fp32(P):
    """The scale is multiplied by log2(e): one that leaves fp32 with it is refused, the largest others and 0 are right."""
    f = Filled(P, [150], hq=2, hkv=2, dim=64, page=16)
    for new in ([1], [150]):
        q = f.queries(new, "f32")
        for scale in (3e38, -3e38):
            with pytest.raises(P.PiError) as e:
                f.attend(new, q, scale=scale)
            assert e.value.code == P.PI_ERR_INVALID_ARG
        small = torch.full_like(q, 2.0 ** -126)
        big = f.attend(new, small, scale=2.0 ** 126)             # scores of q * scale = 1 in every column
        one = f.attend(new, torch.ones_like(q), scale=1.0)
        assert (big - one).norm() <= 1e-5 * one.norm()
        flat = f.attend(new, q, scale=0.0)
        mean = f.attend(new, torch.zeros_like(q))
        assert (flat - mean).norm() <= 1e-6 * mean.norm() and f.cache.status() == 0


# ------------------------------------------------------------------------------------------------ NaN codes

def spoil(f, seq, pos, h, col, which="v"):
    x = (f.v if which == "v" else f.k).view(torch.uint8)
    x[f.table[seq, pos // f.page].long(), h, pos % f.page, col] = 0x7f


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,page,group", SIZES)
@pytest.mark.parametrize("seqs", [1, 40])
def test_nan_codes_reach_the_rows_that_see_them(P, dim, page, group, kind, seqs):
    """NaN values in the last, partial tile, at a window's edge and among the first tokens, for few rows and for prompts
    (of one sequence, whose cache is split, and of many), and NaN keys, which reach every column."""
    lens = [700 + i for i in range(seqs)]
    f = Filled(P, lens, hq=2 * group, hkv=2, dim=dim, page=page)
    last = seqs - 1
    for pos, h, col in ((lens[last] - 1, 0, 5), (lens[last] - 3, 1, dim - 1), (lens[last] - 40, 0, 0), (600, 1, 17), (2, 0, 9)):
        spoil(f, last, pos, h, col)
    spoil(f, 0, 650, 1, 3, "k")
    for m in (1, 2, 8, 160):
        if m * group * seqs > 20000:
            continue
        new = [m] * seqs
        q = f.queries(new, kind)
        for kw in (dict(), dict(window=101, sinks=0), dict(window=40, sinks=3), dict(window=650, sinks=1)):
            got = f.attend(new, q, **kw).double()
            want, _ = f.exact(new, q, by_column=True, **kw)
            assert f.cache.status() == 0
            assert torch.equal(got.isnan(), want.isnan()), (m, kw, torch.nonzero(got.isnan() != want.isnan())[:6].tolist())
            ok = ~want.isnan()
            a, b = torch.where(ok, got, 0.0), torch.where(ok, want, 0.0)
            err = (a - b).norm(dim=-1) / b.norm(dim=-1).clamp(min=1e-300)
            assert (err <= ROW_TOL[kind] + 740 / 8 * 2.0 ** -23).all(), (m, kw, err.max().item())


# ------------------------------------------------------------------------------------------------ ends of the ranges

@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim,group", [(64, 1), (64, 16), (128, 3), (128, 16), (256, 2), (256, 16)])
def test_as_many_sequences_as_a_call_takes(P, dim, group, kind):
    """1024 sequences: the call's tables leave the ring the fewest slots. Single tokens, and short prompts among them."""
    lens = [1 + 29 * i % 190 for i in range(1024)]
    f = Filled(P, lens, hq=group, hkv=1, dim=dim, page=16)
    f.check([1] * 1024, kind, repeat=5)
    f.check([min(n, 3 if i % 3 else 50) for i, n in enumerate(lens)], kind, repeat=5)
    f.check([min(n, i % 2) for i, n in enumerate(lens)], kind, window=20, sinks=2, repeat=5)


def test_offsets_past_32_bits(P):
    """Pools of more than 2^32 bytes with the sequences' pages at their ends: append, attention and page copies."""
    dim, page, hkv, n_pages = 256, 64, 2, 140000
    k, v = (torch.empty((n_pages, hkv, page, dim), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            for _ in range(2))
    ks, vs = (torch.ones((n_pages, hkv), device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 32
    cols = 14
    table = torch.arange(n_pages - 1, n_pages - 1 - cols, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    ref[table[0].long()] = 1
    f = Filled(P, [cols * page - 5], hq=8, hkv=hkv, dim=dim, page=page)      # the same sequence in a small pool
    small = f.table[0, :cols].long()
    f.cache.append(0, dev([0]), starts(f.lens), *[torch.randn((f.lens[0], hkv, dim), device="cuda") for _ in range(2)])
    cache = P.KVCache([dict(k=k, v=v, k_scale=ks, v_scale=vs)], table, dev(f.lens), ref, n_heads=8)
    g = torch.Generator(device="cuda").manual_seed(5)
    new = [torch.randn((f.lens[0], hkv, dim), generator=g, device="cuda") for _ in range(2)]
    f.cache.append(0, dev([0]), starts(f.lens), *new)
    cache.append(0, dev([0]), starts(f.lens), *new)
    for a, b in ((k, f.k), (v, f.v)):
        at = a.view(torch.uint8)[table[0].long()].transpose(1, 2).reshape(-1, hkv, dim)[:f.lens[0]]
        assert torch.equal(at, b.view(torch.uint8)[small].transpose(1, 2).reshape(-1, hkv, dim)[:f.lens[0]])
    for m in (1, 3, 300):
        q = f.queries([m], "bf16")
        assert torch.equal(cache.attend(0, dev([0]), starts([m]), q), f.attend([m], q))
    cache.compact()                                              # from the pool's end to its start
    assert table[0].sort().values.tolist() == list(range(cols))
    q = f.queries([70], "f32")
    assert torch.equal(cache.attend(0, dev([0]), starts([70]), q), f.attend([70], q)) and cache.status() == 0
    cache.copy_pages(table[0, :1].contiguous(), dev([n_pages - 1]))
    assert torch.equal(k.view(torch.uint8)[n_pages - 1], k.view(torch.uint8)[table[0, 0].long()]) and cache.status() == 0
