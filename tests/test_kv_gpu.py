"""The paged 8-bit cache on the GPU against the plain NumPy cache: bookkeeping, codes and scales exactly, attention in
fp64 within what its types round.

Tolerances (relative L2 over a call's outputs): one rounding to bf16 is at most 2^-9 of a value, to fp16 2^-12 + its
weights' 2^-22; fp32 outputs carry logits of size up to ~40 in base 2 (each rounded to 2^-24 of itself: ~3e-6 of a
weight), 22-bit weights and queries, and fp32 sums.
"""
import numpy as np
import pytest
import torch

from tests.kv_plain import PlainCache

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 2.0 ** -9 + 2.0 ** -11, "f16": 2.0 ** -12 + 1e-5}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def P():
    import activation_sparse_decode_pi_gb300 as P

    return P


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), device="cuda").to(dtype)


class Both:
    """One cache on the GPU, its plain twin, and the calls made on both."""

    def __init__(self, P, *, layers=1, hq=4, hkv=2, dim=64, page=16, n_pages=64, max_seqs=8, max_pages=16, seed=0):
        self.rng = np.random.default_rng(seed)
        self.plain = PlainCache(layers, hq, hkv, dim, page, n_pages, max_seqs, max_pages, rng=self.rng)
        p = self.plain
        self.k, self.v = (torch.tensor(x, device="cuda").view(torch.float8_e4m3fn) for x in (p.k, p.v))
        self.ks, self.vs = (torch.tensor(x, device="cuda", dtype=torch.float32) for x in (p.ks, p.vs))
        self.cache = P.KVCache([dict(k=self.k[i], v=self.v[i], k_scale=self.ks[i], v_scale=self.vs[i])
                                for i in range(layers)], dev(p.table), dev(p.length), dev(p.ref), n_heads=hq)

    def args(self, seqs, new):
        return dev(seqs), dev(np.concatenate([[0], np.cumsum(new)]))

    def reserve(self, seqs, new):
        self.plain.reserve(seqs, new)
        self.cache.reserve(*self.args(seqs, new))

    def tokens(self, new, kind, heads, fused=0, spread=2):
        """[T, heads, dim] values of a type, rows `fused` elements wider than they have to be."""
        T, w = int(sum(new)), heads * self.plain.dim
        x = self.rng.standard_normal((T, w + fused)) * 2.0 ** self.rng.integers(-spread, spread + 1, (T, 1))
        full = torch.tensor(x, device="cuda").to(TYPES[kind])
        part = full[:, fused // 2:fused // 2 + w].unflatten(1, (heads, self.plain.dim))
        return part, part.double().cpu().numpy()

    def append(self, layer, seqs, new, kind="f32", fused=0, change=None):
        k, kn = self.tokens(new, kind, self.plain.hkv, fused)
        v, vn = self.tokens(new, kind, self.plain.hkv, fused)
        if change is not None:
            for x, n in ((k, kn), (v, vn)):
                change(n)
                x.copy_(torch.tensor(n, device="cuda").to(x.dtype))
        self.plain.append(layer, seqs, new, kn, vn)
        self.cache.append(layer, *self.args(seqs, new), k, v)

    def grow(self, seqs, new, **kw):
        self.reserve(seqs, new)
        for layer in range(self.plain.k.shape[0]):
            self.append(layer, seqs, new, **kw)

    def same(self, status=0):
        p = self.plain
        assert self.cache.status() == status
        for name in ("table", "length", "ref"):
            assert np.array_equal(getattr(self.cache, name).cpu().numpy(), getattr(p, name)), name
        for name, mine in (("k", self.k), ("v", self.v)):
            assert np.array_equal(mine.view(torch.uint8).cpu().numpy(), getattr(p, name)), name
        for name, mine in (("ks", self.ks), ("vs", self.vs)):
            assert np.array_equal(mine.double().cpu().numpy(), getattr(p, name), equal_nan=True), name

    def attend(self, seqs, new, kind="f32", window=0, sinks=0, fused=0, layer=0, scale=None, sharp=1.0):
        p = self.plain
        q, qn = self.tokens(new, kind, p.hq, fused, spread=0)
        q *= sharp
        qn = q.double().cpu().numpy()
        scale = p.dim ** -0.5 if scale is None else scale
        lse = torch.full(q.shape[:2], 123.0, device="cuda")
        out = self.cache.attend(layer, *self.args(seqs, new), q, lse=lse, scale=scale, window=window, sinks=sinks)
        want, want_lse = p.attend(layer, seqs, new, qn, scale, window, sinks)
        got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert out.dtype is TYPES[kind] and self.cache.status() == 0
        nothing = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), nothing)
        assert not got[nothing].any()
        assert np.allclose(got_lse[~nothing], want_lse[~nothing], rtol=1e-5, atol=2e-5)
        assert np.isfinite(got).all()
        if want.any():
            err = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert err <= TOL[kind], err
        return out


# ------------------------------------------------------------------------------------------------ append

@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,page,hkv", [(64, 16, 3), (128, 32, 2), (128, 128, 1), (256, 64, 1)])
def test_append_codes_and_scales(P, kind, dim, page, hkv):
    b = Both(P, hq=hkv, hkv=hkv, dim=dim, page=page, n_pages=40, max_pages=10)
    b.grow([3, 0, 5], [1, page, page + 1], kind=kind)
    b.same()
    b.grow([5, 3, 1], [page - 1, 3, 0], kind=kind, fused=64)     # ends a page exactly; none for one
    b.grow([0, 5, 3], [2 * page + 5, 1, 1], kind=kind, fused=64)
    b.same()


def test_append_scale_grows_and_requantises(P):
    b = Both(P, hq=1, hkv=1, dim=64, page=16)
    for i in range(12):                                          # each token 2.7 times the last
        b.grow([2], [1], change=lambda x, i=i: x.__imul__(2.7 ** i / 50))
    b.same()
    for i in range(3):                                           # and smaller ones leave the scale alone
        b.grow([2], [1], change=lambda x: x.__imul__(1e-6))
    b.same()


def test_append_extreme_values(P):
    b = Both(P, hq=2, hkv=2, dim=64, page=16)

    def put(x):
        x[0, 0, :5] = [np.inf, -np.inf, np.nan, 448.0, -0.0]
        x[0, 1] = 0.0                                            # an all-zero block
        x[1, 0, :4] = [1e38, -3e38, 1e-38, 0.0]
        x[2, 1] = np.nan
    b.grow([1], [3], change=put)
    b.grow([4], [1], change=lambda x: x.fill(448.0 * 2.0 ** -30))       # exactly the largest code
    b.grow([5], [1], change=lambda x: x.fill(np.float32(448.0 * (1 + 2.0 ** -20))))
    b.grow([6], [2], change=lambda x: x.fill(0.0))
    b.grow([6], [2])
    b.same()


# ------------------------------------------------------------------------------------------------ attention

SHAPES = [
    dict(hq=2, hkv=2, dim=64, page=16),
    dict(hq=8, hkv=2, dim=128, page=64),
    dict(hq=15, hkv=3, dim=128, page=32),
    dict(hq=16, hkv=1, dim=128, page=128),
    dict(hq=20, hkv=1, dim=64, page=32),
    dict(hq=4, hkv=4, dim=256, page=64),
    dict(hq=12, hkv=1, dim=256, page=16),
]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s['hq']}of{s['hkv']}x{s['dim']}p{s['page']}")
def test_attend_one_token(P, shape, kind):
    lens = [1, 63, 64, 65, 517, 128, 16, 1000]
    b = Both(P, n_pages=-(-2000 // shape["page"]) + 16, max_pages=-(-1024 // shape["page"]), **shape)
    b.grow(list(range(8)), lens)
    new = [1] * 8
    b.attend(list(range(8)), new, kind)
    b.attend([5], [1], kind, fused=128, sharp=8.0)               # a peaked softmax, a strided query
    b.attend([7, 2, 4], [1, 1, 1], kind, window=100, sinks=5)
    b.attend([7, 0], [1, 1], kind, window=1)
    b.attend([7, 4], [1, 1], kind, window=65, sinks=130)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s['hq']}of{s['hkv']}x{s['dim']}p{s['page']}")
def test_attend_many_tokens(P, shape, kind):
    """Prompt chunks beside single tokens, sequences without a token, queries before position 0."""
    lens = [40, 64, 130, 3, 300]
    b = Both(P, n_pages=-(-600 // shape["page"]) + 12, max_pages=-(-320 // shape["page"]), **shape)
    b.grow(list(range(5)), lens)
    b.attend([4, 0, 2, 1], [100, 40, 130, 1], kind)
    b.attend([3, 4, 1], [5, 0, 64], kind)                        # two queries of sequence 3 see nothing
    b.attend([4, 2], [300, 77], kind, window=50, sinks=3)
    b.attend([4], [200], kind, window=130, sinks=70, fused=64)
    b.attend([6, 4], [2, 1], kind)                               # an empty sequence


def test_attend_long_sequence_is_split(P):
    b = Both(P, hq=8, hkv=1, dim=128, page=64, n_pages=400, max_pages=320)
    b.grow([0, 1], [20000, 77])
    b.attend([0], [1], "f32")
    b.attend([0, 1], [1, 1], "f32")
    b.attend([0], [3], "bf16", window=15000, sinks=100)


def test_attend_same_bits_every_time(P):
    b = Both(P, hq=16, hkv=2, dim=128, page=64, n_pages=200, max_pages=128)
    b.grow([0, 1, 2], [8000, 63, 2500])
    q = torch.randn(3, 16, 128, device="cuda")
    a = b.args([0, 1, 2], [1, 1, 1])
    first = b.cache.attend(0, *a, q)
    for _ in range(20):
        assert torch.equal(b.cache.attend(0, *a, q), first)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_attend_many_short_sequences(P, kind):
    """Thousands of items of one to five tiles, call after call without a pause: every share is a chain of short
    segments that some warps have no tile of. No wait may run out, and the bits stay the same."""
    heads, seqs = 40, 85
    lens = [3 + 7 * i % 299 for i in range(seqs)]
    b = Both(P, hq=heads, hkv=heads, dim=128, page=32, n_pages=600, max_seqs=seqs, max_pages=10)
    b.cache.reserve(*b.args(range(seqs), lens))
    k = torch.randn(sum(lens), heads, 128, device="cuda", dtype=TYPES[kind])
    b.cache.append(0, *b.args(range(seqs), lens), k, k.flip(0))
    q = torch.randn(seqs, heads, 128, device="cuda", dtype=TYPES[kind])
    a = b.args(range(seqs), [1] * seqs)
    first = b.cache.attend(0, *a, q)
    outs = [b.cache.attend(0, *a, q) for _ in range(300)]
    assert b.cache.status() == 0
    assert all(torch.equal(o, first) for o in outs)


def test_attend_block_scales_far_apart(P):
    """Pages whose scales differ by many powers of two, and a page of zeros, in one sequence."""
    b = Both(P, hq=2, hkv=1, dim=128, page=16, n_pages=32, max_pages=16)
    for i in range(10):
        b.grow([0], [16], change=lambda x, i=i: x.__imul__(0.0 if i == 4 else 2.0 ** ((7 * i) % 11 - 8)))
    b.attend([0], [1], "f32")
    b.attend([0], [1], "f32", sharp=0.01)


def test_attend_nan_only_reaches_who_sees_it(P):
    """A NaN value is seen by later queries only, and by none once a window has passed it."""
    for dim, page in ((64, 16), (128, 64), (256, 32)):
        b = Both(P, hq=2, hkv=1, dim=dim, page=page, n_pages=40, max_pages=20)

        def put(x):
            x[50, 0, 3] = np.nan
        b.reserve([0], [120])
        k, kn = b.tokens([120], "f32", 1)
        v, vn = b.tokens([120], "f32", 1)
        put(vn)
        v.copy_(torch.tensor(vn, device="cuda"))
        b.plain.append(0, [0], [120], kn, vn)
        b.cache.append(0, *b.args([0], [120]), k, v)
        for window in (0, 20):
            q, qn = b.tokens([120], "f32", 2, spread=0)
            got = b.cache.attend(0, *b.args([0], [120]), q, scale=0.1, window=window).cpu().numpy()
            want, _ = b.plain.attend(0, [0], [120], qn, 0.1, window)
            assert np.array_equal(np.isnan(got), np.isnan(want)), (dim, window)
            ok = ~np.isnan(want)
            assert np.linalg.norm(got[ok] - want[ok]) <= TOL["f32"] * np.linalg.norm(want[ok])


def test_attend_does_not_touch_other_rows(P):
    b = Both(P, hq=4, hkv=2, dim=128, page=32, n_pages=16)
    b.grow([0], [40])
    out = torch.full((6, 4, 160), 7.0, device="cuda")            # wider rows; more of them than the call has tokens
    q = torch.randn(6, 4, 128, device="cuda")
    wide = torch.full((6, 4 * 128 + 32), 7.0, device="cuda")
    view = wide[:, :512].unflatten(1, (4, 128))
    b.cache.attend(0, *b.args([0], [4]), q, out=view)
    assert (wide[4:] == 7).all() and (wide[:, 512:] == 7).all() and not (wide[:4, :512] == 7).any()
    assert out.eq(7).all()


# ------------------------------------------------------------------------------------------------ pages

@pytest.mark.parametrize("seed", range(4))
def test_session_of_every_call(P, seed):
    """Random calls in a row; state, codes and scales equal after each, attention along the way."""
    page, dim, hkv = [(16, 64, 2), (32, 128, 1), (64, 128, 2), (16, 256, 1)][seed]
    b = Both(P, layers=2, hq=4, hkv=hkv, dim=dim, page=page, n_pages=60, max_seqs=10, max_pages=12, seed=seed)
    rng = np.random.default_rng(100 + seed)
    b.grow([0, 1, 2], [5, page, 3 * page + 1])
    for _ in range(25):
        live = [s for s in range(10) if b.plain.length[s] > 0]
        idle = [s for s in range(10) if b.plain.length[s] == 0]
        what = rng.choice(["grow", "grow", "fork", "free", "trim", "compact", "attend"])
        if what == "grow":
            seqs = list(rng.permutation(10)[:rng.integers(1, 5)])
            room = [12 * page - int(b.plain.length[s]) for s in seqs]
            new = [int(min(r, rng.integers(0, 2 * page + 2))) for r in room]
            need = sum(b.plain.pages(b.plain.length[s] + n) - b.plain.pages(b.plain.length[s])
                       for s, n in zip(seqs, new))
            if need <= (b.plain.ref == 0).sum():
                b.grow(seqs, new, kind=str(rng.choice(["f32", "bf16", "f16"])))
        elif what == "fork" and live and idle and (b.plain.ref == 0).sum() > 10:
            src = [int(rng.choice(live)) for _ in range(min(3, len(idle)))]
            dst = [int(x) for x in rng.permutation(idle)[:len(src)]]
            b.plain.fork(src, dst)
            b.cache.fork(dev(src), dev(dst))
        elif what == "free" and live:
            s = [int(x) for x in rng.permutation(live)[:2]]
            for x in s:
                b.plain.free(x)
            b.cache.free(dev(s))
        elif what == "trim" and live:
            s, w, k = int(rng.choice(live)), int(rng.integers(1, 3 * page)), int(rng.integers(0, page + 2))
            b.plain.trim(s, w, k)
            b.cache.trim(dev([s]), w, k)
        elif what == "compact":
            m = b.plain.compact()
            assert int(b.cache.compact()) == m
        b.same()
        whole = [s for s in live if not (b.plain.table[s, :b.plain.pages(b.plain.length[s])] < 0).any()
                 and b.plain.length[s] > 0]
        if what == "attend" and whole:
            b.attend(whole, [int(min(b.plain.length[s], rng.integers(1, 20))) for s in whole], layer=1)


def test_fork_replaces_what_dst_held(P):
    b = Both(P, hkv=1, n_pages=30)
    b.grow([0, 1], [37, 50])
    b.plain.fork([0], [1])
    b.cache.fork(dev([0]), dev([1]))
    b.same()
    b.grow([1, 0], [20, 20])                                     # each in its own copy of the last page
    b.same()
    b.attend([0, 1], [1, 1])


def test_window_with_trimmed_pages(P):
    """Decode under a window: trimmed pages are reused by others and never read."""
    b = Both(P, hq=4, hkv=2, dim=128, page=16, n_pages=24, max_pages=64)
    b.grow([0], [150])
    for step in range(12):
        b.plain.trim(0, 60, 4)
        b.cache.trim(dev([0]), 60, 4)
        b.grow([0, 1], [7, 3])
        b.same()
        b.attend([0, 1], [7, 3], window=60, sinks=4)
    assert (b.plain.table[0, :b.plain.pages(b.plain.length[0])] < 0).any()


def test_copy_pages(P):
    b = Both(P, layers=2, hkv=3, hq=3, n_pages=20)
    b.grow([0], [100])
    for s, d in ((0, 15), (3, 9), (6, 19)):
        b.plain.copy(s, d)
    b.cache.copy_pages(dev([0, 3, 6]), dev([15, 9, 19]))
    b.same()
    b.cache.copy_pages(dev([0, 20, -1]), dev([14, 13, 12]))      # ids outside the pool: skipped, flagged
    b.plain.copy(0, 14)
    b.same(status=P.PI_ERR_DEVICE_CHECK)
    b.same()


def test_pool_and_rows_run_out(P):
    b = Both(P, hkv=1, n_pages=10, max_pages=6)
    b.reserve([0, 1, 2, 3], [16 * 5, 16 * 4, 30, 1])             # 5 + 4 + (2, one left) + (1, after a failure)
    assert b.plain.oom and list(b.plain.length[:4]) == [80, 64, 0, 0]
    b.same(status=P.PI_ERR_OOM)
    b.plain.oom = False
    b.reserve([0, 4], [16 * 2, 8])                               # row 0 is too short; sequence 4 still gets its page
    assert list(b.plain.length[:5]) == [80, 64, 0, 0, 8]
    b.same(status=P.PI_ERR_OOM)
    b.plain.fork([4], [5])                                       # no page for the copy
    b.cache.fork(dev([4]), dev([5]))
    assert b.plain.length[5] == 0
    b.same(status=P.PI_ERR_OOM)
    b.plain.fork([0], [5])                                       # needs none
    b.cache.fork(dev([0]), dev([5]))
    b.same()


def test_large_pool_and_compaction(P):
    """More pages than one pass of the scan covers; shared pages move once."""
    b = Both(P, hq=1, hkv=1, dim=64, page=16, n_pages=20000, max_seqs=40, max_pages=600)
    b.reserve(list(range(30)), [16 * 590 + i for i in range(30)])
    for s in range(0, 30, 2):
        b.plain.free(s)
    b.cache.free(dev(list(range(0, 30, 2))))
    b.plain.fork([1, 3], [30, 31])
    b.cache.fork(dev([1, 3]), dev([30, 31]))
    b.same()
    assert int(b.cache.compact()) == b.plain.compact()
    b.same()


# ------------------------------------------------------------------------------------------------ refusals, flags

def test_refusals(P):
    b = Both(P, hq=4, hkv=2, dim=64, page=16)
    seqs, start = b.args([0], [1])
    q, k = torch.zeros(1, 4, 64, device="cuda"), torch.zeros(1, 2, 64, device="cuda")
    h = b.cache.h

    def refused(call, code=1):
        with pytest.raises(P.PiError) as e:
            call()
        assert e.value.code == code
    good = dict(layer=0, seqs=seqs, tok_start=start, n=1, n_tokens=1, q=q, ld_q=256, out=q, ld_out=256, lse=None,
                dtype=P.PI_F32, scale=0.1, window=0, sinks=0)
    P.pi_kv_attend(h, **good)
    for bad in (dict(layer=1), dict(layer=-1), dict(n=-1), dict(n=1025), dict(n_tokens=-1), dict(ld_q=255),
                dict(ld_q=258), dict(ld_out=128), dict(dtype=3), dict(dtype=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(sinks=-1), dict(q=None), dict(out=None), dict(seqs=None),
                dict(tok_start=None), dict(q=q.cpu()), dict(q=q.data_ptr() + 4), dict(lse=8)):
        refused(lambda: P.pi_kv_attend(h, **{**good, **bad}))
    refused(lambda: P.pi_kv_append(h, 0, seqs, start, 1, 1, k, k.cpu(), 128, P.PI_F32))
    refused(lambda: P.pi_kv_append(h, 0, seqs, start, 1, 1, k, k, 127, P.PI_F32))
    refused(lambda: P.pi_kv_append(h, 2, seqs, start, 1, 1, k, k, 128, P.PI_F32))
    refused(lambda: P.pi_kv_trim(h, seqs, 1, 0, 0))
    refused(lambda: P.pi_kv_trim(h, seqs, 1, 1, -1))
    refused(lambda: P.pi_kv_copy_pages(h, seqs, seqs, 65))
    refused(lambda: P.pi_kv_fork(h, seqs, None, 1))
    refused(lambda: P.pi_kv_compact(h, torch.zeros(1, dtype=torch.int32)))
    P.pi_kv_attend(h, **{**good, "n": 0})                        # nothing to do
    P.pi_kv_reserve(h, None, None, 0)
    for call in (lambda: b.cache.attend(0, seqs.long(), start, q), lambda: b.cache.attend(0, seqs, seqs, q),
                 lambda: b.cache.attend(0, seqs, start, q[:, :3]), lambda: b.cache.append(0, seqs, start, k, k.half()),
                 lambda: b.cache.attend(0, seqs, start, torch.zeros(1, 64, 4, device="cuda").transpose(1, 2))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(P.PiError):
        b.cache.attend(0, seqs, start, q.double())
    b.same()


def test_device_flags(P):
    """Bad entries on the device are skipped and reported; what is around them is done."""
    b = Both(P, hq=2, hkv=1, n_pages=20)
    b.grow([0, 1], [20, 33])
    flag = P.PI_ERR_DEVICE_CHECK
    q = torch.randn(2, 2, 64, device="cuda")
    want = b.cache.attend(0, dev([0, 1]), dev([0, 1, 2]), q)
    assert b.cache.status() == 0
    got = b.cache.attend(0, dev([0, 99, -1, 1]), dev([0, 1, 1, 1, 2]), q)
    assert torch.equal(got, want) and b.cache.status() == flag and b.cache.status() == 0
    got = torch.full_like(q, 5.0)
    b.cache.attend(0, dev([0, 1]), dev([0, 1, 3]), q, out=got)   # rows past the arrays
    assert torch.equal(got[0], want[0]) and (got[1] == 5).all() and b.cache.status() == flag
    b.cache.reserve(dev([0, 8]), dev([0, 0, 4]))
    assert b.cache.status() == flag
    b.cache.free(dev([77]))
    assert b.cache.status() == flag
    b.cache.fork(dev([0]), dev([0]))
    assert b.cache.status() == flag
    b.cache.append(0, dev([5]), dev([0, 1]), q[:1, :1], q[:1, :1])   # no room was reserved
    assert b.cache.status() == flag
    b.same()
    keep = b.cache.table.clone()
    b.cache.table[1, 1] = -1                                     # a page in view is gone: left out, flagged
    b.plain.table[1, 1] = -1
    got = b.cache.attend(0, dev([1]), dev([0, 1]), q[:1], scale=0.125)
    assert b.cache.status() == flag
    exact, _ = b.plain.attend(0, [1], [1], q[:1].double().cpu().numpy(), 0.125)
    assert np.linalg.norm(got.cpu().numpy() - exact) <= TOL["f32"] * np.linalg.norm(exact)
    b.cache.table[1, 1] = 20                                     # not a page of the pool
    again = b.cache.attend(0, dev([1]), dev([0, 1]), q[:1], scale=0.125)
    assert torch.equal(again, got) and b.cache.status() == flag
    b.cache.table.copy_(keep)


@pytest.mark.parametrize("fault,code", [("alloc", 4), ("upload", 3), ("badarg", 1)])
def test_create_failure_paths(P, fault, code, monkeypatch):
    torch.cuda.synchronize()
    b = Both(P)
    args = (b.cache.layers, b.cache.table, b.cache.length, b.cache.ref)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    monkeypatch.setenv("PI_FAULT", fault)
    with pytest.raises(P.PiError) as e:
        P.KVCache(*args, n_heads=4)
    monkeypatch.delenv("PI_FAULT")
    assert e.value.code == code and torch.cuda.mem_get_info()[0] == free
    c = P.KVCache(*args, n_heads=4)
    c.close()
    c.close()


# ------------------------------------------------------------------------------------------------ streams, graphs

def test_other_stream_and_graph(P):
    """A step on a stream of its own, and the same step captured in a graph and replayed."""
    b = Both(P, layers=2, hq=4, hkv=2, dim=128, page=16, n_pages=64, max_pages=32)
    b.grow([0, 1], [37, 100])
    seqs, start = b.args([0, 1], [1, 1])
    q = torch.randn(2, 4, 128, device="cuda")
    kv = torch.randn(2, 2, 128, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(q) for _ in range(2)]

    def step(stream=None):
        b.cache.reserve(seqs, start, stream=stream)
        for layer in range(2):
            b.cache.append(layer, seqs, start, kv, kv, stream=stream)
            b.cache.attend(layer, seqs, start, q, out=out[layer], stream=stream)

    def plain_step():
        b.plain.reserve([0, 1], [1, 1])
        n = kv.double().cpu().numpy()
        for layer in range(2):
            b.plain.append(layer, [0, 1], [1, 1], n, n)
    step(side)
    side.synchronize()
    plain_step()
    b.same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for _ in range(20):                                          # over a page's end
        g.replay()
        plain_step()
    torch.cuda.synchronize()
    b.same()
    for layer in range(2):
        want, _ = b.plain.attend(layer, [0, 1], [1, 1], q.double().cpu().numpy(), 128 ** -0.5)
        got = out[layer].double().cpu().numpy()
        assert np.linalg.norm(got - want) <= TOL["f32"] * np.linalg.norm(want)


def test_a_cache_made_by_a_thread_without_a_context(P):
    """A handle is made and used by host threads whose first CUDA call that is."""
    import threading

    b = Both(P)
    b.grow([0], [20])
    torch.cuda.synchronize()
    made = []
    layers = [dict(k=b.k[0], v=b.v[0], k_scale=b.ks[0], v_scale=b.vs[0])]
    seqs, start = b.args([0], [1])

    def make():
        made.append(P.KVCache(layers, b.cache.table, b.cache.length, b.cache.ref, n_heads=4))

    def reserve():
        P.pi_kv_reserve(made[0].h, seqs, start, 1, 0)

    for work in (make, reserve):
        t = threading.Thread(target=work)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert made[0].length[0] == 21 and made[0].status() == 0
