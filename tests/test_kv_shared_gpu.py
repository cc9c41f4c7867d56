"""Attention over shared prefixes on the GPU against the plain cache's attention in fp64, which knows nothing of them.

Bound of an element's error: half a step of its type, and of A = sum_j p_j |v_j|: 2^-11 for weights held as one f16 term
(half a step of f16; 16-bit types) or 2^-22 for two (fp32); 1e-5 for the exponential and for fp32 sums of some hundred
terms (joining two partial sums adds three roundings of 2^-24); and twice what a logit is off by: with L >= scale sum_d
|q_d k_jd|, 22-bit queries 2^-22 L, and a sum that the tensor cores cut off to 24 bits in at most 10 steps of 16 (the
other term's, the scales'), 10 * 2^-23 L.
"""
import numpy as np
import pytest
import torch

from tests.kv_plain import TABLE
from tests.test_kv_gpu import TYPES, Both, dev
from tests.test_proj_gpu import HALF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import activation_sparse_decode_pi_gb300 as P

    return P


class Shared(Both):
    def fork(self, src, dst):
        self.plain.fork(src, dst)
        self.cache.fork(dev(src), dev(dst))

    def prefix(self, seqs, new, groups):
        """What each group shares, from the plain table."""
        p, out = self.plain, []
        for a, b in zip(groups, groups[1:]):
            live = [(s, n) for s, n in zip(seqs[a:b], new[a:b]) if n]
            cols = min((int(p.length[s]) - n) // p.page for s, n in live) if len(live) > 1 else 0
            room = min((int(p.length[s]) - n) for s, n in live) if live else 0
            c = 0
            while c < cols and p.table[live[0][0], c] >= 0 and len({int(p.table[s, c]) for s, _ in live}) == 1:
                c += 1
            out.append(min(c * p.page, room) // 128 * 128)
        return out

    def key_norms(self, seqs, new):
        """For each row and query head the largest norm of its sequence's keys: [rows, heads, 1]."""
        p, out = self.plain, []
        for s, n in zip(seqs, new):
            j = np.arange(int(p.length[s]))
            page = p.table[s, j // p.page]
            k = TABLE[p.k[0, page, :, j % p.page]] * p.ks[0, page][..., None]          # [keys, kv heads, dim]
            top = np.linalg.norm(k, axis=-1).max(0, initial=0.0)
            out += [np.repeat(top, p.hq // p.hkv)[:, None]] * n
        return np.array(out)

    def check(self, seqs, new, groups, kind="f32", want_shared=None, fused=0, scale=None, sharp=1.0, plan=None):
        p = self.plain
        shared = self.prefix(seqs, new, groups)
        if want_shared is not None:
            assert shared == want_shared
        args = self.args(seqs, new)
        plan = self.cache.share(*args, dev(groups)) if plan is None else plan
        g = len(groups) - 1
        got = plan.cpu().numpy()
        assert got[2 * g + 1:3 * g + 1].tolist() == shared
        skip = np.zeros(len(seqs), int)
        for a, b, s in zip(groups, groups[1:], shared):
            skip[a:b] = [s if n else 0 for n in new[a:b]]
        assert got[3 * g + 1:3 * g + 1 + len(seqs)].tolist() == skip.tolist()
        q, _ = self.tokens(new, kind, p.hq, fused, spread=0)
        q *= sharp
        qn = q.double().cpu().numpy()
        scale = p.dim ** -0.5 if scale is None else scale
        lse = torch.full(q.shape[:2], 123.0, device="cuda")
        work = torch.full((q.shape[0] * p.hq * (p.dim + 2),), float("nan"), device="cuda")
        out = self.cache.attend_shared(0, *args, plan, q, lse=lse, scale=scale, work=work)
        want, want_lse = p.attend(0, seqs, new, qn, scale)
        out_n, lse_n = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert out.dtype is TYPES[kind] and self.cache.status() == 0
        assert np.isfinite(out_n).all() and np.allclose(lse_n, want_lse, rtol=1e-5, atol=2e-5)
        signed, p.v = p.v, p.v & 0x7f
        size, _ = p.attend(0, seqs, new, qn, scale)                             # sum_j p_j |v_j|
        p.v = signed
        largest = scale * np.linalg.norm(qn, axis=-1, keepdims=True) * self.key_norms(seqs, new)
        tol = HALF[kind] * np.abs(want) + size * (1e-5 + 2 * 12 * 2.0 ** -23 * largest + (2.0 ** -22 if kind == "f32" else 2.0 ** -11))
        ratio = np.abs(out_n - want) / tol
        assert ratio.max() <= 1, (np.argwhere(ratio > 1)[:5], ratio.max())
        return out, plan


SHAPES = [
    dict(hq=2, hkv=2, dim=64, page=16),
    dict(hq=8, hkv=2, dim=128, page=64),
    dict(hq=15, hkv=3, dim=128, page=32),
    dict(hq=16, hkv=1, dim=64, page=128),
    dict(hq=4, hkv=2, dim=256, page=64),
    dict(hq=40, hkv=1, dim=128, page=16),
]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s['hq']}of{s['hkv']}x{s['dim']}p{s['page']}")
def test_forks_of_one_prompt(P, shape, kind):
    page = shape["page"]
    b = Shared(P, n_pages=-(-1500 // page) + 40, max_seqs=12, max_pages=-(-1100 // page), **shape)
    b.grow([0], [700])
    b.fork([0, 0, 0, 0, 0], [3, 1, 7, 5, 9])
    b.grow([3, 1, 0, 7, 5, 9], [1, 2, 1, 1, 90, 1])
    seqs, new = [3, 1, 0, 7, 5, 9], [1] * 6
    whole = min(700 // page * page, 700) // 128 * 128
    b.check(seqs, new, [0, 6], kind, [whole])
    b.check(seqs, new, [0, 6], kind, fused=64, sharp=8.0)
    b.check([5, 9, 1], [1, 1, 1], [0, 1, 3], kind, [0, whole])                  # a group of one shares nothing
    b.check([7, 3], [1, 1], [0, 2], kind)
    b.check([0, 5, 3], [1, 80, 1], [0, 3], kind)                               # many rows of one sequence behind it
    b.check([1, 3, 0], [2, 1, 0], [0, 3], kind)                                # no new token for one


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_groups_of_different_prompts(P, kind):
    b = Shared(P, hq=8, hkv=2, dim=128, page=32, n_pages=220, max_seqs=20, max_pages=60)
    b.grow([0, 1, 2, 3], [1000, 130, 100, 515])
    b.fork([0, 0, 0, 1, 1, 2, 3, 3], [4, 5, 6, 7, 8, 9, 10, 11])
    seqs = [0, 4, 5, 6, 1, 7, 8, 2, 9, 3, 10, 11, 15]
    b.grow(seqs, [3, 1, 40, 200, 2, 1, 1, 5, 5, 1, 1, 300, 77])
    groups = [0, 4, 7, 9, 12]                                                   # the last sequence is in no group
    b.check(seqs, [1] * 13, groups, kind, [896, 128, 0, 512])
    b.check(seqs, [3, 1, 1, 2, 1, 1, 1, 5, 1, 1, 0, 260, 77], groups, kind, [896, 128, 0, 512])
    b.check(seqs[4:], [1] * 9, [1, 1, 3, 3, 5, 8], kind, [0, 128, 0, 0, 512])   # empty groups, a first one left out
    b.check(seqs, [1] * 13, [0], kind, [])                                     # no groups at all
    b.check([0, 4, 1], [1] * 3, [0, 3], kind, [0])                              # nothing in common
    b.check([5, 5, 4, 5], [1, 4, 1, 1], [0, 4], kind, [896])                    # one sequence thrice


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_groups_of_some_dozen_rows(P, dim, page, kind):
    """Prefixes that fill a part of a 128-row tile, all of one, and more than one beside a smaller group."""
    b = Shared(P, hq=8, hkv=2, dim=dim, page=page, n_pages=-(-3000 // page) + 150, max_seqs=60, max_pages=-(-1300 // page))
    b.grow([0, 1], [1100, 530])
    first, second = list(range(2, 40)), list(range(40, 48))
    b.fork([0] * len(first), first)
    b.fork([1] * len(second), second)
    one, two = [0] + first, [1] + second
    b.grow(one + two, [1 + i % 4 for i in range(len(one) + len(two))])
    b.check(one[:9], [1] * 9, [0, 9], kind, [1024])                             # 36 rows, split along the prefix
    b.check(one[:32], [1] * 32, [0, 32], kind, [1024])                          # 128
    b.check(one + two, [1] * 48, [0, 39, 48], kind, [1024, 512])                # 156 and 36
    b.check(two + one[:12], [1] * 21, [0, 9, 21], kind, [512, 1024])
    b.check(one[:3] + two, [1] * 12, [0, 3, 12], kind, [1024, 512])             # 12 rows beside 36


def test_long_prefix_is_split(P):
    b = Shared(P, hq=16, hkv=2, dim=128, page=64, n_pages=500, max_seqs=70, max_pages=360)
    b.grow([0], [20000])
    others = list(range(1, 70))
    b.fork([0] * 40, others[:40])
    seqs = [0] + others[:40]
    b.grow(seqs, [1 + 7 * i % 50 for i in range(41)])
    b.check(seqs, [1] * 41, [0, 41], "bf16", [19968])
    b.check(seqs, [1] * 41, [0, 41], "f32")
    b.check(seqs[:3], [1] * 3, [0, 3], "f32")                                   # few rows over the whole prefix


def test_the_same_plan_over_steps_and_compaction(P):
    """A plan outlives steps that only grow, and pages that move with their table rows."""
    b = Shared(P, hq=4, hkv=2, dim=64, page=16, n_pages=120, max_seqs=8, max_pages=40)
    b.grow([6], [200])                                                          # pages below, given back later
    b.grow([0], [300])
    b.fork([0, 0], [1, 2])
    seqs, new = [0, 1, 2], [1, 1, 1]
    b.grow(seqs, new)
    _, plan = b.check(seqs, new, [0, 3], "bf16", [256])
    for i in range(20):
        b.grow(seqs, new)
        if i == 8:
            b.plain.free(6)
            b.cache.free(dev([6]))
            assert int(b.cache.compact()) == b.plain.compact()
            b.same()
        b.check(seqs, new, [0, 3], "bf16", [256], plan=plan)


def test_same_bits_each_time_on_another_stream_and_in_a_graph(P):
    b = Shared(P, hq=16, hkv=2, dim=128, page=64, n_pages=200, max_seqs=20, max_pages=80)
    b.grow([0], [4000])
    b.fork([0] * 9, list(range(1, 10)))
    seqs, new = list(range(10)), [1] * 10
    b.grow(seqs, [1 + i for i in range(10)])
    first, plan = b.check(seqs, new, [0, 4, 10], "bf16")
    args = b.args(seqs, new)
    q, _ = b.tokens(new, "bf16", 16)
    first = b.cache.attend_shared(0, *args, plan, q)
    for _ in range(20):
        assert torch.equal(b.cache.attend_shared(0, *args, plan, q), first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = b.cache.attend_shared(0, *args, b.cache.share(*args, dev([0, 4, 10]), stream=stream), q, stream=stream)
        s.synchronize()
        assert torch.equal(got, first)
    out, groups = torch.zeros_like(q), dev([0, 4, 10])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graphs = []
        for _ in range(2):                                                      # two graphs, each with a work of its own
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                b.cache.attend_shared(0, *args, b.cache.share(*args, groups), q, out=out)
            graphs.append(g)
    for g in graphs:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert b.cache.status() == 0


def test_rows_past_the_last_sequence_and_strided_outputs(P):
    b = Shared(P, hq=4, hkv=2, dim=128, page=32, n_pages=40, max_pages=20)
    b.grow([0], [300])
    b.fork([0], [1])
    b.grow([0, 1], [2, 3])
    args = b.args([0, 1], [2, 3])
    plan = b.cache.share(*args, dev([0, 2]))
    q = torch.randn(8, 4, 128, device="cuda")
    wide = torch.full((8, 4 * 128 + 32), 7.0, device="cuda")
    lse = torch.full((8, 4), 7.0, device="cuda")
    b.cache.attend_shared(0, *args, plan, q, out=wide[:, :512].unflatten(1, (4, 128)), lse=lse)
    want = b.cache.attend(0, *args, q[:5].contiguous())
    assert (wide[5:] == 7).all() and (wide[:, 512:] == 7).all() and (lse[5:] == 7).all()
    # (both within 1.1e-5 of A, and the values here are below 24)
    assert torch.allclose(wide[:5, :512].unflatten(1, (4, 128)), want, rtol=0, atol=2.2e-5 * 24)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
def test_queries_before_the_first_position(P, dim, page):
    """More new tokens than positions, beside a group that shares: what sees nothing gives 0 and -infinity."""
    b = Shared(P, hq=4, hkv=2, dim=dim, page=page, n_pages=60, max_pages=20)
    b.grow([0, 3], [300, 2])
    b.fork([0], [1])
    b.grow([0, 1], [3, 2])
    seqs, new = [0, 1, 3, 5], [1, 2, 5, 3]                                      # 3 of sequence 3's, all of 5's see nothing
    args = b.args(seqs, new)
    q, qn = b.tokens(new, "f32", 4, spread=0)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    out = b.cache.attend_shared(0, *args, b.cache.share(*args, dev([0, 2])), q, lse=lse, scale=0.1)
    want, want_lse = b.plain.attend(0, seqs, new, qn, 0.1)
    nothing = np.isneginf(want_lse)
    assert nothing.sum() == 6 * 4 and np.array_equal(np.isneginf(lse.cpu().numpy()), nothing)
    assert not out.cpu().numpy()[nothing].any() and b.cache.status() == 0
    assert np.allclose(out.double().cpu().numpy(), want, rtol=0, atol=1.1e-5 * 24)     # (A is below 24 here)


def test_one_long_sequence_among_short_ones(P):
    """Shares that cut an item over many CTAs, with and without a prefix."""
    b = Shared(P, hq=8, hkv=2, dim=128, page=32, n_pages=500, max_seqs=12, max_pages=400)
    b.grow([0], [260])
    b.fork([0] * 5, [1, 2, 3, 4, 5])
    b.grow([0, 1, 2, 3, 4, 5, 7], [3, 9000, 70, 1, 200, 64, 2500])
    for kind in ("f32", "bf16"):
        b.check([0, 1, 2, 3, 4, 5, 7], [1, 1, 1, 1, 3, 1, 2], [0, 6], kind, [256])


def test_1024_sequences_in_256_groups(P):
    b = Shared(P, hq=2, hkv=1, dim=64, page=16, n_pages=4200, max_seqs=1024, max_pages=20)
    lead = list(range(0, 1024, 4))
    b.cache.reserve(*b.args(lead, [150] * 256))
    k, v = (torch.randn((150 * 256, 1, 64), device="cuda") for _ in range(2))
    b.cache.append(0, *b.args(lead, [150] * 256), k, v)
    b.cache.fork(dev(np.repeat(lead, 3)), dev([s + i for s in lead for i in (1, 2, 3)]))
    seqs, new = list(range(1024)), [1 + i % 3 for i in range(1024)]
    args = b.args(seqs, new)
    b.cache.reserve(*args)
    k, v = (torch.randn((sum(new), 1, 64), device="cuda") for _ in range(2))
    b.cache.append(0, *args, k, v)
    plan = b.cache.share(*args, dev(range(0, 1025, 4)))
    assert (plan[2 * 256 + 1:3 * 256 + 1] == 128).all()
    for kind in ("f32", "bf16"):
        q, _ = b.tokens(new, kind, 2, spread=0)
        got, want = b.cache.attend_shared(0, *args, plan, q), b.cache.attend(0, *args, q)
        # (values are below 6: A <= 6; one rounding and one-term weights each for 16-bit types)
        tol = 6 * 2.2e-5 if kind == "f32" else 6 * (2 * HALF[kind] + 2 * 2.0 ** -11 + 2.2e-5)
        assert torch.allclose(got.float(), want.float(), rtol=0, atol=tol) and b.cache.status() == 0


def test_output_in_the_queries_place(P):
    b = Shared(P, hq=16, hkv=2, dim=128, page=64, n_pages=120, max_seqs=8, max_pages=60)
    b.grow([0], [2500])
    b.fork([0] * 5, [1, 2, 3, 4, 5])
    b.grow([0, 1, 2, 3, 4, 5], [1, 30, 900, 2, 1, 64])
    args = b.args(range(6), [1, 1, 2, 1, 1, 40])
    plan = b.cache.share(*args, dev([0, 6]))
    q, _ = b.tokens([46], "bf16", 16)
    want = b.cache.attend_shared(0, *args, plan, q)
    assert torch.equal(b.cache.attend_shared(0, *args, plan, q, out=q), want) and b.cache.status() == 0


def test_pools_past_32_bits(P):
    """Prefix and what lies behind it at the end of pools of more than 2^32 bytes."""
    dim, page, hkv, n_pages = 128, 64, 2, 270000
    k, v = (torch.zeros((n_pages, hkv, page, dim), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones((n_pages, hkv), device="cuda") for _ in range(2))
    ids = torch.arange(n_pages - 1, n_pages - 31, -1, dtype=torch.int32, device="cuda")
    table = torch.stack([torch.cat([ids[:10], ids[10 + 4 * i:14 + 4 * i]]) for i in range(5)])
    ref = torch.bincount(table.flatten().long(), minlength=n_pages).to(torch.int32)
    length = dev([890, 650, 700, 641, 895])
    for pool in (k, v):
        pool.view(torch.uint8)[ids.long()] = torch.randint(0, 0x60, (30, hkv, page, dim), device="cuda", dtype=torch.uint8)
    ks[ids.long()] = vs[ids.long()] = 1 / 16
    big = P.KVCache([dict(k=k, v=v, k_scale=ks, v_scale=vs)], table, length, ref, n_heads=8)
    take = lambda x: x[ids.long()].contiguous()  # noqa: E731
    small = P.KVCache([dict(k=take(k.view(torch.uint8)).view(torch.float8_e4m3fn), v=take(v.view(torch.uint8)).view(torch.float8_e4m3fn),
                            k_scale=take(ks), v_scale=take(vs))], (n_pages - 1 - table).to(torch.int32).contiguous(), length.clone(),
                      ref[ids.long()].contiguous(), n_heads=8)
    seqs, start, groups = dev(range(5)), dev(range(6)), dev([0, 5])
    for kind in ("bf16", "f32"):
        q = torch.randn((5, 8, dim), device="cuda").to(TYPES[kind])
        outs = [c.attend_shared(0, seqs, start, c.share(seqs, start, groups), q) for c in (big, small)]
        assert torch.equal(*outs) and torch.isfinite(outs[0]).all()
    assert big.status() == 0 and small.status() == 0


@pytest.mark.parametrize("rows", [1, 40])
def test_nan_in_the_prefix_reaches_all_and_behind_it_one(P, rows):
    b = Shared(P, hq=2, hkv=1, dim=64, page=16, n_pages=80, max_pages=40)
    b.grow([0], [260])
    b.fork([0, 0], [1, 2])
    new = [rows, rows, rows]
    b.grow([0, 1, 2], new)
    args = b.args([0, 1, 2], new)
    plan = b.cache.share(*args, dev([0, 3]))
    q, _ = b.tokens(new, "f32", 2)
    clean = b.cache.attend_shared(0, *args, plan, q)
    own = int(b.cache.table[1, 262 // 16])                                      # a page behind the prefix, of sequence 1
    codes = b.v.view(torch.uint8)
    was = codes[0, own, 0, 260 % 16, 7].clone()
    codes[0, own, 0, 260 % 16, 7] = 0x7f
    got = b.cache.attend_shared(0, *args, plan, q)
    bad = torch.isnan(got)
    assert bad[rows:2 * rows, :, 7].all() and bad.sum() == 2 * rows and torch.equal(got[~bad], clean[~bad])
    codes[0, own, 0, 260 % 16, 7] = was
    codes[0, int(b.cache.table[0, 3]), 0, 5, 9] = 0x7f                          # position 53 of all three
    bad = torch.isnan(b.cache.attend_shared(0, *args, plan, q))
    assert bad[:, :, 9].all() and bad.sum() == 6 * rows
    assert b.cache.status() == 0


def test_a_plan_of_another_batch_is_flagged(P):
    b = Shared(P, hq=4, hkv=2, dim=64, page=16, n_pages=80, max_pages=30)
    b.grow([0], [300])
    b.fork([0, 0], [1, 2])
    b.grow([0, 1, 2], [4, 4, 4])
    args = b.args([0, 1, 2], [1, 1, 1])
    plan = b.cache.share(*args, dev([0, 3]))
    q = torch.randn(6, 4, 64, device="cuda")
    out = torch.full_like(q, 7.0)
    b.cache.attend_shared(0, *b.args([0, 1, 2], [1, 2, 1]), plan, q, out=out)    # other rows from the second sequence on
    assert b.cache.status() == P.PI_ERR_DEVICE_CHECK
    assert (out[1:] == 7).all() and not (out[0] == 7).any()
    out.fill_(7.0)
    b.cache.attend_shared(0, *b.args([0, 2, 1], [1, 1, 1]), plan, q, out=out)    # other sequences
    assert b.cache.status() == P.PI_ERR_DEVICE_CHECK and (out[1:] == 7).all()
    b.cache.free(dev([1]))                                                      # shorter than the prefix now
    out.fill_(7.0)
    b.cache.attend_shared(0, *args, plan, q, out=out)
    assert b.cache.status() == P.PI_ERR_DEVICE_CHECK and (out[1] == 7).all() and not (out[2] == 7).any()


@pytest.mark.parametrize("groups", [[0, 3, 1, 4], [0, 5], [-1, 2], [2, 1]])
def test_groups_out_of_order_share_nothing(P, groups):
    b = Shared(P, hq=2, hkv=1, dim=64, page=16, n_pages=80, max_pages=30)
    b.grow([0], [300])
    b.fork([0, 0, 0], [1, 2, 3])
    b.grow([0, 1, 2, 3], [1, 1, 1, 1])
    args = b.args([0, 1, 2, 3], [1] * 4)
    plan = b.cache.share(*args, dev(groups))
    assert b.cache.status() == P.PI_ERR_DEVICE_CHECK
    n = len(groups) - 1
    assert (plan[2 * n + 1:3 * n + 5] == 0).all()
    q = torch.randn(4, 2, 64, device="cuda")
    got, want = b.cache.attend_shared(0, *args, plan, q), b.cache.attend(0, *args, q)
    assert torch.allclose(got, want, rtol=0, atol=2.2e-5 * 24) and b.cache.status() == 0     # (as above)


def test_refusals(P):
    b = Shared(P, hq=4, hkv=2, dim=64, page=16, n_pages=40, max_pages=30)
    b.grow([0], [300])
    b.fork([0], [1])
    b.grow([0, 1], [1, 1])
    args, q = b.args([0, 1], [1, 1]), torch.randn(2, 4, 64, device="cuda")
    with pytest.raises(P.PiError):
        b.cache.share(*args, dev([0, 1, 2, 2]))                                 # more groups than sequences
    for bad in (dev([0, 2]).long(), dev([0, 2]).cpu(), dev([[0, 2]])):
        with pytest.raises(ValueError):
            b.cache.share(*args, bad)
    plan = b.cache.share(*args, dev([0, 2]))
    for bad in (plan[:-1], plan[:6], plan.long(), plan.cpu(), plan.view(1, -1)):
        with pytest.raises(ValueError):
            b.cache.attend_shared(0, *args, bad, q)
    for kw in (dict(work=torch.empty(100, device="cuda")), dict(work=torch.empty(2 * 4 * 66, device="cuda").half()),
               dict(out=torch.empty(3, 4, 64, device="cuda")), dict(lse=torch.empty(2, 3, device="cuda"))):
        with pytest.raises(ValueError):
            b.cache.attend_shared(0, *args, plan, q, **kw)
    room = torch.zeros(2 * 4 * 66, device="cuda")                               # work over the queries
    for call in (lambda: b.cache.attend_shared(1, *args, plan, q), lambda: b.cache.attend_shared(0, *args, plan, q.double()),
                 lambda: b.cache.attend_shared(0, *args, plan, q, scale=float("nan")),
                 lambda: b.cache.attend_shared(0, *args, plan, q, work=torch.empty(2 * 4 * 66 + 1, device="cuda")[1:]),
                 lambda: b.cache.attend_shared(0, *args, plan, room[:512].view(2, 4, 64), work=room)):
        with pytest.raises(P.PiError):
            call()
    none = dev([])
    empty = b.cache.share(none, dev([0]), dev([0]))
    assert b.cache.attend_shared(0, none, dev([0]), empty, q[:0]).shape == (0, 4, 64)
    assert b.cache.status() == 0


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_weights_of_16_bit_types_keep_two_terms(P, dim, page, kind):
    """Outputs are the rounding of what fp32 would give: they lie between the roundings of both ends of its bound (the head
    of this file, with two terms). One value of each sequence's own and one of the prefix make a column, so that the
    roundings of weights do not average out."""
    b = Shared(P, hq=8, hkv=2, dim=dim, page=page, n_pages=-(-6000 // page), max_seqs=44, max_pages=-(-800 // page))
    p = b.plain
    b.grow([0], [700])
    b.fork([0] * 40, range(1, 41))
    b.grow(range(41), [40 if i == 3 else 1 + i % 3 for i in range(41)])
    p.v[:] = 0
    for seq in range(41):
        for at, columns in ((77, slice(0, None, 2)), (700, slice(1, None, 2))):
            codes = p.v[0, p.table[seq, at // page], :, at % page]
            if not codes[:, columns].any():
                codes[:, columns] = b.rng.integers(0x20, 0x7e, codes[:, columns].shape)
    b.v.view(torch.uint8).copy_(torch.tensor(p.v, device="cuda"))
    # rows to a group and behind it: few; 36; 128; 160; many new tokens of one sequence
    for seqs, new in ((range(3), [1] * 3), (range(9), [1] * 9), (range(32), [1] * 32), (range(40), [1] * 40),
                      ([0, 40, 3], [1, 1, 40])):
        args = b.args(seqs, new)
        plan = b.cache.share(*args, dev([0, len(new)]))
        assert (plan[3:4 + len(new)] == 640).all()
        q, qn = b.tokens(new, kind, p.hq, spread=0)
        scale = 1 / 64
        out = b.cache.attend_shared(0, *args, plan, q, scale=scale)
        want, _ = p.attend(0, seqs, new, qn, scale)
        signed, p.v = p.v, p.v & 0x7f
        size, _ = p.attend(0, seqs, new, qn, scale)
        p.v = signed
        largest = scale * np.linalg.norm(qn, axis=-1, keepdims=True) * b.key_norms(seqs, new)
        off = size * (1e-5 + 2 * 12 * 2.0 ** -23 * largest + 2.0 ** -22)
        lo, hi = (torch.tensor(want + x, device="cuda").to(TYPES[kind]) for x in (-off, off))
        beyond = (out < lo) | (out > hi)
        assert not beyond.any() and b.cache.status() == 0, (len(new), int(beyond.sum()), beyond.numel())


def test_refuses_outputs_over_what_the_call_reads(P):
    """work, out, lse and plan over other arrays of their call; beside them they are taken."""
    b = Shared(P, hq=4, hkv=2, dim=64, page=16, n_pages=60, max_pages=30)
    b.grow([0], [300])
    b.fork([0], [1])
    b.grow([0, 1], [1, 1])
    seqs, start = b.args([0, 1], [1, 1])
    groups = dev([0, 2])
    plan = b.cache.share(seqs, start, groups)
    room = torch.zeros(4096, device="cuda")
    q, need = torch.randn(2, 4, 64, device="cuda"), 2 * 4 * 66

    def at(x, first):                                                # a copy of x in the room
        y = room[first:first + x.numel()].view(x.dtype)
        return y.copy_(x.flatten()).view(x.shape)

    def attend(first, *, seqs=seqs, start=start, plan=plan, q=q, out=None, lse=None):
        room[:need].zero_()
        return b.cache.attend_shared(0, seqs, start, plan, q, out=out, lse=lse, work=room[:need])

    lse = torch.zeros(2, 4, device="cuda")
    for first, fine in ((need - 4, False), (need, True)):
        for name, x in (("plan", plan), ("seqs", seqs), ("start", start), ("q", q), ("out", q), ("lse", lse)):
            if fine:
                assert torch.isfinite(attend(first, **{name: at(x, first)})).all()
            else:
                with pytest.raises(P.PiError):
                    attend(first, **{name: at(x, first)})
    out = room[:512].view(2, 4, 64)
    for first, fine in ((508, False), (512, True)):
        for name, x in (("plan", plan), ("seqs", seqs), ("tok_start", start), ("lse", lse), ("q", q)):
            args = dict(seqs=seqs, tok_start=start, plan=plan, q=q, lse=None)
            args[name] = at(x, first)
            if fine:
                b.cache.attend_shared(0, out=out, **args)
            else:
                with pytest.raises(P.PiError):
                    b.cache.attend_shared(0, out=out, **args)
    for name, x in (("plan", plan), ("seqs", seqs), ("tok_start", start), ("q", q)):      # the sums' logarithms likewise
        args = dict(seqs=seqs, tok_start=start, plan=plan, q=q)
        args[name] = at(x, 4)
        with pytest.raises(P.PiError):
            b.cache.attend_shared(0, lse=room[:8].view(2, 4), **args)
    pool = b.v.view(torch.float32).flatten()
    with pytest.raises(P.PiError):
        b.cache.attend_shared(0, seqs, start, plan, q, out=pool[:512].view(2, 4, 64))
    with pytest.raises(P.PiError):
        b.cache.attend_shared(0, seqs, start, plan, q, work=pool[:need])
    words = torch.zeros(40, dtype=torch.int32, device="cuda")
    size = plan.numel()
    for i, x in enumerate((seqs, start, groups)):                    # the plan over what it is made from
        for first, code in ((size - 1, 1), (size, 0)):
            args = [seqs, start, groups]
            args[i] = words[first:first + x.numel()].copy_(x)
            assert P._lib.pi_kv_share(b.cache.h, args[0].data_ptr(), args[1].data_ptr(), 2, args[2].data_ptr(), 1, words.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream) == code
    assert torch.equal(words[:size], plan) and b.cache.status() == 0


@pytest.mark.parametrize("dim,page,hq,hkv,samples,length,run", [
    (128, 32, 8, 2, 12, 5000, 512), (128, 64, 8, 1, 17, 9000, 2048), (64, 16, 4, 2, 17, 3000, 512), (256, 64, 4, 1, 17, 7000, 2048),
    (64, 64, 16, 1, 17, 4000, 512)])
def test_long_prefixes_of_values_of_one_sign(P, dim, page, hq, hkv, samples, length, run):
    """Sums over thousands of positions that all add up stay within fp32, however many: groups enough that no prefix is split
    over CTAs. Bound: the head of this file, where its 1e-5 of A is: `run` positions to a running sum are run / 16 products,
    each of which cuts off 2^-23 of it at most, which is half of the final one on the way: run / 16 2^-24; and 1e-6 for sums
    of these (some ten, 2^-24 each) and exponentials (2^-22)."""
    groups = 60
    pages = -(-(length + 40) // page)
    b = Shared(P, hq=hq, hkv=hkv, dim=dim, page=page, n_pages=groups * (pages + samples * 2), max_seqs=groups * samples, max_pages=pages + 1)
    lead = list(range(0, groups * samples, samples))
    b.cache.reserve(*b.args(lead, [length - 38 * g for g in range(groups)]))
    b.k.view(torch.uint8).copy_(torch.randint(0, 0x3c, b.k.shape, device="cuda", dtype=torch.uint8) +
                                128 * torch.randint(0, 2, b.k.shape, device="cuda", dtype=torch.uint8))
    b.v.view(torch.uint8).copy_(torch.randint(0x30, 0x40, b.v.shape, device="cuda", dtype=torch.uint8))
    b.ks.fill_(0.25)
    b.vs.copy_(2.0 ** torch.randint(-2, 3, b.vs.shape, device="cuda").float())
    b.cache.fork(dev(np.repeat(lead, samples - 1)), dev([s + i for s in lead for i in range(1, samples)]))
    seqs = list(range(groups * samples))
    args = b.args(seqs, [1] * len(seqs))
    b.cache.reserve(*args)
    plan = b.cache.share(*args, dev([samples * g for g in range(groups + 1)]))
    assert (plan[2 * groups + 1:3 * groups + 1] > 512).all()
    q = torch.randn(len(seqs), hq, dim, device="cuda")
    got = b.cache.attend_shared(0, *args, plan, q)
    assert b.cache.status() == 0
    scale, G = dim ** -0.5, hq // hkv
    table, lengths = b.cache.table.long(), b.cache.length.tolist()
    for s in (0, 1, samples - 1, 7 * samples + 2, len(seqs) - 1):
        j = torch.arange(lengths[s], device="cuda")
        at = table[s, j // page]
        k, v = (x.view(torch.uint8)[0, at, :, j % page].view(torch.float8_e4m3fn).double() * y[0, at].double()[..., None]
                for x, y in ((b.k, b.ks), (b.v, b.vs)))
        x = torch.einsum("hgd,khd->hgk", q[s].double().view(hkv, G, dim), k) * scale
        want = torch.einsum("hgk,khd->hgd", torch.softmax(x, -1), v).view(hq, dim)
        largest = scale * q[s].double().norm(dim=-1, keepdim=True) * k.norm(dim=-1).max()
        sums = run / 16 * 2.0 ** -24 + 1e-6
        off = (got[s].double() - want) / want
        assert (off.abs() <= sums + 2.0 ** -24 + 2 * 12 * 2.0 ** -23 * largest).all(), off.abs().max()
        assert off.mean().abs() <= sums, off.mean()                 # (a logit's errors have either sign)
