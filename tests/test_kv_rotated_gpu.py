"""append_rotated on the GPU against the plain cache and the plain rotation in fp64: scales and values' codes exactly, keys'
codes to half a step of what was rotated, queries as pi_rotate's.

Bounds: a rotated element is within 2^-18 of its pair's size (tests/test_proj_gpu.py); an e4m3 code adds half a step, 2^-4
of the value or 2^-10 of the block scale among the subnormals.
"""
import numpy as np
import pytest
import torch

from tests import proj_plain as plain
from tests.kv_plain import TABLE, block_scale
from tests.test_kv_gpu import Both
from tests.test_proj_gpu import close, num, rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import activation_sparse_decode_pi_gb300 as P

    return P


def step(P, b, seqs, new, kind, r, freq, opts, *, fused=0, in_place=False, change=None):
    """reserve and one append_rotated on `b`, checked."""
    p = b.plain
    b.reserve(seqs, new)
    T, dim = int(sum(new)), p.dim
    wide = torch.tensor(b.rng.standard_normal((T, (p.hq + 2 * p.hkv) * dim + fused)) *
                        2.0 ** b.rng.integers(-2, 3, (T, 1)), device="cuda").to({"f32": torch.float32, "bf16": torch.bfloat16,
                                                                                "f16": torch.float16}[kind])
    h = wide[:, fused // 2:fused // 2 + (p.hq + 2 * p.hkv) * dim].unflatten(1, (-1, dim))
    if change is not None:
        change(h)
    q, k, v = h[:, :p.hq], h[:, p.hq:p.hq + p.hkv], h[:, p.hq + p.hkv:]
    qn, kn, vn = num(q), num(k), num(v)
    p.k[:], p.ks[:] = b.k.view(torch.uint8).cpu().numpy(), num(b.ks)       # earlier keys as they were coded
    old_k, old_s = p.k.copy(), p.ks.copy()
    got = b.cache.append_rotated(0, *b.args(seqs, new), r, q, k, v, q_out=q if in_place else None)
    pos = np.concatenate([np.arange(p.length[s] - n, p.length[s]) for s, n in zip(seqs, new)] or [[]]).astype(int)
    close(got, *plain.rotate(qn, freq, pos, **opts[0]), kind)
    want, size = plain.rotate(kn, freq, pos, **opts[1])
    p.append(0, seqs, new, want, vn)                                       # values' codes, keys' scales, recoded keys
    new_k = b.k.view(torch.uint8).cpu().numpy()
    assert np.array_equal(num(b.ks), p.ks, equal_nan=True)
    row = 0
    for s, n in zip(seqs, new):
        for i in range(n):
            at = p.length[s] - n + i
            page, slot = p.table[s, at // p.page], at % p.page
            sc = p.ks[0, page][:, None]
            code = TABLE[new_k[0, page, :, slot]] * sc
            x = want[row]
            tol = size[row] * 2.0 ** -18 + np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)
            assert (np.abs(code - x) <= tol * (1 + 2.0 ** -18)).all(), (s, at)
            p.k[0, page, :, slot] = new_k[0, page, :, slot]
            row += 1
    assert not np.isnan(old_s[old_s == old_s]).any() and old_k.shape == new_k.shape
    b.same()
    if fused:
        assert h.shape[0] == T
    return got


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,rot,interleaved,norm,page,hq,hkv", [
    (64, 64, False, True, 16, 3, 3), (64, 32, True, False, 128, 8, 2), (128, 128, False, True, 64, 8, 2),
    (128, 32, False, False, 32, 5, 1), (256, 256, False, True, 128, 4, 2), (256, 128, True, True, 16, 2, 2),
    (128, 0, False, True, 32, 4, 4)])
def test_append_rotated(P, kind, dim, rot, interleaved, norm, page, hq, hkv):
    b = Both(P, hq=hq, hkv=hkv, dim=dim, page=page, n_pages=64, max_pages=24)
    r, freq, opts = rotary(P, b.rng, dim, rot, norm=norm, interleaved=interleaved, amp=1.125)
    step(P, b, [3, 0, 5], [1, page, page + 1], kind, r, freq, opts)
    step(P, b, [5, 3, 1], [page - 1, 3, 0], kind, r, freq, opts, fused=64)
    step(P, b, [0, 5, 3, 2], [2 * page + 5, 1, 1, 3 * page - 1], kind, r, freq, opts, in_place=True)
    step(P, b, [2, 3, 0, 5, 1], [1, 1, 1, 1, 1], kind, r, freq, opts, fused=16)
    step(P, b, [4], [1], kind, r, freq, opts)


def test_matches_rotate_then_append(P):
    """Queries bit for bit those of pi_rotate; keys of an fp32 model those of pi_rotate and pi_kv_append."""
    a, b = (Both(P, hq=6, hkv=2, dim=128, page=32, n_pages=40, max_pages=12, seed=7) for _ in range(2))
    r, _, _ = rotary(P, a.rng, 128, 128, norm=True, interleaved=False)
    for new in ([70, 1, 33], [1, 1, 1]):
        seqs = [0, 2, 5]
        a.reserve(seqs, new)
        b.reserve(seqs, new)
        T = sum(new)
        q, k, v = (torch.randn((T, n, 128), device="cuda") for n in (6, 2, 2))
        pos = torch.cat([torch.arange(int(a.plain.length[s]) - n, int(a.plain.length[s])) for s, n in zip(seqs, new)])
        qo, ko = r.rotate(pos.to(torch.int32).cuda(), q, k)
        a.cache.append(0, *a.args(seqs, new), ko, v)
        got = b.cache.append_rotated(0, *b.args(seqs, new), r, q, k, v)
        assert torch.equal(got, qo)
        for x, y in ((a.k.view(torch.uint8), b.k.view(torch.uint8)), (a.v.view(torch.uint8), b.v.view(torch.uint8))):
            assert torch.equal(x, y)
        assert a.cache.status() == 0 and b.cache.status() == 0


def test_scale_grows_and_recodes(P):
    b = Both(P, hq=1, hkv=1, dim=64, page=16)
    r, freq, opts = rotary(P, b.rng, 64, 64, norm=False, interleaved=False)
    for i in range(8):
        step(P, b, [2], [1], "f32", r, freq, opts, change=lambda h, i=i: h.mul_(2.7 ** i / 50))


def test_extreme_values(P):
    """NaN and infinite keys: coded as pi_kv_append codes them, their partners NaN; other heads and tokens untouched."""
    b = Both(P, hq=2, hkv=2, dim=64, page=16)
    r, _, _ = rotary(P, b.rng, 64, 32, norm=False, interleaved=True)
    b.reserve([1], [3])
    q, k, v = (torch.randn((3, 2, 64), device="cuda") for _ in range(3))
    k[0, 0, 50], k[1, 1, 3], v[2, 1, 0], v[0, 0, 1] = float("inf"), float("nan"), float("nan"), -float("inf")
    b.cache.append_rotated(0, *b.args([1], [3]), r, q, k, v)
    page = int(b.cache.table[1, 0])
    kk, vv = (x.view(torch.uint8)[0, page].cpu().numpy() for x in (b.k, b.v))
    assert kk[0, 0, 50] == 0x7e and (kk[1, 1, 2:4] & 0x7f == 0x7f).all() and vv[1, 2, 0] & 0x7f == 0x7f and vv[0, 0, 1] == 0xfe
    assert (kk[:, :3] & 0x7f == 0x7f).sum() == 2 and (vv[:, :3] & 0x7f == 0x7f).sum() == 1


def test_skipped_and_flagged(P):
    """A sequence without room, a table row out of range and rows past the last sequence are left as they were."""
    b = Both(P, hq=2, hkv=1, dim=64, page=16, n_pages=8, max_seqs=3, max_pages=4)
    r, _, _ = rotary(P, b.rng, 64, 64, norm=False, interleaved=False)
    b.reserve([0], [2])
    q, k, v = (torch.randn((7, n, 64), device="cuda") for n in (2, 1, 1))
    out = torch.full_like(q, 5.0)
    before = b.k.view(torch.uint8).clone()
    seqs, start = torch.tensor([0, 1, 9], device="cuda", dtype=torch.int32), torch.tensor([0, 2, 4, 5], device="cuda", dtype=torch.int32)
    b.cache.append_rotated(0, seqs, start, r, q, k, v, q_out=out)
    assert b.cache.status() == P.PI_ERR_DEVICE_CHECK and b.cache.status() == 0
    assert (out[2:] == 5.0).all() and not (out[:2] == 5.0).any()
    page = int(b.cache.table[0, 0])
    after = b.k.view(torch.uint8)
    changed = (after != before).flatten(2).any(2)
    assert changed[0, page].item() and changed.sum() == 1


def test_far_positions_and_the_same_bits_in_a_graph(P):
    b = Both(P, hq=4, hkv=2, dim=128, page=64, n_pages=16, max_seqs=2, max_pages=4000)
    far = 4000 * 64 - 70
    b.plain.length[1] = far                                          # its earlier pages are gone
    b.cache.length[1] = far
    r, freq, opts = rotary(P, b.rng, 128, 128, norm=True, interleaved=False, base=5e5)
    b.plain.table[1, far // 64] = 3
    b.cache.table[1, far // 64] = 3
    b.plain.ref[3] = 1
    b.cache.ref[3] = 1
    b.ks[0, 3], b.vs[0, 3] = 0.5, 0.5
    b.plain.vs[0, 3] = 0.5
    step(P, b, [1], [37], "bf16", r, freq, opts)
    T = 30
    b.reserve([1], [T])
    q, k, v = (torch.randn((T, n, 128), device="cuda") for n in (4, 2, 2))
    out = torch.empty_like(q)
    args = b.args([1], [T])
    kept = [x.view(torch.uint8).clone() for x in (b.k, b.v)] + [b.ks.clone(), b.vs.clone()]
    b.cache.append_rotated(0, *args, r, q, k, v, q_out=out)
    torch.cuda.synchronize()
    first = [x.clone() for x in (out, b.k.view(torch.uint8), b.v.view(torch.uint8), b.ks, b.vs)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            b.cache.append_rotated(0, *args, r, q, k, v, q_out=out)
    for x, y in zip((b.k.view(torch.uint8), b.v.view(torch.uint8), b.ks, b.vs), kept):
        x.copy_(y)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip((out, b.k.view(torch.uint8), b.v.view(torch.uint8), b.ks, b.vs), first):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())


def test_refusals(P):
    b = Both(P, hq=4, hkv=2, dim=64, page=16)
    r, _, _ = rotary(P, b.rng, 64, 64, norm=False, interleaved=False)
    b.reserve([0], [3])
    q, k, v = (torch.randn((3, n, 64), device="cuda") for n in (4, 2, 2))
    args = b.args([0], [3])
    other = P.Rotary(P.rotary_frequencies(128), 128)
    for call in (lambda: b.cache.append_rotated(0, *args, other, q, k, v),
                 lambda: b.cache.append_rotated(0, *args, r, q[:, :3], k, v),
                 lambda: b.cache.append_rotated(0, *args, r, q, k[:2], v),
                 lambda: b.cache.append_rotated(0, *args, r, q, k, v.half()),
                 lambda: b.cache.append_rotated(0, *args, r, q.half(), k, v),
                 lambda: b.cache.append_rotated(0, *args, r, q, k, torch.randn((3, 4, 64), device="cuda")[:, ::2]),
                 lambda: b.cache.append_rotated(0, *args, r, q, k, v, q_out=torch.empty((4, 4, 64), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: b.cache.append_rotated(1, *args, r, q, k, v),
                 lambda: b.cache.append_rotated(-1, *args, r, q, k, v),
                 lambda: b.cache.append_rotated(0, *args, r, q.double(), k.double(), v.double())):
        with pytest.raises(P.PiError):
            call()
    flat = torch.zeros(3 * 512 + 256, device="cuda")
    h = flat[:1536].view(3, 8, 64)
    with pytest.raises(P.PiError):                                   # q_out over the keys of the same rows
        b.cache.append_rotated(0, *args, r, h[:, :4], h[:, 4:6], h[:, 6:], q_out=h[:, 2:6])
    b.cache.append_rotated(0, *args, r, h[:, :4], h[:, 4:6], h[:, 6:], q_out=h[:, :4])
    assert b.cache.status() == 0 and block_scale(0.0) == float(b.ks[0, int(b.cache.table[0, 0]), 0])


@pytest.mark.parametrize("per", [1, 6])
def test_1024_sequences(P, per):
    """As many sequences as a call takes, some without a new token: as rotation and append one after the other."""
    a, b = (Both(P, hq=4, hkv=2, dim=64, page=16, n_pages=2100, max_seqs=1024, max_pages=6, seed=3) for _ in range(2))
    r, _, _ = rotary(P, a.rng, 64, 64, norm=True, interleaved=False)
    for turn in range(3):
        new = [(per + i + turn) % (per + 2) for i in range(1024)]
        seqs = [(7 * i + turn) % 1024 for i in range(1024)]
        args = a.args(seqs, new)
        for x in (a, b):
            x.cache.reserve(*args)
        pos = torch.cat([torch.arange(n - m, n) for n, m in zip(a.cache.length.cpu()[torch.tensor(seqs)].tolist(), new)])
        q, k, v = (torch.randn((sum(new), n, 64), device="cuda") for n in (4, 2, 2))
        qo, ko = r.rotate(pos.to(torch.int32).cuda(), q, k)
        a.cache.append(0, *args, ko, v)
        assert torch.equal(b.cache.append_rotated(0, *args, r, q, k, v), qo)
        assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8))
        assert a.cache.status() == 0 and b.cache.status() == 0


def test_pools_past_32_bits(P):
    """A pool of more than 2^32 bytes, the sequence's pages at its end: as in a small one."""
    dim, page, hkv, n_pages = 256, 64, 2, 140000
    b = Both(P, hq=4, hkv=hkv, dim=dim, page=page, n_pages=20, max_seqs=1, max_pages=14)
    r, _, _ = rotary(P, b.rng, dim, 128, norm=True, interleaved=True)
    b.cache.reserve(*b.args([0], [700]))
    k, v = (torch.zeros((n_pages, hkv, page, dim), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones((n_pages, hkv), device="cuda") for _ in range(2))
    table = torch.arange(n_pages - 1, n_pages - 15, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    ref[table[0].long()] = 1
    big = P.KVCache([dict(k=k, v=v, k_scale=ks, v_scale=vs)], table, torch.tensor([700], dtype=torch.int32, device="cuda"), ref, n_heads=4)
    q, kn, vn = (torch.randn((700, n, dim), device="cuda") for n in (4, hkv, hkv))
    outs = [c.append_rotated(0, *b.args([0], [700]), r, q, kn, vn) for c in (b.cache, big)]
    assert torch.equal(*outs)
    small = b.cache.table[0, :11].long()
    for x, y in ((k, b.k[0]), (v, b.v[0])):
        at, to = (z.view(torch.uint8)[p].transpose(1, 2).reshape(-1, hkv, dim)[:700] for z, p in ((x, table[0, :11].long()), (y, small)))
        assert torch.equal(at, to)
    assert big.status() == 0 and b.cache.status() == 0


@pytest.mark.parametrize("n,at", [(257, 256), (700, 300), (1024, 1023)])
def test_flags_sequences_far_down_the_call(P, n, at):
    """One entry out of range, then one without room, behind more sequences than a CTA looks at in one go."""
    b = Both(P, hq=2, hkv=1, dim=64, page=16, n_pages=1100, max_seqs=1024, max_pages=2)
    r, _, _ = rotary(P, b.rng, 64, 64, norm=False, interleaved=False)
    seqs, start = (torch.arange(n + i, device="cuda", dtype=torch.int32) for i in (0, 1))
    room = torch.cat([seqs[:at], seqs[at + 1:]])
    b.cache.reserve(room, torch.arange(n, device="cuda", dtype=torch.int32))
    q, k, v = (torch.randn((n, h, 64), device="cuda") for h in (2, 1, 1))
    far = seqs.clone()
    far[at] = 5000
    for call in (far, seqs):
        out = torch.full_like(q, 5.0)
        b.cache.append_rotated(0, call, start, r, q, k, v, q_out=out)
        assert b.cache.status() == P.PI_ERR_DEVICE_CHECK and b.cache.status() == 0
        left = (out == 5.0).flatten(1).all(1)
        assert left[at] and left.sum() == 1
    b.cache.append_rotated(0, room, start[:n], r, q[:n - 1], k[:n - 1], v[:n - 1])
    assert b.cache.status() == 0


def test_refuses_outputs_over_what_the_call_reads(P):
    """q_out over the batch, the rotation's tables, the handle's state or its pools; beside them it is taken."""
    b = Both(P, hq=2, hkv=1, dim=64, page=16)
    b.reserve([0, 1], [1, 2])
    room = torch.zeros(3 * 128 + 512, device="cuda")
    out, rest = room[:384].view(3, 2, 64), room[384:]
    q, k, v = (torch.randn((3, n, 64), device="cuda") for n in (2, 1, 1))
    seqs, start = b.args([0, 1], [1, 2])

    def at(place, x):                                                # a copy of x in the room
        y = place[:x.numel() * x.element_size() // 4].view(x.dtype)
        return y.copy_(x)

    def made(place):
        r = P.Rotary(P.rotary_frequencies(64), 64, norm=True, q_norm=torch.ones(64, device="cuda"), k_norm=torch.ones(64, device="cuda"))
        for name, x in (("turns", r.turns), ("q_norm", r.q_norm), ("k_norm", r.k_norm)):
            if name in place:
                setattr(r, name, at(place[name], x))
                setattr(r.desc, name, getattr(r, name).data_ptr())
        return r

    plain = made({})
    for place, fine in ((room[128:], False), (rest, True)):
        for r, s, t in ((made(dict(turns=place)), seqs, start), (made(dict(q_norm=place)), seqs, start),
                        (made(dict(k_norm=place)), seqs, start), (plain, at(place, seqs), start), (plain, seqs, at(place, start))):
            if fine:
                b.cache.append_rotated(0, s, t, r, q, k, v, q_out=out)
            else:
                with pytest.raises(P.PiError):
                    b.cache.append_rotated(0, s, t, r, q, k, v, q_out=out)
    for x in (b.k, b.v):
        with pytest.raises(P.PiError):                               # over the layer's pool
            b.cache.append_rotated(0, seqs, start, plain, q, k, v, q_out=x.view(torch.float32).flatten()[:384].view(3, 2, 64))
    assert b.cache.status() == 0
