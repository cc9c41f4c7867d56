"""Projections with 4-bit weights and the rotation of heads on the GPU, against NumPy in fp64.

Bounds (largest error of an element): a rounding to a type of p bits is at most 2^-p of the value. A group's products
(integer times f16) are exact in fp32; the tensor cores add 16 of them at a time to a sum that they cut off to 24 bits,
in 8 steps: 2^-19 of the sum of absolute products covers 17 addends cut off 8 times. x is held to 2^-22 of itself or 2^-34
of its group's largest, whose products are at most 8 / mean |q| ~ 2 of the sum; group sums add G roundings of 2^-24.
A rotated element has fp32 cosines and sines (angles to 2^-26 of a turn: 2^-23.3), three products and a sum, a mean square
of `dim` roundings at worst 2^-24 dim / 2 of itself and its root: below 2^-18 of the pair's size.
"""
import numpy as np
import pytest
import torch

from tests import proj_plain as plain

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def P():
    import activation_sparse_decode_pi_gb300 as P

    return P


def wide(rng, rows, width, kind, more=0, scale=None):
    """[rows, width] values of a type in rows `more` elements wider."""
    x = rng.standard_normal((rows, width + more))
    if scale is not None:
        x = x * scale
    full = torch.tensor(x, device="cuda").to(TYPES[kind])
    return full[:, more // 2:more // 2 + width]


def num(x):
    return x.double().cpu().numpy()


# ------------------------------------------------------------------------------------------------ 4-bit projections

def weights(rng, n, k):
    w = rng.integers(0, 256, (n, k // 2)).astype(np.uint8)
    s = (rng.uniform(0.2, 1.0, (n, k // 128)) / 8).astype(np.float16)
    return w, s


def check_linear(P, rng, rows, n, k, kind, *, bias=True, add="other", more=0, x=None):
    w, s = weights(rng, n, k)
    b = torch.tensor(rng.standard_normal(n), device="cuda", dtype=torch.float32) if bias else None
    x = wide(rng, rows, k, kind, more) if x is None else x
    plus = wide(rng, rows, n, kind, more // 2) if add else None
    given = None if plus is None else num(plus)
    lin = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s, device="cuda"), b)
    room = torch.full((rows, n + more), 7.0, device="cuda", dtype=TYPES[kind])
    out = plus if add == "same" else room[:, :n] if more else None
    y = lin(x, out=out, add=plus)
    assert out is None or y is out
    v, xs = plain.int4_values(w, s), num(x)
    want, size = xs @ v.T, np.abs(xs) @ np.abs(v).T
    for extra in ([] if b is None else [num(b)]) + ([] if given is None else [given]):
        want, size = want + extra, size + np.abs(extra)
    tol = size * (2.0 ** -19 + 2.0 ** -21 + (k // 128 + 3) * 2.0 ** -24) + HALF[kind] * np.abs(want) + TINY[kind]
    err = np.abs(num(y) - want)
    assert (err <= tol).all(), (err / tol).max()
    if more and add != "same":
        assert (room[:, n:] == 7.0).all()
    return lin, x, y


SHAPES = [(1, 1, 128), (1, 17, 256), (1, 4099, 384), (2, 100, 4096), (8, 129, 1280), (9, 64, 5120), (16, 333, 640),
          (17, 257, 2048), (32, 48, 12288), (33, 200, 256), (64, 1000, 128), (256, 40, 512), (1, 16, 128 * 97),
          (5, 20001, 128), (24, 16, 128 * 131), (3, 5120, 5120)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,n,k", SHAPES)
def test_int4_linear(P, rows, n, k, kind):
    check_linear(P, np.random.default_rng(n + k), rows, n, k, kind)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bias,add,more", [(False, None, 0), (True, None, 16), (False, "same", 0), (True, "same", 32),
                                           (False, "other", 64)])
def test_int4_linear_epilogues_and_strides(P, kind, bias, add, more):
    for rows, n, k in [(1, 50, 256), (13, 200, 1024)]:
        check_linear(P, np.random.default_rng(more), rows, n, k, kind, bias=bias, add=add, more=more)


def test_int4_linear_groups_of_very_different_size(P):
    rng = np.random.default_rng(1)
    scale = np.repeat(2.0 ** rng.integers(-60, 60, (3, 16)), 128, axis=1)
    check_linear(P, rng, 3, 70, 2048, "f32", x=wide(rng, 3, 2048, "f32", scale=scale), bias=False, add=None)
    check_linear(P, rng, 3, 70, 2048, "bf16", x=wide(rng, 3, 2048, "bf16", scale=scale), bias=False, add=None)


def test_int4_linear_same_bits_each_time_and_in_a_graph(P):
    rng = np.random.default_rng(2)
    lin, x, y = check_linear(P, rng, 16, 700, 5120, "f32", add=None)
    for _ in range(5):
        assert torch.equal(lin(x), y)
    out = torch.empty_like(y)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lin(x, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            lin(x, out=out)
    out.zero_()
    x2 = x.clone()
    x.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, lin(x)) and not torch.equal(out, y)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_int4_linear_infinite_and_nan_inputs_stay_in_their_rows(P, kind):
    rng = np.random.default_rng(3)
    n, k = 40, 512
    w, s = weights(rng, n, k)
    w[w == 0] = 0x11
    w[:, 50] = 0x23                                   # elements 100 and 101: 3 and 2
    lin = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s, device="cuda"))
    x = wide(rng, 12, k, kind)
    clean = lin(x)
    x[4, 100], x[7, 300], x[9, 101] = float("inf"), float("nan"), -float("inf")
    y = lin(x)
    keep = [i for i in range(12) if i not in (4, 7, 9)]
    assert torch.equal(y[keep], clean[keep])
    assert (y[4] == float("inf")).all() and torch.isnan(y[7]).all() and (y[9] == -float("inf")).all()


def test_int4_linear_zero_rows_and_zero_scales(P):
    rng = np.random.default_rng(4)
    w, s = weights(rng, 30, 256)
    lin = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s * 0, device="cuda"))
    assert lin(torch.zeros((0, 256), device="cuda")).shape == (0, 30)
    assert (lin(wide(rng, 3, 256, "f32")) == 0).all()
    lin = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s, device="cuda"))
    assert (lin(torch.zeros((2, 256), device="cuda", dtype=torch.bfloat16)) == 0).all()


def test_int4_linear_on_another_stream(P):
    rng = np.random.default_rng(5)
    lin, x, y = check_linear(P, rng, 4, 300, 1024, "bf16", add=None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        z = lin(x, stream=stream)
        s.synchronize()
        assert torch.equal(z, y)


def test_int4_linear_two_streams_at_once(P):
    """Nothing is shared between calls: many under way on two streams."""
    rng = np.random.default_rng(7)
    calls = [check_linear(P, rng, rows, n, k, kind, add=None) for rows, n, k, kind in
             [(1, 3000, 4096, "bf16"), (16, 2000, 5120, "f32"), (3, 500, 12288, "f32"), (40, 700, 1024, "f16")]]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(40):
        for j, s in enumerate(streams):
            lin, x, want = calls[(i + j) % 4]
            outs.append((lin(x, stream=s), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)


def test_int4_linear_offsets_past_32_bits(P):
    """More than 2^32 bytes of weights: the last outputs against fp64."""
    n, k = 300001, 32768
    w = torch.randint(0, 256, (n, k // 2), device="cuda", dtype=torch.uint8)
    s = torch.rand((n, k // 128), device="cuda").half()
    assert w.numel() > 2 ** 32
    for rows, kind in ((1, "f32"), (9, "bf16")):
        x = torch.randn((rows, k), device="cuda").to(TYPES[kind])
        y = P.Int4Linear(w, s)(x)
        for at in (0, 131071, n - 40):
            v = plain.int4_values(w[at:at + 40].cpu().numpy(), s[at:at + 40].cpu().numpy())
            want, size = num(x) @ v.T, np.abs(num(x)) @ np.abs(v).T
            tol = size * (2.0 ** -19 + 2.0 ** -21 + (k // 128 + 3) * 2.0 ** -24) + HALF[kind] * np.abs(want)
            assert (np.abs(num(y[:, at:at + 40]) - want) <= tol).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,n,k", [(17, 40000, 640), (40, 20000, 1280), (64, 30000, 384), (100, 5000, 2048), (200, 300, 5120),
                                      (33, 129, 12288), (48, 700, 128 * 257), (18, 40, 1 << 18)])
def test_int4_linear_many_rows(P, rows, n, k, kind):
    """Many tiles to a CTA, shares of the contraction of every parity, several slices of the rows, the longest contraction."""
    lin, x, y = check_linear(P, np.random.default_rng(rows), rows, n, k, kind, add=None)
    assert torch.equal(lin(x), y)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_int4_linear_infinite_and_nan_inputs_among_many_rows(P, kind):
    rng = np.random.default_rng(8)
    w, s = weights(rng, 300, 1024)
    w[w == 0] = 0x11
    w[:, 50] = 0x23
    lin = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s, device="cuda"))
    x = wide(rng, 40, 1024, kind)
    clean = lin(x)
    x[4, 100], x[37, 300], x[39, 101] = float("inf"), float("nan"), -float("inf")
    y = lin(x)
    keep = [i for i in range(40) if i not in (4, 37, 39)]
    assert torch.equal(y[keep], clean[keep])
    assert (y[4] == float("inf")).all() and torch.isnan(y[37]).all() and (y[39] == -float("inf")).all()


def test_int4_linear_many_rows_two_streams_at_once(P):
    """CTAs of two calls with clusters, side by side: each SM has one call's tensor memory at a time."""
    rng = np.random.default_rng(9)
    calls = [check_linear(P, rng, rows, n, k, kind, add=None) for rows, n, k, kind in
             [(20, 3000, 1024, "bf16"), (30, 20000, 512, "f32"), (64, 2000, 5120, "f16")]]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(30):
        for j, st in enumerate(streams):
            lin, x, want = calls[(i + j) % 3]
            outs.append((lin(x, stream=st), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)


def test_int4_linear_refusals(P):
    rng = np.random.default_rng(6)
    w, s = (torch.tensor(a, device="cuda") for a in weights(rng, 8, 256))
    lin = P.Int4Linear(w, s)
    x = torch.zeros((4, 256), device="cuda")
    for bad in (x[:, :128], x.T, x.cpu(), torch.zeros((4, 512), device="cuda")[:, ::2], x[0]):
        with pytest.raises(ValueError):
            lin(bad)
    for kw in (dict(out=torch.zeros((4, 9), device="cuda")), dict(out=torch.zeros((3, 8), device="cuda")),
               dict(out=torch.zeros((4, 8), device="cuda", dtype=torch.float16)), dict(add=torch.zeros((5, 8), device="cuda"))):
        with pytest.raises(ValueError):
            lin(x, **kw)
    with pytest.raises(P.PiError):
        lin(torch.zeros((4, 256), device="cuda", dtype=torch.float64))
    with pytest.raises(P.PiError):
        lin(torch.zeros((257, 256), device="cuda"))
    flat = torch.zeros(4 * 256 + 64, device="cuda")
    with pytest.raises(P.PiError):                                   # not on 16 bytes
        lin(flat[1:1025].view(4, 256))
    with pytest.raises(P.PiError):                                   # out lies in x
        lin(x, out=x[:, :8])
    both = torch.zeros(40, device="cuda")
    with pytest.raises(P.PiError):                                   # out and add a row apart
        lin(x, out=both[:32].view(4, 8), add=both[8:].view(4, 8))
    for bad in (w.to(torch.int8), w[:, :100], w.T):
        with pytest.raises(ValueError):
            P.Int4Linear(bad, s)
    with pytest.raises(ValueError):
        P.Int4Linear(w, s.float())
    with pytest.raises(ValueError):
        P.Int4Linear(w, s, torch.zeros(8, device="cuda", dtype=torch.float16))
    assert P._lib.pi_int4_linear(w.data_ptr(), s.data_ptr(), None, 1 << 24, 256, x.data_ptr(), 256, 4, None, 0,
                                 flat.data_ptr(), 1 << 24, 0, None) == 1      # 2 GB of weights in another allocation
    x1 = torch.zeros((1, 256), device="cuda")
    assert (lin(x1) == 0).all()


def test_ranges_are_checked_for_a_thread_without_a_context(P):
    """The first call of a new host thread works as every other does, and refuses arrays past their allocation."""
    import threading

    rng = np.random.default_rng(6)
    w, s = (torch.tensor(a, device="cuda") for a in weights(rng, 8, 256))
    x, y = torch.zeros((4, 256), device="cuda"), torch.zeros((4, 8), device="cuda")
    torch.cuda.synchronize()
    codes = []

    def call(n):
        codes.append(P._lib.pi_int4_linear(w.data_ptr(), s.data_ptr(), None, n, 256, x.data_ptr(), 256, 4, None, 0, y.data_ptr(),
                                           n, 0, None))

    for n in (1 << 24, 8):                                           # 2 GB of weights in another allocation; as they are
        t = threading.Thread(target=call, args=(n,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert codes == [1, 0] and (y == 0).all()


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_int4_linear_zero_weights_give_zero(P, kind, rows):
    """Groups of zeros with scales that are not add nothing, whatever x is."""
    rng = np.random.default_rng(10)
    w, s = weights(rng, 200, 1024)
    w[:] = 0
    y = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s, device="cuda"))(wide(rng, rows, 1024, kind))
    assert (y == 0).all()


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_int4_linear_large_elements_of_zero_weight(P, kind, rows):
    """One element of each group thousands of times the others, its weight 0: the others keep their bits (f16 terms hold them
    to 2^-39 of the large one, 2^-25 of themselves)."""
    rng = np.random.default_rng(11)
    n, k = 150, 1280
    w, s = weights(rng, n, k)
    w[:, 2::64] &= 0x0f                                              # element 5 of every group
    w[:, 40::64] &= 0xf0                                             # element 80
    x = rng.standard_normal((rows, k)) * 2.0 ** -10
    x[:, 5::128], x[:, 80::128] = rng.uniform(8, 16, (rows, k // 128)), -rng.uniform(4, 8, (rows, k // 128))
    x = torch.tensor(x, device="cuda").to(TYPES[kind])
    y = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s, device="cuda"))(x)
    v, xs = plain.int4_values(w, s), num(x)
    want, size = xs @ v.T, np.abs(xs) @ np.abs(v).T
    tol = size * (2.0 ** -19 + 2.0 ** -21 + (k // 128 + 3) * 2.0 ** -24) + HALF[kind] * np.abs(want) + TINY[kind]
    assert (np.abs(num(y) - want) <= tol).all()


@pytest.mark.parametrize("rows,n,k", [(1, 300, 512), (1, 300, 5120), (8, 300, 12288), (1, 200, 128 * 257), (16, 300, 5120),
                                      (20, 300, 12288), (16, 200, 128 * 257)])
def test_int4_linear_error_of_long_contractions(P, rows, n, k):
    """fp32 rows in the L2 norm, whose bound does not grow with k: errors of groups are independent, so that their sum is to
    the result as one group's error is to one group's sum. That is 8 cut-offs of a running sum, of 2^-24 of it on average,
    all of one sign; over the 8 steps it is 2/3 of the final one in the norm: 2^-21.6 in all. x's terms are off by 2^-23 of an
    element at most, of either sign. Below 2^-21, where operands are normal numbers (products of subnormals are cut off
    further up). x's second term left out of one group of 257 costs 1.2e-5."""
    rng = np.random.default_rng(k + rows)
    w, s = weights(rng, n, k)
    x = wide(rng, rows, k, "f32")
    y = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s, device="cuda"))(x)
    want = num(x) @ plain.int4_values(w, s).T
    err = np.linalg.norm(num(y) - want, axis=1) / np.linalg.norm(want, axis=1)
    assert err.max() <= 2.0 ** -21, err.max()


@pytest.mark.parametrize("rows", [6, 20])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_int4_linear_infinities_meet_every_weight(P, kind, rows):
    """An infinity times 0 is NaN, and two of different sign are; else it gives its own."""
    rng = np.random.default_rng(12)
    w, s = weights(rng, 300, 512)
    s[7] = 0
    x = wide(rng, rows, 512, kind)
    inf = float("inf")
    x[0, 3], x[1, 200], x[3, 1], x[3, 257], x[4, 128], x[4, 129] = inf, -inf, inf, inf, -inf, float("nan")
    y = P.Int4Linear(torch.tensor(w, device="cuda"), torch.tensor(s, device="cuda"))(x)
    with np.errstate(invalid="ignore"):
        want = (num(x)[:, None, :] * plain.int4_values(w, s)[None]).sum(-1)
    assert np.array_equal(np.isnan(num(y)), np.isnan(want)) and np.isnan(want[4]).all() and not np.isnan(want[2]).any()
    bad = np.isinf(want)
    assert bad.any() and np.array_equal(num(y)[bad], want[bad]) and np.isfinite(num(y)[~bad & ~np.isnan(want)]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("rows,n,k", [(9, 6600, 1280), (13, 20001, 256), (16, 9000, 5120), (16, 15360, 128), (10, 7000, 128 * 97)])
def test_int4_linear_some_rows_of_many_outputs(P, rows, n, k, kind):
    lin, x, y = check_linear(P, np.random.default_rng(rows + n), rows, n, k, kind)
    assert torch.equal(lin(x), lin(x))


# ------------------------------------------------------------------------------------------------ rotation

POS = [0, 1, 2, 77, 4095, 131071, 1000003, 2 ** 30 + 1, 2 ** 31 - 1, -1, -100, -2 ** 31]


def rotary(P, rng, dim, rot, *, norm, interleaved, amp=1.0, weights=True, base=1e4, eps=1e-6, **kw):
    freq = P.rotary_frequencies(rot, base, **kw)
    w = [torch.tensor(1 + 0.3 * rng.standard_normal(dim), device="cuda", dtype=torch.float32) if norm and weights else None
         for _ in range(2)]
    r = P.Rotary(freq, dim, interleaved=interleaved, amp=amp, norm=norm, q_norm=w[0], k_norm=w[1], eps=eps)
    opts = [dict(interleaved=interleaved, amp=amp, norm=norm, weight=None if x is None else num(x), eps=eps) for x in w]
    return r, freq, opts


def heads(rng, T, n, dim, kind, more=0, spread=3):
    x = wide(rng, T, n * dim, kind, more, scale=2.0 ** rng.integers(-spread, spread + 1, (T, 1)))
    return x.unflatten(1, (n, dim))


def close(got, want, size, kind):
    tol = size * 2.0 ** -18 + HALF[kind] * np.abs(want) + TINY[kind]
    err = np.abs(num(got) - want)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (64, 16, True), (128, 128, False), (128, 32, False),
                                                 (128, 48, True), (128, 96, False), (256, 256, False), (256, 64, True),
                                                 (64, 0, False)])
def test_rotate(P, kind, norm, dim, rot, interleaved):
    rng = np.random.default_rng(dim + rot)
    r, freq, opts = rotary(P, rng, dim, rot, norm=norm, interleaved=interleaved, amp=1.25)
    for T, hq, hk in [(1, 1, 1), (1, 32, 8), (12, 7, 3), (300, 5, 5)]:
        pos = np.array((POS * 25)[:T], np.int64)
        q, k = heads(rng, T, hq, dim, kind, 16), heads(rng, T, hk, dim, kind)
        qo, ko = r.rotate(torch.tensor(pos, device="cuda").to(torch.int32), q, k)
        for x, y, o in ((q, qo, opts[0]), (k, ko, opts[1])):
            close(y, *plain.rotate(num(x), freq, pos, **o), kind)


def test_rotate_many_tokens(P):
    rng = np.random.default_rng(1)
    r, freq, opts = rotary(P, rng, 128, 128, norm=True, interleaved=False, base=5e5, stretch=8.0, trained=8192)
    T = 2999
    q, k = heads(rng, T, 6, 128, "bf16"), heads(rng, T, 2, 128, "bf16")
    pos = np.arange(T) + 70000
    qo, ko = r.rotate(torch.arange(70000, 70000 + T, device="cuda", dtype=torch.int32), q, k)
    close(qo, *plain.rotate(num(q), freq, pos, **opts[0]), "bf16")
    close(ko, *plain.rotate(num(k), freq, pos, **opts[1]), "bf16")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rotate_in_place_in_a_fused_projection(P, kind):
    rng = np.random.default_rng(2)
    r, freq, opts = rotary(P, rng, 64, 64, norm=True, interleaved=False, weights=False)
    for T in (1, 50):
        qkv = wide(rng, T, (6 + 2 + 2) * 64, kind)
        before = qkv.clone()
        h = qkv.unflatten(1, (10, 64))
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        want_q, want_k = r.rotate(pos, h[:, :6], h[:, 6:8])
        qo, ko = r.rotate(pos, h[:, :6], h[:, 6:8], q_out=h[:, :6], k_out=h[:, 6:8])
        assert torch.equal(qo, want_q) and torch.equal(ko, want_k) and torch.equal(qkv[:, 512:], before[:, 512:])
        assert torch.equal(qkv[:, :384], want_q.flatten(1)) and torch.equal(qkv[:, 384:512], want_k.flatten(1))
        close(want_q, *plain.rotate(num(before[:, :384].unflatten(1, (6, 64))), freq, np.arange(T), **opts[0]), kind)


def test_rotate_queries_only_and_no_tokens(P):
    rng = np.random.default_rng(3)
    r, freq, opts = rotary(P, rng, 128, 64, norm=False, interleaved=True)
    q = heads(rng, 9, 4, 128, "f32")
    qo, ko = r.rotate(torch.arange(9, device="cuda", dtype=torch.int32), q)
    assert ko is None
    close(qo, *plain.rotate(num(q), freq, np.arange(9), **opts[0]), "f32")
    none = torch.zeros(0, device="cuda", dtype=torch.int32)
    assert r.rotate(none, q[:0], q[:0])[1].shape == (0, 4, 128)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_infinite_and_nan_elements(P, interleaved):
    """What is not turned passes through; a bad element reaches its partner (without a norm) and nothing else."""
    rng = np.random.default_rng(4)
    r, _, _ = rotary(P, rng, 64, 32, norm=False, interleaved=interleaved)
    q = heads(rng, 3, 4, 64, "f32")
    pos = torch.tensor([5, 6, 7], device="cuda", dtype=torch.int32)
    clean, _ = r.rotate(pos, q)
    q[0, 1, 40], q[1, 2, 4], q[2, 3, 63] = float("inf"), float("nan"), float("nan")
    got, _ = r.rotate(pos, q)
    touched = torch.zeros_like(clean, dtype=torch.bool)
    touched[0, 1, 40] = touched[1, 2, 4] = touched[2, 3, 63] = touched[1, 2, 5 if interleaved else 20] = True
    assert torch.equal(got[~touched], clean[~touched])
    assert got[0, 1, 40] == float("inf") and torch.isnan(got[1, 2, 4]) and torch.isnan(got[2, 3, 63])
    assert torch.isnan(got[1, 2, 5 if interleaved else 20])


def test_rotate_zero_heads_keep_zero(P):
    r = P.Rotary(P.rotary_frequencies(64), 64, norm=True)
    x = torch.zeros((4, 3, 64), device="cuda", dtype=torch.bfloat16)
    y, _ = r.rotate(torch.arange(4, device="cuda", dtype=torch.int32), x)
    assert (y == 0).all()


def test_rotate_in_a_graph(P):
    rng = np.random.default_rng(5)
    r, _, _ = rotary(P, rng, 128, 128, norm=True, interleaved=False)
    q, k, pos = heads(rng, 3, 8, 128, "bf16"), heads(rng, 3, 2, 128, "bf16"), torch.tensor([3, 9, 1], device="cuda", dtype=torch.int32)
    qo, ko = r.rotate(pos, q, k)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            r.rotate(pos, q, k, q_out=qo, k_out=ko)
    pos.add_(1)
    g.replay()
    torch.cuda.synchronize()
    want = r.rotate(pos, q, k)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_rotate_refusals(P):
    rng = np.random.default_rng(6)
    r, _, _ = rotary(P, rng, 64, 64, norm=True, interleaved=False)
    q, k = heads(rng, 4, 4, 64, "f32"), heads(rng, 4, 2, 64, "f32")
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    for bad in (pos.long(), pos[:3], pos.cpu(), pos[None], torch.arange(8, device="cuda", dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            r.rotate(bad, q, k)
    for a, b in ((q[..., :32], k), (q, k.half()), (q, k[:3]), (q.transpose(0, 1), k), (q.cpu(), k)):
        with pytest.raises(ValueError):
            r.rotate(pos, a, b)
    with pytest.raises(ValueError):
        r.rotate(pos, q, k, q_out=torch.empty((4, 4, 64), device="cuda", dtype=torch.float16))
    with pytest.raises(P.PiError):
        r.rotate(pos, q.double(), k.double())
    with pytest.raises(P.PiError):                                   # k's output over the queries
        r.rotate(pos, q, k, k_out=q.view(4, 256)[:, :128].unflatten(1, (2, 64)))
    with pytest.raises(P.PiError):                                   # a row of the output over another row of the input
        flat = torch.zeros(5 * 256, device="cuda")
        r.rotate(pos, flat[:1024].view(4, 4, 64), None, q_out=flat[256:].view(4, 4, 64))
    with pytest.raises(P.PiError):
        P.Rotary(P.rotary_frequencies(8), 64).rotate(pos, q)         # 8 of 64 elements
    with pytest.raises(P.PiError):
        P.Rotary(P.rotary_frequencies(128), 64).rotate(pos, q)       # more than the head
    for kw in (dict(amp=float("nan")), dict(norm=True, eps=-1.0)):
        with pytest.raises(P.PiError):
            P.Rotary(P.rotary_frequencies(64), 64, **kw).rotate(pos, q)
    with pytest.raises(ValueError):
        P.Rotary(P.rotary_frequencies(64), 64, q_norm=torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        P.Rotary(P.rotary_frequencies(64), 64, norm=True, k_norm=torch.ones(32, device="cuda"))
    flat = torch.zeros(4 * 256, device="cuda")
    with pytest.raises(P.PiError):                                   # the positions lie in the output
        r.rotate(flat[8:12].view(torch.int32), q, q_out=flat.view(4, 4, 64))
    odd = torch.zeros(4 * 256 + 8, device="cuda")
    with pytest.raises(P.PiError):
        r.rotate(pos, odd[1:1025].view(4, 4, 64))
