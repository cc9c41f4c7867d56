"""The example decoder's attention with all of its operators in a row: 4-bit projections, norms and rotation of the heads
into the 8-bit cache, attention with the prefix read once, the output projection added to the residual; against the same in
NumPy in fp64, which reads the GPU's codes (after these have been checked).

Bounds, each from its operator's tests: a projection is off by 2^-18 of its sum of absolute products, a rotated element by
2^-18 of its pair's size (and by what its inputs are off, whose norm leaves their relative size), a logit by that of its
query, 2^-16 L with L >= scale |q| |k|, an output by twice that and 1e-5 of A = sum_j p_j |v_j|; rows in the L2 norm, which
the output projection grows by its spectral norm at most.
"""
import numpy as np
import pytest
import torch

from tests import proj_plain as plain
from tests.kv_plain import TABLE, PlainCache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from examples import decode_with_cache

    return decode_with_cache


def num(x):
    return x.double().cpu().numpy()


class Twin:
    """The first layer's attention of a decoder in fp64, on the decoder's own cache."""

    def __init__(self, E, m):
        self.m = m
        self.w = [plain.int4_values(w.w.cpu().numpy(), w.s.cpu().numpy()) for w in (m.qkv[0], m.o[0])]
        self.freq = E.P.rotary_frequencies(m.dim)

    def project(self, i, x):
        return x @ self.w[i].T, np.abs(x) @ np.abs(self.w[i]).T

    def check(self, seqs, new, x, got):
        m, dim = self.m, self.m.dim
        length, table = m.cache.length.cpu().numpy(), m.cache.table.cpu().numpy()
        x = num(x)
        r = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        h, size = (a.reshape(len(x), -1, dim) for a in self.project(0, r))
        off = 2.0 ** -18 * np.linalg.norm(size, axis=-1, keepdims=True) / np.linalg.norm(h, axis=-1, keepdims=True)
        pos = np.concatenate([np.arange(length[s] - n, length[s]) for s, n in zip(seqs, new)])
        q, _ = plain.rotate(h[:, :m.heads], self.freq, pos, norm=True)
        k, k_size = plain.rotate(h[:, m.heads:m.heads + m.kv_heads], self.freq, pos, norm=True)
        v = h[:, m.heads + m.kv_heads:]
        # the codes that this call has written: half a step from what they stand for
        c = PlainCache(1, m.heads, m.kv_heads, dim, m.cache.page_tokens, m.cache.desc.n_pages, table.shape[0], table.shape[1])
        c.k[0], c.v[0] = (m.cache.layers[0][n].view(torch.uint8).cpu().numpy() for n in ("k", "v"))
        c.ks[0], c.vs[0] = (num(m.cache.layers[0][n]) for n in ("k_scale", "v_scale"))
        c.table, c.length = table, length
        page, slot = np.concatenate([table[s, np.arange(length[s] - n, length[s]) // c.page] for s, n in zip(seqs, new)]), pos % c.page
        both = 2.0 ** -18 + 2 * off.max()
        for codes, scales, want, wide in ((c.k, c.ks, k, k_size), (c.v, c.vs, v, size[:, m.heads + m.kv_heads:])):
            sc = scales[0, page][..., None]
            value = TABLE[codes[0, page, :, slot]] * sc
            assert (np.abs(value - want) <= wide * both + np.maximum(np.abs(want) * 2.0 ** -4, sc * 2.0 ** -10)).all()
        scale = dim ** -0.5
        out, _ = c.attend(0, seqs, new, q, scale)
        signed, c.v = c.v, c.v & 0x7f
        A, _ = c.attend(0, seqs, new, q, scale)
        c.v = signed
        k_norm = np.linalg.norm(TABLE[c.k[0]] * c.ks[0][..., None, None], axis=-1)[np.unique(table[table >= 0])].max()
        L = scale * np.linalg.norm(q, axis=-1).max() * k_norm
        att_off = A * (2 * (2.0 ** -16 + both) * L + 1e-5)
        y, y_size = self.project(1, out.reshape(len(x), -1))
        norm = lambda z: np.linalg.norm(z.reshape(len(x), -1), axis=-1)  # noqa: E731
        tol = np.linalg.norm(self.w[1], 2) * norm(att_off) + 2.0 ** -18 * norm(y_size) + 2.0 ** -23 * norm(x)
        err = norm(num(got) - (x + y))
        assert (err <= tol).all(), (err / tol).max()
        assert (tol < 0.25 * norm(y)).all()                        # (a wrong position, head or page is off by about |y|)


def test_attention_of_all_operators(E):
    m = E.Decoder(layers=1, rope=True, int4=True, page=16, n_pages=300, max_seqs=8, max_batch=64)
    twin, g = Twin(E, m), torch.Generator(device="cuda").manual_seed(1)

    def run(seqs, new, plan=None):
        s, start = E.ids(*seqs), E.ids(*np.concatenate([[0], np.cumsum(new)]).tolist())
        x = torch.randn(sum(new), m.d, device="cuda", generator=g)
        m.cache.reserve(s, start)
        twin.check(seqs, new, x, m.attention(0, s, start, x, plan))

    run([0, 1], [170, 37])                                        # prompts, the longer in parts of 64 rows
    m.cache.fork(E.ids(0, 0, 0), E.ids(2, 3, 5))
    seqs = [0, 2, 3, 5, 1]
    s = E.ids(*seqs)
    plan = m.cache.share(s, E.ids(0, 1, 2, 3, 4, 5), E.ids(0, 4))
    for _ in range(3):
        run(seqs, [1] * 5, plan)                                  # the prefix of four of them once
    run(seqs, [1] * 5)                                            # and for each
    run([1, 0], [1, 40])
    m.check()
    m.close()


def test_steps_with_and_without_a_plan(E):
    """All layers, FFN included: finite outputs, the same lengths, no status."""
    a, b = (E.Decoder(rope=True, int4=True, layers=2, seed=3) for _ in range(2))
    x = torch.randn(200, a.d, device="cuda")
    outs = []
    for m, shared in ((a, True), (b, False)):
        m.forward(E.ids(0), E.ids(0, 200), x)
        m.cache.fork(E.ids(0, 0), E.ids(1, 2))
        plan = m.share(E.ids(0, 1, 2)) if shared else None
        h = x[:3]
        for _ in range(4):
            h = m.step(E.ids(0, 1, 2), E.rms(h), plan)
        assert torch.isfinite(h).all()
        m.check()
        outs.append(m.cache.length.clone())
    assert torch.equal(outs[0], outs[1])
    a.close(), b.close()


@pytest.mark.parametrize("args", [["--steps", "4", "--rope"], ["--steps", "4", "--int4", "--window", "40"],
                                  ["--steps", "5", "--rope", "--int4", "--samples", "5"], ["--steps", "3", "--samples", "9"]])
def test_example_runs(E, monkeypatch, capsys, args):
    monkeypatch.setattr("sys.argv", ["decode_with_cache.py"] + args)
    E.main()
    assert "output rms" in capsys.readouterr().out
