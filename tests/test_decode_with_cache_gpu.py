"""The example decoder (attention over the paged cache + sparse FFN): prompts fill the cache as single tokens do, a fork
carries on as its source does, and compaction moves nothing that matters."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    from examples import decode_with_cache

    return decode_with_cache


def test_prompt_fills_the_cache_as_single_tokens_do(E):
    """The first layer's keys and values (a function of the tokens alone; later layers see the predictor's list, which
    for a chunk is the union over its tokens): the same block scales from one chunk as from one token at a time, and
    codes at most a step apart (matrix products of 90 rows and of one differ in their last bits, and a code among the
    subnormals is rounded again when its page's scale grows)."""
    a, b = E.Decoder(), E.Decoder()
    x = torch.randn(90, a.d, device="cuda")
    whole = a.forward(E.ids(0), E.ids(0, 90), x)
    for t in range(90):
        b.step(E.ids(0), x[t:t + 1])
    a.check(), b.check()
    assert torch.isfinite(whole).all() and torch.equal(a.cache.length, b.cache.length)
    assert torch.equal(a.cache.table, b.cache.table)
    pages = a.cache.table[0, :-(-90 // a.cache.page_tokens)].long()
    for name in ("k", "v"):
        ca, cb = (m.cache.layers[0][name][pages].float() for m in (a, b))
        sa, sb = (m.cache.layers[0][name + "_scale"][pages] for m in (a, b))
        assert torch.equal(sa, sb)
        step = torch.maximum(ca.abs(), cb.abs()) / 8 + 2.0 ** -9
        assert ((ca - cb).abs() <= step).all()
    a.close(), b.close()


def test_fork_and_compaction_leave_the_outputs(E):
    m = E.Decoder()
    x = torch.randn(75, m.d, device="cuda")
    m.forward(E.ids(0, 1), E.ids(0, 70, 75), x)
    m.cache.fork(E.ids(0, 0), E.ids(3, 5))
    t = torch.randn(1, m.d, device="cuda")
    y = m.step(E.ids(0, 3, 5), t.expand(3, -1).contiguous())             # the same token for source and copies
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    m.cache.free(E.ids(0, 1))
    u = torch.randn(1, m.d, device="cuda")
    m.cache.fork(E.ids(3), E.ids(1))                                     # a spare copy for the step before compaction
    before = m.step(E.ids(1), u)
    m.cache.free(E.ids(1))
    live = int(m.cache.compact())
    assert live == int((m.cache.ref > 0).sum()) and (m.cache.ref[live:] == 0).all()
    after = m.step(E.ids(5), u)
    assert torch.equal(before, after)
    m.check()
    m.close()


def test_example_runs(E, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["decode_with_cache.py", "--steps", "5", "--window", "24"])
    E.main()
    assert "pages in use" in capsys.readouterr().out
