"""The paged cache's host side without a GPU: descriptors and NULL arguments are refused before CUDA is touched, and
the plain NumPy cache that the GPU tests compare with is pinned to hand-made values."""
import ctypes
import math

import numpy as np
import pytest

from tests.kv_plain import TABLE, PlainCache, block_scale, encode


@pytest.fixture(scope="module")
def P():
    import __graft_entry__

    __graft_entry__.build()
    import activation_sparse_decode_pi_gb300 as P

    return P


GOOD = dict(n_layers=1, n_heads=8, n_kv_heads=2, head_dim=128, page_tokens=32, n_pages=10, max_seqs=4, max_pages=8)


@pytest.mark.parametrize("fields,code", [
    (dict(n_layers=0), 1), (dict(n_heads=7), 1), (dict(n_heads=0), 1), (dict(n_kv_heads=0), 1),
    (dict(n_kv_heads=-2), 1), (dict(n_heads=1), 1), (dict(n_pages=0), 1), (dict(max_seqs=0), 1),
    (dict(max_pages=0), 1), (dict(head_dim=0), 1), (dict(page_tokens=-16), 1),
    (dict(head_dim=96), 2), (dict(page_tokens=8), 2), (dict(page_tokens=48), 2), (dict(page_tokens=256), 2),
    (dict(n_pages=1 << 26), 2), (dict(max_pages=1 << 26), 2), (dict(n_heads=1 << 20), 2),
])
def test_descriptor_validation(P, fields, code):
    desc = P.PiKvDesc(**{**GOOD, **fields})
    h = ctypes.c_void_p(99)
    assert P._lib.pi_kv_create(ctypes.byref(h), ctypes.byref(desc), None, None) == code
    assert h.value is None


def test_null_arguments(P):
    desc, state = P.PiKvDesc(**GOOD), P.PiKvState()
    h = ctypes.c_void_p(99)
    assert P._lib.pi_kv_create(None, ctypes.byref(desc), None, None) == 1
    assert P._lib.pi_kv_create(ctypes.byref(h), None, None, None) == 1
    assert P._lib.pi_kv_create(ctypes.byref(h), ctypes.byref(desc), None, ctypes.byref(state)) == 1 and not h.value
    assert P._lib.pi_kv_get_status(None) == 1
    assert P._lib.pi_kv_reserve(None, None, None, 1, None) == 1
    assert P._lib.pi_kv_append(None, 0, None, None, 1, 1, None, None, 64, 0, None) == 1
    assert P._lib.pi_kv_attend(None, 0, None, None, 1, 1, None, 64, None, 64, None, 0, 1.0, 0, 0, None) == 1
    assert P._lib.pi_kv_fork(None, None, None, 1, None) == 1
    assert P._lib.pi_kv_free(None, None, 1, None) == 1
    assert P._lib.pi_kv_trim(None, None, 1, 1, 0, None) == 1
    assert P._lib.pi_kv_copy_pages(None, None, None, 1, None) == 1
    assert P._lib.pi_kv_compact(None, None, None) == 1
    P._lib.pi_kv_destroy(None)


def test_e4m3_values():
    assert TABLE[0x38] == 1.0 and TABLE[0x7e] == 448.0 and TABLE[1] == 2.0 ** -9 and TABLE[8] == 2.0 ** -6
    assert math.isnan(TABLE[0x7f]) and math.isnan(TABLE[0xff]) and TABLE[0xb8] == -1.0
    x = np.array([1.0, 1.0625, 1.1875, 464.0, 1e9, -2.0 ** -10, 2.0 ** -10 * 1.01, -0.0, np.nan, np.inf])
    assert list(encode(x)) == [0x38, 0x38, 0x3a, 0x7e, 0x7e, 0x80, 0x01, 0x80, 0x7f, 0x7e]
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    assert np.array_equal(encode(TABLE[codes]), codes)


def test_block_scales():
    assert block_scale(448.0) == 1.0 and block_scale(448.1) == 2.0 and block_scale(224.0) == 0.5
    assert block_scale(0.0) == 2.0 ** -120 and block_scale(1e-45) == 2.0 ** -120


def test_plain_attention_by_hand():
    c = PlainCache(1, 1, 1, 2, 2, 4, 1, 3)
    c.reserve([0], [3])
    k = np.array([[[0.0, 0.0]], [[math.log(2), 0.0]], [[0.0, 0.0]]])
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[4.0, 4.0]]])
    c.append(0, [0], [3], k, v)
    kk = TABLE[c.k[0, c.table[0, 0], 0, 1, 0]] * c.ks[0, c.table[0, 0], 0]      # the rounded log 2
    out, lse = c.attend(0, [0], [3], np.ones((3, 1, 2)), 1.0)
    w = math.exp(kk)
    assert np.allclose(out[:, 0], [[1, 0], [1 / (1 + w), w / (1 + w)],
                                   [(1 + 4) / (2 + w), (w + 4) / (2 + w)]])
    assert np.allclose(lse[:, 0], [0, math.log(1 + w), math.log(2 + w)])
    out, _ = c.attend(0, [0], [3], np.ones((3, 1, 2)), 1.0, window=1, sinks=1)
    assert np.allclose(out[:, 0], [[1, 0], [1 / (1 + w), w / (1 + w)], [2.5, 2]])


def test_plain_pages_by_hand():
    c = PlainCache(1, 1, 1, 2, 2, 6, 3, 4)
    c.reserve([0, 1], [3, 2])
    assert c.table[0].tolist() == [0, 1, -1, -1] and c.table[1].tolist() == [2, -1, -1, -1]
    c.fork([0], [2])
    assert c.table[2].tolist() == [0, 3, -1, -1] and c.ref.tolist() == [2, 1, 1, 1, 0, 0]
    c.free(0)
    assert c.ref.tolist() == [1, 0, 1, 1, 0, 0]
    assert c.compact() == 3 and c.table[2].tolist() == [0, 1, -1, -1] and c.ref.tolist() == [1, 1, 1, 0, 0, 0]
    c.trim(2, 1, 0)
    assert c.table[2].tolist() == [-1, 1, -1, -1]
