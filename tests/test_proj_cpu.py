"""Projections and rotation without a GPU: bad arguments are refused before CUDA is touched, frequencies become turns
exactly, and the plain forms that the GPU tests compare with are pinned to hand-made values."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from tests import proj_plain as plain


@pytest.fixture(scope="module")
def P():
    import __graft_entry__

    __graft_entry__.build()
    import activation_sparse_decode_pi_gb300 as P

    return P


@pytest.mark.parametrize("n,k,rows,ld_x,ld_y,dtype,code", [
    (0, 128, 1, 128, 1, 0, 1), (1, 0, 1, 128, 1, 0, 1), (1, 128, -1, 128, 1, 0, 1), (1, 128, 257, 128, 1, 0, 1),
    (1, 128, 1, 128, 1, 3, 1), (1, 128, 1, 128, 1, -1, 1), (4, 64, 1, 64, 4, 0, 2), (4, 200, 1, 200, 4, 0, 2),
    (4, 128, 2, 127, 4, 0, 1), (4, 128, 2, 128, 3, 0, 1), (4, 128, 2, 130, 4, 0, 1), (4, 128, 2, 132, 4, 1, 1),
    (4, 128, 2, 1 << 62, 4, 0, 1), (4, 128, 2, 128, 1 << 62, 0, 1),
    (4, 128, 0, 128, 4, 0, 0),
])
def test_int4_linear_refusals(P, n, k, rows, ld_x, ld_y, dtype, code):
    assert P._lib.pi_int4_linear(None, None, None, n, k, None, ld_x, rows, None, 0, None, ld_y, dtype, None) == code


GOOD = dict(turns=None, rot_dim=0, interleaved=0, norm=0, amp=1.0, eps=1e-6)


@pytest.mark.parametrize("fields,tokens,heads,dim,dtype", [
    (dict(rot_dim=-16), 1, 1, 64, 0), (dict(rot_dim=80), 1, 1, 64, 0), (dict(interleaved=2), 1, 1, 64, 0),
    (dict(norm=-1), 1, 1, 64, 0), (dict(amp=math.inf), 1, 1, 64, 0), (dict(amp=math.nan), 1, 1, 64, 0),
    (dict(norm=1, eps=-1.0), 1, 1, 64, 0), (dict(norm=1, eps=math.nan), 1, 1, 64, 0), ({}, -1, 1, 64, 0),
    ({}, (1 << 30) + 1, 1, 64, 0), ({}, 1, -1, 64, 0), ({}, 1, 1, 0, 0), ({}, 1, 1, 64, 3),
])
def test_rotate_refusals(P, fields, tokens, heads, dim, dtype):
    """PI_ERR_INVALID_ARG, or without a driver PI_ERR_CUDA where the sizes are fine and only a device could tell."""
    r = P.PiRotary(**{**GOOD, **fields})
    code = P._lib.pi_rotate(ctypes.byref(r), None, tokens, heads, 0, dim, None, 64, None, 64, None, 0, None, 0, dtype, None)
    assert code == 1 or (fields and code == 3)
    assert P._lib.pi_rotate(ctypes.byref(P.PiRotary(**GOOD)), None, 1, 1, 0, 96, None, 96, None, 96, None, 0, None, 0, 0, None) == 2


def test_null_handle(P):
    r = P.PiRotary(**GOOD)
    assert P._lib.pi_kv_append_rotated(None, 0, None, None, 1, 1, ctypes.byref(r), None, 64, None, 64, None, None, 64, 0, None) == 1


def test_null_handle_of_shared_attention(P):
    assert P._lib.pi_kv_share(None, None, None, 1, None, 1, None, None) == 1
    assert P._lib.pi_kv_attend_shared(None, 0, None, None, 1, 1, None, 1, None, 64, None, 64, None, 0, 1.0, None, None) == 1


def test_turns(P):
    freq = [1.0, 0.5, 1e4 ** -0.7, 5e-324, 3e-6, 2 * math.pi, 1e300, 0.0, -0.25]
    for f, got in zip(freq, P.rotary_turns(freq)):
        want = round(Fraction(f) / (2 * plain.PI) * 2 ** 64) if abs(f) < 1e200 else None
        if want is not None:
            assert got == want % (1 << 64), f
    assert P.rotary_turns([]) == []


def test_frequencies(P):
    f = P.rotary_frequencies(8, 100.0)
    assert np.allclose(f, [1, 100 ** -0.25, 0.1, 100 ** -0.75])
    assert np.allclose(P.rotary_frequencies(8, 100.0, stretch=4.0), np.array(f) / 4)
    turns = 1000 * np.array(f) / (2 * math.pi)                      # 159, 50, 16, 5
    part = P.rotary_frequencies(8, 100.0, stretch=4.0, trained=1000, slow=10.0, fast=100.0)
    keep = np.clip((turns - 10) / 90, 0, 1)
    assert keep[0] == 1 and 0 < keep[1] < 1 and keep[3] == 0
    assert np.allclose(part, np.array(f) * (keep + (1 - keep) / 4))


def test_plain_int4_by_hand():
    w = np.zeros((2, 128), np.uint8)
    w[0, 0], w[0, 64], w[1, 127] = 0x81, 0x0f, 0x70      # elements 0, 1; 128; 255
    v = plain.int4_values(w, np.array([[2.0, 0.5], [1.0, 4.0]], np.float16))
    assert v[0, :2].tolist() == [2.0, -16.0] and v[0, 128] == -0.5 and v[1, 255] == 28.0 and np.abs(v).sum() == 46.5


def test_plain_rotation_by_hand():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = math.pi / 2
    y, size = plain.rotate(x, [quarter, 2 * quarter], [1], amp=2.0)
    assert np.allclose(y[0, 0], [-6, -4, 2, -8, 5, 6, 7, 8]) and size[0, 0, 0] == 8 and size[0, 0, 7] == 8
    y, _ = plain.rotate(x, [quarter, 2 * quarter], [1], interleaved=True)
    assert np.allclose(y[0, 0], [-2, 1, -3, -4, 5, 6, 7, 8])
    y, _ = plain.rotate(x, [], [5], norm=True, weight=np.full(8, 3.0), eps=0.0)
    assert np.allclose(y[0, 0], np.arange(1, 9) * 3 / math.sqrt(204 / 8))
    far = plain.angles([1.0], [2 ** 31 - 1])[0, 0]
    assert abs(math.sin(far) - math.sin(2 ** 31 - 1)) < 1e-12
