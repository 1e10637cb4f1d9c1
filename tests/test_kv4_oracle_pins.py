"""Pins of the 4-bit cache oracle (CPU): the format's tables and rounding worked by hand,
its invariants, and the attention against a direct softmax."""
import numpy as np
import pytest

from oracle.kv4 import (E2M1, e2m1_decode, e2m1_encode, kv4_attention, kv4_dequantize, kv4_quantize, kv4_rows)


def test_e2m1_table_and_rounding():
    assert e2m1_decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert (e2m1_encode(e2m1_decode(np.arange(1, 8))) == np.arange(1, 8)).all()
    # borders: ties go to the even code (0, 1, 2, 4 in value)
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for v, c in ties.items():
        assert e2m1_encode(v) == c and e2m1_encode(-v) == c + 8
        assert e2m1_encode(np.nextafter(v, 0)) <= c and e2m1_encode(np.nextafter(v, 9)) >= c
    assert e2m1_encode(100.0) == 7 and e2m1_encode(-np.inf) == 15


def test_block_worked_by_hand():
    # max 6 -> s = 1 (E4M3 byte 0x38); codes are the values' own
    x = np.array([6, -6, 3, -3, .5, .25, .76, 0, 1, 1.5, 2, 4, 5, -5, 2.5, 3.5])
    codes, sf = kv4_quantize(x)
    assert sf.tolist() == [0x38]
    assert kv4_dequantize(codes, sf).tolist() == [6, -6, 3, -3, .5, 0, 1, 0, 1, 1.5, 2, 4, 4, -4, 2, 4]
    assert codes[0] == (7 | 15 << 4) and codes[1] == (5 | 13 << 4)       # low nibble first
    # the exponent scales exactly
    c2, s2 = kv4_quantize(x * 2.0 ** -7, e=-7)
    assert (c2 == codes).all() and (s2 == sf).all()
    # limits: an all-zero block has the smallest scale; large values saturate; a NaN takes its block
    assert kv4_quantize(np.zeros(16))[1].tolist() == [1]
    c, s = kv4_quantize(np.array([1e9] + [0.0] * 15))
    assert s.tolist() == [0x7E] and kv4_dequantize(c, s)[0] == 2688
    c, s = kv4_quantize(np.array([np.nan] + [1.0] * 31))
    assert s[0] == 0x7F and np.isnan(kv4_dequantize(c, s)[:16]).all()
    assert (kv4_dequantize(c, s)[16:] == 6 * 0.171875).all()        # 1 / 6 lies nearest to E4M3's 11 * 2^-6


@pytest.mark.parametrize("d", [64, 128])
def test_error_bound_and_idempotence(d):
    g = np.random.default_rng(d)
    x = g.standard_normal((50, d)) * np.exp(g.standard_normal((50, 1)))
    c, s = kv4_quantize(x)
    v = kv4_dequantize(c, s)
    # E2M1's widest gap is 4..6 (half: 1) and the scale rounds by at most 1/16, so a value is off by at
    # most max|x| / 6 * 17/16, plus what saturates: 6.4 / 6 - 1 of the maximum when s rounds down
    amax = np.abs(x).reshape(50, -1, 16).max(-1).repeat(16, -1)
    assert (np.abs(v - x) <= amax / 6 * 17 / 16 + 1e-12).all()
    # 6 significant bits
    m, _ = np.frexp(v)
    assert (m * 64 == np.rint(m * 64)).all()


def test_attention_against_direct_softmax():
    g = np.random.default_rng(3)
    q, k, v = g.standard_normal((4, 3, 64)), g.standard_normal((2, 9, 64)), g.standard_normal((2, 9, 64))
    o, lse = kv4_attention(q, k, v, 3, True, 0.125)
    for h in range(4):
        s = 0.125 * q[h] @ k[h // 2].T
        s[np.arange(9) > np.array([6, 7, 8])[:, None]] = -np.inf
        p = np.exp(s) / np.exp(s).sum(1, keepdims=True)
        assert np.allclose(o[h], p @ v[h // 2]) and np.allclose(lse[h], np.log(np.exp(s).sum(1)))
    o, lse = kv4_attention(q, k[:, :1], v[:, :1], 3, True, 0.125)       # two rows stand before the first key
    assert (o[:, :2] == 0).all() and np.isneginf(lse[:, :2]).all() and np.allclose(o[:, 2], v[[0, 0, 1, 1], 0])
    assert len(E2M1) == 8


def test_rows_of_pages():
    pages = np.arange(5 * 2 * 4 * 3).reshape(5, 2, 4, 3)
    r = kv4_rows(pages, [3, 0, 4], 4, 2, 9)
    assert r.shape == (2, 7, 3)
    assert (r[1, 0] == pages[3, 1, 2]).all() and (r[0, 2] == pages[0, 0, 0]).all() and (r[1, 6] == pages[4, 1, 0]).all()
