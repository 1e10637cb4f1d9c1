"""CPU oracle for the 4-bit key/value cache and the attention over it.

TEST INFRASTRUCTURE ONLY. Only tests/, __graft_entry__.smoke() and bench.py's
cpu_baseline / reference leg may import or call anything under oracle/.

Format (include/kv4_b200.h): blocks of 16 consecutive values of a row share one E4M3 scale
s; a value is an E2M1 code; it reads back as code * s * 2^e.
  * y = x * 2^-e;  s = E4M3(max |y| / 6) clamped to [2^-9, 448];  code = E2M1(y / s),
    both round-to-nearest-even, the code saturating;
  * a block that holds a NaN has scale byte 0x7F and zero codes, and reads back as NaN.
The quotients are taken in fp64 here and in fp32 by the kernels. Both round alike: a 16-bit
y has at most 11 significant bits and s at most 4, a rounding border t of E2M1 at most 3,
so y / s is either exactly t or differs from it by a relative 2^-11 at least (y and t s are
multiples of a common unit), far more than an fp32 quotient's 2^-24; and max|y| / 6 against
a border of E4M3 (5 significant bits) the same way.

Pinned by tests/test_kv4_oracle_pins.py.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_decode, e4m3_encode

BLOCK = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_encode(x):
    """Codes 0..15 of real x: nearest value, ties to the even code, saturating at 6."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)
    dist = np.abs(a[..., None] - E2M1)
    best = dist.min(-1, keepdims=True)
    hit = dist == best
    even = hit & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True), even, hit)
    return (pick.argmax(-1) + 8 * (np.signbit(x))).astype(np.uint8)


def e2m1_decode(code):
    code = np.asarray(code, dtype=np.uint8)
    return np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]


def kv4_quantize(x, e=0):
    """x: [..., d] values. Returns (packed codes uint8 [..., d / 2], scale bytes uint8 [..., d / 16])."""
    x = np.asarray(x, dtype=np.float64)
    y = (x * 2.0 ** -e).reshape(x.shape[:-1] + (-1, BLOCK))
    nan = np.isnan(y).any(-1)
    y = np.where(nan[..., None], 0.0, y)
    want = np.clip(np.abs(y).max(-1) / 6.0, 2.0 ** -9, 448.0)
    byte = e4m3_encode(want)
    s = e4m3_decode(byte)
    with np.errstate(invalid="ignore"):
        code = e2m1_encode(y / s[..., None]).reshape(x.shape)
    code = np.where(np.repeat(nan, BLOCK, -1), 0, code).astype(np.uint8)
    byte = np.where(nan, 0x7F, byte).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte


def kv4_dequantize(codes, sf, e=0):
    """fp64 values of packed codes [..., d / 2] and scale bytes [..., d / 16]."""
    codes, sf = np.asarray(codes, dtype=np.uint8), np.asarray(sf, dtype=np.uint8)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(sf.shape + (BLOCK,))
    s = np.where(sf == 0x7F, np.nan, e4m3_decode(np.where(sf == 0x7F, 0, sf)))
    v = e2m1_decode(c) * s[..., None] * 2.0 ** e
    return v.reshape(codes.shape[:-1] + (2 * codes.shape[-1],))


def kv4_rows(pages, block_table, page_size, first, last):
    """Rows [H, last - first, w] of positions [first, last) of one sequence: `pages`
    [num_pages, H, page_size, w], block_table [max_pages]."""
    pos = np.arange(first, last)
    return pages[np.asarray(block_table)[pos // page_size], :, pos % page_size].transpose(1, 0, 2)


def kv4_attention(q, k, v, q_len, causal, scale):
    """One sequence. q [Hq, N, d], k and v [Hkv, L, d] fp64 (the values read back).
    Returns O [Hq, q_len, d] and LSE [Hq, q_len]; a row without keys: 0 and -inf. A masked
    key takes no part, whatever it holds."""
    Hq, _, d = q.shape
    Hkv, L, _ = k.shape
    o = np.zeros((Hq, q_len, d))
    lse = np.full((Hq, q_len), -np.inf)
    for h in range(Hq):
        kh, vh = k[h // (Hq // Hkv)], v[h // (Hq // Hkv)]
        for i in range(q_len):
            n = max(0, L - q_len + i + 1) if causal else L
            if n == 0:
                continue
            s = scale * (kh[:n] @ q[h, i])
            m = s.max()
            p = np.exp(s - m)
            o[h, i] = (p / p.sum()) @ vh[:n]
            lse[h, i] = m + np.log(p.sum())
    return o, lse
