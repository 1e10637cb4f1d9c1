"""The 4-bit cache calls on the GPU against the fp64 oracle.

append and read are exact: codes, scale bytes and values are compared bit for bit.

Attention tolerance, from the arithmetic (every cached value is exact on both sides):
  * scores: q is exact in f16 up to 2^-34 of its row's largest value; products exact; fp32
    accumulation over d terms on the tensor cores, each step off by at most 2^-23 of the
    running magnitude: |dS| <= ds = (d + 8) 2^-23 scale sum_c |q_c k_c| (the largest over the keys)
    plus 2^-22 |S| for the multiplication by scale and the base change;
  * exp2 2^-22, P rounded to f16: 2^-11 of P, or 2^-25 absolute below f16's normal range
    (P is at most 2^8 and the row's largest P at least 1);
  * sums in fp32: at most (L / 8 + 64) additions in a row, 2^-24 each;
  * O rounded once: half a step of its type.
So with A = sum_j p_j |v_j| / l:
    |O - ref| <= eps/2 |ref| + (2^-11 + 2 ds' + 2^-21 + 2 (L/8 + 64) 2^-24) A + L 2^-25 max|v|
    |LSE - ref| <= ds' + (L/8 + 64) 2^-24 + 2^-21 + 2^-22 |ref|
with ds' = ds + 2^-22 max|S|.
"""
import math
import os
import threading

import numpy as np
import pytest
import torch

from oracle.kv4 import kv4_attention, kv4_dequantize, kv4_quantize, kv4_rows

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def n64(t):
    return t.double().cpu().numpy()


@pytest.fixture(params=["tight", "room"])
def room(request):
    """Block tables as long as the sequences need, and with room for 2^18 more tokens (unset entries): above 32
    rows of a cached head, the two take different kernels at these sizes."""
    Paged.room = request.param == "room"
    yield Paged.room
    Paged.room = False


class Paged:
    """A cache whose pages lie in random order, every unused byte 0xFF (NaN scales, -6 codes)."""

    room = False

    def __init__(self, lib, B, H, d, page, max_pages, k_exp=0, v_exp=0, seed=0, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.lib, self.B, self.H, self.d, self.page, self.max_pages = lib, B, H, d, page, max_pages
        P = B * max_pages + spare
        self.cache = lib.KV4Cache.allocate(P, H, page, d, k_exp=k_exp, v_exp=v_exp)
        for t in self.tensors():
            t.fill_(0xFF)
        self.bt = torch.randperm(P, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32).to(DEV)
        if self.room:
            more = torch.full((B, (1 << 18) // page), -1, dtype=torch.int32, device=DEV)
            self.bt = torch.cat([self.bt, more], 1).contiguous()
            self.max_pages = self.bt.shape[1]

    def tensors(self):
        c = self.cache
        return c.k_codes, c.k_sf, c.v_codes, c.v_sf

    def values(self, b, n):
        """fp64 K, V [H, n, d] of the first n positions, from the cache's bytes."""
        c, bt = self.cache, self.bt[b].cpu().numpy()
        out = []
        for codes, sf, e in ((c.k_codes, c.k_sf, c.k_exp), (c.v_codes, c.v_sf, c.v_exp)):
            out.append(kv4_dequantize(kv4_rows(codes.cpu().numpy(), bt, self.page, 0, n),
                                      kv4_rows(sf.cpu().numpy(), bt, self.page, 0, n), e))
        return out


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def fill(pg, lens, dt, seed, k_std=1.0, v_std=1.0):
    """Appends lens[b] random tokens to each sequence in one call; returns the 16-bit K, V."""
    g = torch.Generator().manual_seed(seed)
    N = max(1, max(lens))
    k = (torch.randn((pg.B, pg.H, N, pg.d), generator=g) * k_std).to(dt).to(DEV)
    v = (torch.randn((pg.B, pg.H, N, pg.d), generator=g) * v_std).to(dt).to(DEV)
    pg.lib.kv4_append(pg.cache, k, v, pg.bt, ints(lens), new_lens=ints(lens), check=True)
    return k, v


def check_attention(o, lse, q, pg, lens, qlens, causal, scale=None, rows=None):
    eps = torch.finfo(o.dtype).eps
    scale = 1 / math.sqrt(pg.d) if scale is None else scale
    o64, l64, q64 = n64(o), n64(lse), n64(q)
    for b in range(pg.B):
        L, n = lens[b], qlens[b]
        k, v = pg.values(b, L)
        ro, rl = kv4_attention(q64[b], k, v, n, causal, scale)
        G = q64.shape[1] // pg.H
        for h in range(q64.shape[1]):
            for i in (range(n) if rows is None else [r for r in rows if r < n]):
                vis = max(0, L - n + i + 1) if causal else L
                if vis == 0:
                    assert (o64[b, h, i] == 0).all() and np.isneginf(l64[b, h, i])
                    continue
                kk, vv = k[h // G][:vis], v[h // G][:vis]
                s = scale * kk @ q64[b, h, i]
                p = np.exp(s - rl[h, i])
                ds = (pg.d + 8) * 2.0 ** -23 * scale * (np.abs(kk) @ np.abs(q64[b, h, i])).max() + 2.0 ** -22 * np.abs(s).max()
                add = (vis / 8 + 64) * 2.0 ** -24
                bound = eps / 2 * np.abs(ro[h, i]) + (2.0 ** -11 + 2 * ds + 2.0 ** -21 + 2 * add) * (p @ np.abs(vv)) \
                    + vis * 2.0 ** -25 * np.abs(vv).max()
                err = np.abs(o64[b, h, i] - ro[h, i])
                assert (err <= bound).all(), (b, h, i, err.max(), (err / bound).max())
                lerr, lb = abs(l64[b, h, i] - rl[h, i]), ds + add + 2.0 ** -21 + 2.0 ** -22 * abs(rl[h, i])
                assert lerr <= lb, (b, h, i, lerr, lb)


# ---------------------------------------------------------------- append and read
@pytest.mark.parametrize("d,page,dt,N,lens,new,exps", [
    (128, 16, torch.bfloat16, 1, [1], [1], (0, 0)),                       # the first token of a sequence
    (128, 16, torch.float16, 1, [17, 16, 33], [1, 1, 1], (0, 0)),         # either side of a page border
    (64, 16, torch.bfloat16, 5, [5, 19], [5, 5], (-3, 2)),                # across a page border
    (64, 32, torch.float16, 37, [37, 101, 0], [37, 20, 0], (0, -5)),      # ragged, an empty sequence
    (128, 64, torch.bfloat16, 130, [130, 255], [0, 130], (4, 0)),         # nothing new for one of them
])
def test_append_is_exact_and_writes_nothing_else(cuda_lib, d, page, dt, N, lens, new, exps):
    lib, B, H = cuda_lib, len(lens), 3
    pg = Paged(lib, B, H, d, page, -(-max(max(lens), 1) // page), *exps, seed=N)
    g = torch.Generator().manual_seed(d + N)
    k, v = ((torch.randn((B, H, N, d), generator=g) * torch.exp(2 * torch.randn((B, H, N, 1), generator=g))).to(dt)
            for _ in range(2))
    want = [t.cpu().numpy().copy() for t in pg.tensors()]
    for b in range(B):
        for x, at, e in ((k, 0, exps[0]), (v, 2, exps[1])):
            c, s = kv4_quantize(n64(x[b]), e)
            for i in range(new[b]):
                p = lens[b] - new[b] + i
                pid = int(pg.bt[b, p // page])
                want[at][pid, :, p % page] = c[:, i]
                want[at + 1][pid, :, p % page] = s[:, i]
    lib.kv4_append(pg.cache, k.to(DEV), v.to(DEV), pg.bt, ints(lens),
                   new_lens=None if new == [N] * B else ints(new), check=True)
    for t, w in zip(pg.tensors(), want):
        assert (t.cpu().numpy() == w).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_append_at_the_rounding_borders(cuda_lib, dt):
    """Blocks whose quotients lie on and next to the borders of E2M1 and E4M3, zeros, infinities, NaN,
    the largest and the smallest values of the type."""
    lib, d = cuda_lib, 128
    one = torch.finfo(dt)
    rows = []
    g = torch.Generator().manual_seed(5)
    for _ in range(64):
        s = 2.0 ** int(torch.randint(-8, 8, (1,), generator=g)) * (8 + int(torch.randint(0, 8, (1,), generator=g))) / 8
        base = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]) * s
        up = (base * (1 + one.eps)).to(dt).float()
        down = (base * (1 - one.eps)).to(dt).float()
        up[0] = down[0] = base[0]
        amax = torch.full((16,), 0.5) * s
        amax[3] = 6 * s * (1 + 1 / 16)                                       # max / 6 between two scales
        rows.append(torch.cat([base, up, down, amax, torch.zeros(16), base * 2.0 ** -9,
                               base.flip(0), torch.full((16,), float(one.tiny))]))
    x = torch.stack(rows).to(dt)
    x[0, 5], x[1, 20], x[1, 21], x[2, 40] = float("inf"), float("nan"), float("inf"), float("-inf")
    x[3, :16], x[4, :16] = one.max, -one.max
    x[5, :16] = float("nan")
    N = x.shape[0]
    pg = Paged(lib, 1, 1, d, 16, 4)
    lib.kv4_append(pg.cache, x.view(1, 1, N, d).to(DEV), x.flip(0).contiguous().view(1, 1, N, d).to(DEV), pg.bt,
                   ints([N]), check=True)
    got = [kv4_rows(t.cpu().numpy(), pg.bt[0].cpu().numpy(), 16, 0, N)[0] for t in pg.tensors()]
    for xs, c, s in ((x, got[0], got[1]), (x.flip(0), got[2], got[3])):
        wc, ws = kv4_quantize(n64(xs))
        assert (s == ws).all()
        assert (kv4_dequantize(c, s)[~np.isnan(kv4_dequantize(c, s))] ==
                kv4_dequantize(wc, ws)[~np.isnan(kv4_dequantize(wc, ws))]).all()
        assert (c == wc).all() or (np.isin(c ^ wc, [0, 0x08, 0x80, 0x88]).all())     # at most the sign of a zero
    k, v = lib.kv4_read(pg.cache, pg.bt, ints([N]), N, dtype=torch.bfloat16, check=True)
    assert np.array_equal(n64(k)[0, 0], kv4_dequantize(got[0], got[1]), equal_nan=True)
    assert np.array_equal(n64(v)[0, 0], kv4_dequantize(got[2], got[3]), equal_nan=True)


@pytest.mark.parametrize("d,page,dt,lens,starts,N,exps", [
    (128, 16, torch.bfloat16, [1], None, 1, (0, 0)),
    (128, 16, torch.float16, [40, 17, 0], [3, 16, 0], 30, (0, 0)),         # past the end, nothing at all
    (64, 16, torch.bfloat16, [100, 63], [99, 0], 64, (-20, 17)),
    (64, 128, torch.float16, [300, 129], [200, 128], 100, (1, -3)),
])
def test_read_is_exact(cuda_lib, d, page, dt, lens, starts, N, exps):
    lib, B = cuda_lib, len(lens)
    pg = Paged(lib, B, 2, d, page, -(-max(lens) // page), *exps, seed=1)
    fill(pg, lens, torch.bfloat16, 7, 2.0 ** exps[0], 2.0 ** exps[1])
    k, v = lib.kv4_read(pg.cache, pg.bt, ints(lens), N, starts=None if starts is None else ints(starts), dtype=dt,
                        check=True)
    for b in range(B):
        s = 0 if starts is None else starts[b]
        m = max(0, min(N, lens[b] - s))
        for got, want in zip((k, v), pg.values(b, lens[b])):
            want = torch.from_numpy(want[:, s:s + m]).to(dt)              # one rounding
            assert torch.equal(got[b, :, :m].cpu(), want) and not got[b, :, m:].any()


# ---------------------------------------------------------------- attention
ATTN_CASES = [
    # d, Hq, Hkv, page, dt, N, lens, q_lens, causal, exps
    (128, 4, 1, 16, torch.bfloat16, 1, [1], None, False, (0, 0)),
    (128, 8, 2, 16, torch.float16, 1, [7, 33, 300], None, False, (0, 0)),
    (64, 3, 3, 32, torch.bfloat16, 1, [0, 64, 129, 513], None, True, (0, -4)),          # an empty sequence, no grouping
    (128, 16, 1, 64, torch.bfloat16, 1, [1000, 257], None, False, (-6, 3)),
    (64, 14, 2, 16, torch.float16, 1, [70, 31], None, False, (0, 0)),                   # 7 to a head
    (128, 8, 2, 16, torch.bfloat16, 3, [3, 50, 600], None, True, (0, 0)),
    (128, 8, 1, 16, torch.float16, 4, [5, 900], [4, 2], True, (0, 0)),                  # padded queries
    (64, 6, 2, 16, torch.bfloat16, 5, [40, 3, 700], [5, 5, 0], True, (0, 0)),           # more queries than keys
    (128, 4, 4, 32, torch.float16, 33, [400, 70], [33, 17], True, (0, 0)),
    (128, 4, 2, 16, torch.bfloat16, 130, [130, 515], [130, 129], True, (0, 0)),
    (64, 4, 1, 128, torch.float16, 100, [777, 100], [100, 100], False, (2, 0)),
    (128, 5, 5, 16, torch.bfloat16, 257, [300], None, True, (0, 0)),
    (64, 8, 8, 16, torch.bfloat16, 65, [65, 64, 200], [65, 64, 1], True, (0, 0)),
    (128, 2, 1, 65536, torch.float16, 200, [1025], None, True, (0, 0)),                 # one page holds everything
    (64, 6, 3, 16, torch.bfloat16, 300, [310, 900], [300, 7], True, (0, 0)),            # more rows than a tile has keys
    (128, 6, 2, 16, torch.float16, 7, [600, 5], None, True, (0, 0)),                    # 21 rows
    (128, 4, 2, 32, torch.bfloat16, 300, [40, 0, 299], [300, 300, 299], True, (0, 0)),  # rows before the first key
]


def make_q(B, Hq, N, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, Hq, N, d), generator=g)
    q[..., 0] *= 8.0
    return q.to(dt).to(DEV)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("d,Hq,Hkv,page,dt,N,lens,qlens,causal,exps", ATTN_CASES)
def test_attention(cuda_lib, d, Hq, Hkv, page, dt, N, lens, qlens, causal, exps):
    lib, B = cuda_lib, len(lens)
    pg = Paged(lib, B, Hkv, d, page, -(-max(lens) // page) + 1, *exps, seed=N, spare=0 if page > 1000 else 2)
    fill(pg, lens, dt, N + d, 2.0 ** exps[0], 2.0 ** exps[1])
    q = make_q(B, Hq, N, d, dt, 11 * N + d)
    if exps[0]:
        q = (q.float() * 2.0 ** -exps[0]).to(dt)
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, Hq, N), 7.0, device=DEV)
    lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), q_lens=None if qlens is None else ints(qlens), causal=causal,
                    out=out, lse=lse, check=True)
    ql = [N] * B if qlens is None else qlens
    check_attention(out, lse, q, pg, lens, ql, causal)
    for b in range(B):                                                    # rows behind the queries: as they were
        assert (out[b, :, ql[b]:] == 7).all() and (lse[b, :, ql[b]:] == 7).all()
    o2, l2 = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), q_lens=None if qlens is None else ints(qlens),
                             causal=causal, check=True)
    for b in range(B):                                                    # bit-identical when repeated
        assert torch.equal(o2[b, :, :ql[b]], out[b, :, :ql[b]]) and torch.equal(l2[b, :, :ql[b]], lse[b, :, :ql[b]])
        assert not o2[b, :, ql[b]:].any()
    o3, none = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), q_lens=None if qlens is None else ints(qlens),
                               causal=causal, with_lse=False, check=True)
    assert none is None and torch.equal(o3, o2)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("scale", [0.03, 1.0])
def test_attention_scale_and_long_rows(cuda_lib, scale):
    """A given scale; rows peaked on few keys (the running maximum moves often) and a longer cache."""
    lib, lens = cuda_lib, [3001, 64]
    pg = Paged(lib, 2, 2, 128, 16, 188, seed=9)
    fill(pg, lens, torch.bfloat16, 3, 2.0, 1.0)
    for N, rows in ((1, None), (48, (0, 1, 47)), (140, (0, 77, 139))):
        q = make_q(2, 4, N, 128, torch.bfloat16, N)
        o, lse = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), q_lens=ints([N, min(N, 64)]), causal=True, scale=scale,
                                 check=True)
        check_attention(o, lse, q, pg, lens, [N, min(N, 64)], True, scale, rows)


def test_extreme_queries(cuda_lib):
    """Query rows of very large, very small and mixed magnitude: a row is scaled by a power of two."""
    lib, d = cuda_lib, 128
    pg = Paged(lib, 1, 1, d, 16, 20, seed=2)
    fill(pg, [300], torch.bfloat16, 4)
    q = make_q(1, 6, 1, d, torch.bfloat16, 1)
    big = [1e30, 1e-30, 1.0, 0.0, 2.0 ** 100, 2.0 ** -120]
    for h, f in enumerate(big):
        q[0, h] *= f
    for h, f in enumerate(big):
        if f in (0.0,):
            continue
        sc = float(0.088 / f) if f != 0 else 0.088
        if not (1e-37 < sc < 1e37):
            continue
        o, lse = lib.forward_kv4(q[:, h:h + 1].contiguous(), pg.cache, pg.bt, ints([300]), scale=sc, check=True)
        check_attention(o, lse, q[:, h:h + 1], pg, [300], [1], False, float(np.float32(sc)))
    o, lse = lib.forward_kv4(q[:, 3:4].contiguous(), pg.cache, pg.bt, ints([300]), check=True)     # q = 0: the mean of V
    check_attention(o, lse, q[:, 3:4], pg, [300], [1], False)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("N,Hq", [(1, 4), (6, 2), (140, 1)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_in_the_cache(cuda_lib, N, Hq, which):
    """A NaN key or value makes the rows that see it NaN (at least the block it lies in) and no other row."""
    lib, L, d = cuda_lib, 400, 128
    for at in (L - N // 2 - 1, 10, L - 1):
        pg = Paged(lib, 1, 1, d, 16, 25, seed=3)
        g = torch.Generator().manual_seed(4)
        k, v = (torch.randn((1, 1, L, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        (k if which == "k" else v)[0, 0, at, 37] = float("nan")
        lib.kv4_append(pg.cache, k, v, pg.bt, ints([L]), check=True)
        q = make_q(1, Hq, N, d, torch.bfloat16, 5)
        o, lse = lib.forward_kv4(q, pg.cache, pg.bt, ints([L]), causal=True, check=True)
        sees = [i for i in range(N) if L - N + i >= at]
        blind = [i for i in range(N) if L - N + i < at]
        assert torch.isnan(o[0, :, sees, 32:48]).all()
        if blind:
            assert torch.isfinite(o[0, :, blind]).all() and torch.isfinite(lse[0, :, blind]).all()
            pg.cache.k_sf[pg.cache.k_sf == 0x7F] = 0x38                      # the same rows without the NaN
            pg.cache.v_sf[pg.cache.v_sf == 0x7F] = 0x38
            o2, l2 = lib.forward_kv4(q, pg.cache, pg.bt, ints([L]), causal=True, check=True)
            assert torch.equal(o[0, :, blind], o2[0, :, blind]) and torch.equal(lse[0, :, blind], l2[0, :, blind])


def test_bad_tables_are_reported_and_skipped(cuda_lib):
    """Page numbers and lengths outside the cache: recorded in the device status, nothing written
    outside, other sequences unaffected."""
    lib, d = cuda_lib, 128
    pg = Paged(lib, 3, 2, d, 16, 6, seed=6)
    lens = [90, 60, 33]
    fill(pg, lens, torch.bfloat16, 8)
    for N in (1, 5, 140):
        q = make_q(3, 4, N, d, torch.bfloat16, 9)
        good, gl = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), check=True)
        bad_bt = pg.bt.clone()
        bad_bt[1, 2] = 1 << 30
        for bt, sl, ql in ((bad_bt, lens, None), (pg.bt, [90, -5, 33], None), (pg.bt, [90, 97, 33], None),
                           (pg.bt, lens, [N, N + 1, N]), (pg.bt, lens, [N, -1, N])):
            if bt is bad_bt:
                bt[1, 2] = -bt[1, 2]
            o, lse = lib.forward_kv4(q, pg.cache, bt, ints(sl), q_lens=None if ql is None else ints(ql))
            torch.cuda.synchronize()
            assert lib.attn_get_device_status(None) == lib.ATTN_ERR_BOUNDS
            assert lib.attn_get_device_status(None) == lib.ATTN_OK
            for b in (0, 2):
                assert torch.equal(o[b], good[b]) and torch.equal(lse[b], gl[b])
    before = [t.clone() for t in pg.tensors()]
    k = torch.ones(3, 2, 2, d, dtype=torch.bfloat16, device=DEV)
    for sl, nl in (([0, 0, 0], None), ([97, 98, 1000], None), ([1, 1, 1], None)):
        lib.kv4_append(pg.cache, k, k, bad_bt if sl[0] > 90 else pg.bt, ints([-1, -1, -1]) if sl == [0, 0, 0] else ints(sl),
                       new_lens=nl)
        torch.cuda.synchronize()
        assert lib.attn_get_device_status(None) == lib.ATTN_ERR_BOUNDS
    lib.kv4_read(pg.cache, bad_bt, ints(lens), 60)
    torch.cuda.synchronize()
    assert lib.attn_get_device_status(None) == lib.ATTN_ERR_BOUNDS
    changed = [int((a != b).sum()) for a, b in zip(before, pg.tensors())]
    assert all(c < 3 * 2 * 4 * d for c in changed)          # only the valid clamped positions were written


def test_offsets_past_32_bits(cuda_lib):
    """Pages whose byte offsets need more than 32 bits."""
    lib, H, d, page = cuda_lib, 8, 128, 64
    P = (1 << 32) // (H * page * (d // 2)) + 40                           # 4.3 GB of key codes
    cache = lib.KV4Cache.allocate(P, H, page, d)
    pg = Paged.__new__(Paged)
    pg.lib, pg.B, pg.H, pg.d, pg.page, pg.max_pages, pg.cache = lib, 1, H, d, page, 3, cache
    pg.bt = ints([[P - 1, 5, P - 20]])
    cache_rows = [P - 1, 5, P - 20]
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((1, H, 150, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    lib.kv4_append(cache, k, v, pg.bt, ints([150]), check=True)
    rk, rv = lib.kv4_read(cache, pg.bt, ints([150]), 150, check=True)
    c, s = kv4_quantize(n64(k[0]))
    assert (n64(rk[0]) == kv4_dequantize(c, s)).all()
    c, s = kv4_quantize(n64(v[0]))
    assert (n64(rv[0]) == kv4_dequantize(c, s)).all()
    small = lib.KV4Cache(*(t[cache_rows].contiguous() for t in (cache.k_codes, cache.k_sf, cache.v_codes, cache.v_sf)))
    for N in (1, 6, 130):
        q = make_q(1, H, N, d, torch.bfloat16, 2)
        o, l = lib.forward_kv4(q, cache, pg.bt, ints([150]), causal=True, check=True)
        o2, l2 = lib.forward_kv4(q, small, ints([[0, 1, 2]]), ints([150]), causal=True, check=True)
        assert torch.equal(o, o2) and torch.equal(l, l2)


# ---------------------------------------------------------------- streams, graphs, a run of them together
@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("N,L", [(1, 2000), (4, 900), (150, 700)])
def test_streams_and_graphs(cuda_lib, N, L):
    """On a side stream; captured, with changed inputs and lengths at replay; two graphs replayed in
    turn and on two streams at once."""
    lib, d = cuda_lib, 128
    pg = Paged(lib, 2, 2, d, 16, 130, seed=1)
    fill(pg, [L, L - 77], torch.bfloat16, 2)
    lens = ints([L, L - 77])
    q = [make_q(2, 4, N, d, torch.bfloat16, s) for s in range(3)]
    want = [lib.forward_kv4(x, pg.cache, pg.bt, lens, causal=True, check=True) for x in q]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = lib.forward_kv4(q[0], pg.cache, pg.bt, lens, causal=True, stream=side, check=True)
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    graphs, outs, ins = [], [], []
    for s in range(2):
        x = q[s].clone()
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            y = lib.forward_kv4(x, pg.cache, pg.bt, lens, causal=True)
        graphs.append(gph)
        outs.append(y)
        ins.append(x)
    for s in range(2):
        graphs[s].replay()
    torch.cuda.synchronize()
    for s in range(2):
        assert torch.equal(outs[s][0], want[s][0]) and torch.equal(outs[s][1], want[s][1])
    ins[0].copy_(q[2])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                graphs[s].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want[2][0]) and torch.equal(outs[1][0], want[1][0])
    lens.fill_(L // 2)                                                   # the captured launch reads the new lengths
    graphs[0].replay()
    torch.cuda.synchronize()
    check = lib.forward_kv4(q[2], pg.cache, pg.bt, lens, causal=True, check=True)
    assert torch.equal(outs[0][0], check[0]) and torch.equal(outs[0][1], check[1])


def test_decoding_run(cuda_lib):
    """The calls together, as a decoding layer uses them: a prompt is written in two chunks that attend
    causally, then single tokens: W4A16 projections of the token, append, attention over the cache, W4A16
    output projection. Every step against the oracle on the cache's own bytes; at the end the cache holds
    exactly what the oracle quantises from all keys and values written."""
    import workloads
    lib, dt, B, Hq, Hkv, d, page = cuda_lib, torch.float16, 2, 4, 2, 128, 16
    D = Hq * d
    pg = Paged(lib, B, Hkv, d, page, 8, seed=12)
    g = torch.Generator().manual_seed(0)
    _, wqkv, sq, zq = workloads.make_w4a16(1, (Hq + 2 * Hkv) * d, D, seed=1)
    _, wo, so, zo = workloads.make_w4a16(1, D, D, seed=2)
    wqkv, sq, zq, wo, so, zo = (t.to(DEV) for t in (wqkv, sq * 0.3, zq, wo, so * 0.3, zo))
    lens = [0, 0]
    written = ([[], []], [[], []])

    def project(x):                                                      # [B, N, D] -> q, k, v [B, H, N, d]
        N = x.shape[1]
        y = lib.w4a16_matmul(x.reshape(B * N, D).contiguous(), wqkv, sq, zq).view(B, N, Hq + 2 * Hkv, d)
        y = y.transpose(1, 2)
        return tuple(t.contiguous() for t in (y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]))

    def step(x, new):
        q, k, v = project(x)
        for b in range(B):
            lens[b] += new[b]
            for w, t in zip(written, (k, v)):
                w[b].append(n64(t[b, :, :new[b]]))
        sl, nl = ints(lens), ints(new)
        lib.kv4_append(pg.cache, k, v, pg.bt, sl, new_lens=nl)
        o, lse = lib.forward_kv4(q, pg.cache, pg.bt, sl, q_lens=nl, causal=True, check=True)
        check_attention(o, lse, q, pg, lens, new, True)
        return lib.w4a16_matmul(o.transpose(1, 2).reshape(-1, D).contiguous(), wo, so, zo).view(B, -1, D)
    x = torch.randn((B, 40, D), generator=g).to(dt).to(DEV)
    step(x, [40, 23])
    x = step(torch.randn((B, 30, D), generator=g).to(dt).to(DEV), [30, 7])[:, :1]
    for _ in range(4):
        x = x / x.float().square().mean(-1, keepdim=True).sqrt().to(dt)
        x = step(x.contiguous(), [1, 1])
        assert torch.isfinite(x).all()
    for b in range(B):
        for w, (codes, sf) in zip(written, ((pg.cache.k_codes, pg.cache.k_sf), (pg.cache.v_codes, pg.cache.v_sf))):
            c, s = kv4_quantize(np.concatenate(w[b], 1))
            bt = pg.bt[b].cpu().numpy()
            assert (kv4_rows(codes.cpu().numpy(), bt, page, 0, lens[b]) == c).all()
            assert (kv4_rows(sf.cpu().numpy(), bt, page, 0, lens[b]) == s).all()


@pytest.mark.usefixtures("room")
def test_one_workspace_for_calls_of_every_shape(cuda_lib):
    """A caller's workspace, full of anything, used by calls of different shapes in turn: the results
    are those of the binding's own, and nothing behind the required size is written."""
    lib, d = cuda_lib, 128
    pg = Paged(lib, 3, 2, d, 16, 200, seed=8)
    lens = [3100, 900, 17]
    fill(pg, lens, torch.bfloat16, 6)
    small = Paged(lib, 1, 1, 64, 32, 40, seed=9)
    fill(small, [1200], torch.bfloat16, 7)
    jobs = [(pg, lens, 1, 4), (small, [1200], 1, 2), (pg, lens, 150, 2), (pg, lens, 5, 4), (small, [1200], 40, 2),
            (pg, lens, 40, 4), (small, [1200], 3, 5), (pg, lens, 1, 4)]
    need = [lib.attn_fwd_kv4_workspace_bytes(g.B, hq, g.H, N, g.d, g.page, g.max_pages) for g, _, N, hq in jobs]
    ws = torch.full((max(need) + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    for (g, ln, N, hq), nb in zip(jobs, need):
        q = make_q(g.B, hq, N, g.d, torch.bfloat16, N)
        want = lib.forward_kv4(q, g.cache, g.bt, ints(ln), causal=True, check=True)
        ws[nb:] = 0x5A
        o, lse = lib.forward_kv4(q, g.cache, g.bt, ints(ln), causal=True, workspace=ws, check=True)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert (ws[nb:] == 0x5A).all()
    with pytest.raises(ValueError):
        lib.forward_kv4(q, g.cache, g.bt, ints(ln), workspace=ws[:need[-1] - 1])


@pytest.mark.parametrize("N", [1, 3])
def test_many_sequences(cuda_lib, N):
    """More sequences than a warp has lanes, most of them short, some empty, one long."""
    lib, B, d = cuda_lib, 77, 64
    lens = [(7 * b * b + 3 * b) % 90 for b in range(B)]
    lens[50], lens[3], lens[76] = 1500, 0, 0
    pg = Paged(lib, B, 2, d, 16, 94, seed=N)
    fill(pg, lens, torch.float16, 5)
    q = make_q(B, 6, N, d, torch.float16, 3)
    o, lse = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), causal=True, check=True)
    check_attention(o, lse, q, pg, lens, [N] * B, True)
    big = make_q(B, 2, 150, d, torch.float16, 4)                 # chunks of all of them
    o, lse = lib.forward_kv4(big, pg.cache, pg.bt, ints(lens), q_lens=ints([min(150, x) for x in lens]), causal=True,
                             check=True)
    check_attention(o, lse, big, pg, lens, [min(150, x) for x in lens], True, rows=(0, 1, 40, 149))


@pytest.mark.usefixtures("room")
def test_debug_build_is_bit_identical(cuda_lib):
    """The debug build's cache calls give the release build's bits, and report a bad page with its site."""
    lib, d = cuda_lib, 128
    from exact_attention_forward_11_b200 import build
    assert os.path.exists(build.build(debug=True))
    lens = [400, 77]
    pg = Paged(lib, 2, 2, d, 16, 25, seed=4)
    k, v = fill(pg, lens, torch.bfloat16, 2)
    qs = [make_q(2, 4, N, d, torch.bfloat16, N) for N in (1, 7, 40, 150)]
    want = [lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), causal=True, check=True) for q in qs]
    codes = [t.clone() for t in pg.tensors()]
    read = lib.kv4_read(pg.cache, pg.bt, ints(lens), 300, check=True)
    prev = lib.use_library(lib.DEBUG_LIB_PATH)
    try:
        assert lib.attn_debug_build() == 1
        lib.kv4_append(pg.cache, k, v, pg.bt, ints(lens), new_lens=ints(lens), check=True)
        assert all(torch.equal(a, b) for a, b in zip(codes, pg.tensors()))
        assert all(torch.equal(a, b) for a, b in zip(read, lib.kv4_read(pg.cache, pg.bt, ints(lens), 300, check=True)))
        for q, w in zip(qs, want):
            o, lse = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), causal=True, check=True)
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
        bad = pg.bt.clone()
        bad[1, 1] = 12345678
        lib.forward_kv4(qs[0], pg.cache, bad, ints(lens))
        torch.cuda.synchronize()
        assert lib.attn_get_device_status(None) == lib.ATTN_ERR_BOUNDS
        assert lib.attn_debug_last_failure(None) == (12, 12345678)
    finally:
        lib.use_library(prev)


def test_offset_tables_and_odd_strides(cuda_lib):
    """int32 arguments that are slices of larger arrays (4-byte aligned), and a refused non-contiguous one."""
    lib, d = cuda_lib, 64
    lens = [33, 250, 90]
    pg = Paged(lib, 3, 2, d, 16, 16, seed=4)
    fill(pg, lens, torch.float16, 2)
    q = make_q(3, 2, 2, d, torch.float16, 1)
    want = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), q_lens=ints([2, 1, 2]), causal=True, check=True)
    sl, ql = ints([9] + lens)[1:], ints([9, 9, 9, 2, 1, 2])[3:]
    bt = torch.cat([pg.bt.new_zeros(1), pg.bt.view(-1)])[1:].view_as(pg.bt)
    got = lib.forward_kv4(q, pg.cache, bt, sl, q_lens=ql, causal=True, check=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError):
        lib.forward_kv4(q, pg.cache, pg.bt.t().contiguous().t(), ints(lens))
    with pytest.raises(ValueError):
        lib.forward_kv4(q, pg.cache, pg.bt, torch.stack([ints(lens), ints(lens)], 1)[:, 0])


@pytest.mark.parametrize("N,Hq", [(150, 4), (60, 4)])
def test_chunk_kernel_timeout_path(cuda_lib, N, Hq):
    """One CTA's first key tile is never handed out: its bounded waits run out, the launch ends by itself
    and reports ATTN_ERR_TIMEOUT once, whole sequences that other CTAs compute are exact, and the next
    ordinary call is exact."""
    lib, d, B = cuda_lib, 128, 40
    lens = [130 + 3 * b for b in range(B)]
    pg = Paged(lib, B, 2, d, 16, 16, seed=5)
    fill(pg, lens, torch.bfloat16, 3)
    q = make_q(B, Hq, N, d, torch.bfloat16, 2)
    want = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), check=True)
    o, lse = torch.zeros_like(q), torch.zeros((B, Hq, N), device=DEV)
    need = lib.attn_fwd_kv4_workspace_bytes(B, Hq, 2, N, d, 16, 16)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    sl = ints(lens)
    for fault in (0, 147, 60):
        st = lib.attn_fwd_kv4_inject_timeout(pg.cache._addr, q.data_ptr(), pg.bt.data_ptr(), sl.data_ptr(), None,
                                             o.data_ptr(), lse.data_ptr(), ws.data_ptr(), need, B, Hq, N, 16, 0.0, 0,
                                             lib.ATTN_BF16, fault, 1 << 22, torch.cuda.current_stream().cuda_stream)
        assert st == lib.ATTN_OK
        torch.cuda.synchronize()
        assert lib.attn_get_device_status(None) == lib.ATTN_ERR_TIMEOUT
        assert lib.attn_get_device_status(None) == lib.ATTN_OK
        same = [torch.equal(o[b], want[0][b]) and torch.equal(lse[b], want[1][b]) for b in range(B)]
        assert sum(same) >= B - 4, (fault, same)                 # a CTA's run covers at most a few sequences
        o.zero_(), lse.zero_()
    again = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), check=True)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("N,lens,H", [
    (1, [5000, 0, 4097, 257, 7000, 3000], 16),                      # runs of 4 to 5 tiles, items of 2 to 28
    (2, [5000, 0, 4097, 257, 7000, 3000], 16),                      # the same in blocks of 16 rows (q heads 6 a head)
    (1, [256 * (b % 4) + b for b in range(40)], 24),                # more sequences than lanes, items of 0 to 4 tiles
    (1, [(37 * b) % 512 for b in range(70)], 8),                    # whole items, two a CTA, the last CTA's one
    (5, [(53 * b) % 700 for b in range(31)], 3)])                   # whole items of 0 to 3 tiles, two blocks of rows
def test_long_runs(cuda_lib, N, lens, H):
    """Runs of several items: segments that start and end anywhere in an item, and runs of whole items."""
    lib, B, d = cuda_lib, len(lens), 64
    pg = Paged(lib, B, H, d, 64, (max(lens) + 63) // 64, seed=B)
    fill(pg, lens, torch.bfloat16, 9)
    q = make_q(B, 6 * H, N, d, torch.bfloat16, 8)
    o, lse = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), causal=True, check=True)
    check_attention(o, lse, q, pg, lens, [N] * B, True)


def test_threads_on_one_stream(cuda_lib):
    """Two host threads that call on one stream: each has its own workspace, since their launches may interleave."""
    lib, d = cuda_lib, 128
    torch.cuda.synchronize()
    pgs, qs, want = [], [], []
    for t, (B, N, lens) in enumerate([(3, 1, [1500, 40, 2100]), (2, 40, [700, 1300])]):
        pg = Paged(lib, B, 2, d, 16, (max(lens) + 15) // 16, seed=t)
        fill(pg, lens, torch.bfloat16, t)
        pgs.append((pg, ints(lens)))
        qs.append(make_q(B, 8, N, d, torch.bfloat16, t))
        want.append(lib.forward_kv4(qs[t], pg.cache, pg.bt, pgs[t][1], causal=True, check=True))
    got, places, both = [[], []], [None, None], threading.Barrier(2)

    def work(t):
        pg, lens = pgs[t]
        both.wait(60)
        for _ in range(200):
            got[t].append(lib.forward_kv4(qs[t], pg.cache, pg.bt, lens, causal=True))
        places[t] = lib._kv4_workspace(pg.cache, torch.cuda.current_stream().cuda_stream, 16).data_ptr()
        both.wait(60)                                              # (a thread's workspace is freed with it)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert None not in places and places[0] != places[1]
    for t in range(2):
        assert len(got[t]) == 200
        for o, lse in got[t]:
            assert torch.equal(o, want[t][0]) and torch.equal(lse, want[t][1])


def test_graph_with_copies_and_a_fork(cuda_lib):
    """Captured behind copies, a memset and another stream's append: every call waits for what it reads."""
    lib, d, lens = cuda_lib, 128, [1500, 900]
    pg, other = Paged(lib, 2, 2, d, 16, 100, seed=1), Paged(lib, 2, 2, d, 16, 100, seed=2)
    k, v = fill(pg, lens, torch.bfloat16, 2)
    q_from, q, n = make_q(2, 4, 1, d, torch.bfloat16, 3), torch.empty(2, 4, 1, d, dtype=torch.bfloat16, device=DEV), ints([0, 0])
    fill(other, lens, torch.bfloat16, 2)                                   # the expected result, from a second cache
    want = lib.forward_kv4(q_from, other.cache, other.bt, ints(lens), causal=True, check=True)
    for t in other.tensors():
        t.fill_(0xFF)
    src = ints(lens)
    side = torch.cuda.Stream()
    gph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        n.zero_()
        n.copy_(src)
        q.copy_(q_from)
        lib.kv4_append(other.cache, k, v, other.bt, src, new_lens=src, stream=side)
        first = lib.forward_kv4(q, pg.cache, pg.bt, n, causal=True)
        main.wait_stream(side)
        second = lib.forward_kv4(q, other.cache, other.bt, n, causal=True)
        kr, _ = lib.kv4_read(other.cache, other.bt, n, 1500)
        back = kr.clone()
    for _ in range(3):
        for t in (*other.tensors(), *first, *second, back):
            t.zero_()
        gph.replay()
        torch.cuda.synchronize()
        for o, lse in (first, second):
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(back, lib.kv4_read(pg.cache, pg.bt, src, 1500, check=True)[0])


@pytest.mark.parametrize("N", [40, 140])
def test_bad_tables_in_long_chunks(cuda_lib, N):
    """The same errors of tables and lengths in the kernel that long tables take."""
    lib, d, lens = cuda_lib, 128, [200, 160, 150]
    Paged.room = True
    try:
        pg = Paged(lib, 3, 2, d, 16, 13, seed=6)
    finally:
        Paged.room = False
    fill(pg, lens, torch.bfloat16, 8)
    q = make_q(3, 4, N, d, torch.bfloat16, 9)
    good, gl = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), check=True)
    bad_bt, missing = pg.bt.clone(), [200, 250, 150]                  # pages past 13 are unset (-1)
    bad_bt[1, 2] = 1 << 30
    for bt, sl, ql in ((bad_bt, lens, None), (pg.bt, [200, -5, 150], None), (pg.bt, missing, None),
                       (pg.bt, lens, [N, N + 1, N]), (pg.bt, lens, [N, -1, N])):
        o, lse = lib.forward_kv4(q, pg.cache, bt, ints(sl), q_lens=None if ql is None else ints(ql))
        torch.cuda.synchronize()
        assert lib.attn_get_device_status(None) == lib.ATTN_ERR_BOUNDS
        assert lib.attn_get_device_status(None) == lib.ATTN_OK
        for b in (0, 2):
            assert torch.equal(o[b], good[b]) and torch.equal(lse[b], gl[b])


def test_plans_agree(cuda_lib):
    """Short chunks with a tight table and with room (two kernels, three block heights): each within the
    tolerance, and every row written."""
    lib, d = cuda_lib, 128
    for N, Hq in ((40, 2), (100, 2), (300, 4), (12, 6)):
        lens = [N + 300, N, 3]
        pg = Paged(lib, 3, 2, d, 16, (N + 300 + 15) // 16, seed=N)
        fill(pg, lens, torch.bfloat16, N)
        wide = torch.cat([pg.bt, torch.full((3, 1 << 14), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
        q = make_q(3, Hq, N, d, torch.bfloat16, N)
        for bt in (pg.bt, wide):
            out, lse = torch.full_like(q, float("nan")), torch.full((3, Hq, N), float("nan"), device=DEV)
            lib.forward_kv4(q, pg.cache, bt, ints(lens), causal=True, out=out, lse=lse, check=True)
            assert not torch.isnan(out).any() and not torch.isnan(lse).any()
            check_attention(out, lse, q, pg, lens, [N] * 3, True, rows=(0, 1, N // 2, N - 1))
