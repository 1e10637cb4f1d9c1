"""Rows with attention sinks, infinities and NaN over the 4-bit cache, against the fp64 oracle.

Tolerance: that of tests/test_kv4_gpu.py with the rounding of P stated from its range. The kernels keep a
row's largest P at 2^7 or more, so that what f16 loses of a P below its normal range, 2^-25, is at most
2^-32 of the row's largest probability p_max:
    |O - ref| <= eps/2 |ref| + (2^-11 + 2 ds' + 2^-21 + 2 (L/8 + 64) 2^-24) A + L 2^-32 p_max max|v|
with p_max relative to the row's sum, A and ds' as there, and half a step of fp16's subnormals, 2^-25, for fp16 outputs.
"""
import math

import numpy as np
import pytest
import torch

from oracle.kv4 import kv4_attention, kv4_quantize, kv4_rows
from test_kv4_gpu import DEV, Paged, fill, ints, make_q, n64

pytestmark = pytest.mark.gpu

# rows of a cached head per kernel form: blocks of 8 and of 16 rows, one row tile, two row tiles
FORMS = {"block8": (1, 4), "block16": (4, 4), "one_tile": (20, 4), "two_tiles": (100, 4)}


def check_rows(o, lse, q, pg, lens, causal, rows, skip=None):
    eps, tiny = torch.finfo(o.dtype).eps, 2.0 ** -25 if o.dtype == torch.float16 else 0.0
    o64, l64, q64, scale = n64(o), n64(lse), n64(q), 1 / math.sqrt(pg.d)
    worst = 0.0
    for b in range(pg.B):
        L, n = lens[b], q64.shape[2]
        k, v = pg.values(b, L)
        ro, rl = kv4_attention(q64[b], k, v, n, causal, scale)
        G = q64.shape[1] // pg.H
        for h in range(q64.shape[1]):
            for i in [r for r in rows if r < n and not (skip is not None and skip[b, h, r])]:
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
                    + vis * 2.0 ** -32 * p.max() * np.abs(vv).max() + tiny
                err = np.abs(o64[b, h, i] - ro[h, i])
                worst = max(worst, (err / bound).max())
                assert (err <= bound).all(), (b, h, i, err.max(), np.abs(ro[h, i]).max(), (err / bound).max())
                assert abs(l64[b, h, i] - rl[h, i]) <= ds + add + 2.0 ** -21 + 2.0 ** -22 * abs(rl[h, i])
    return worst


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("d,dt", [(128, torch.bfloat16), (64, torch.bfloat16), (128, torch.float16)])
@pytest.mark.parametrize("margin,every,sink", [(18.5, 32, 0.0), (15.0, 32, 0.01), (18.5, 1 << 30, 0.0), (12.0, 32, 0.0),
                                               (21.0, 32, 0.0)])
def test_attention_sinks(cuda_lib, form, d, dt, margin, every, sink):
    """Keys whose score lies `margin` above all others and whose value is zero or small (every 32nd key, or the first
    alone): what is left of O is the many small probabilities."""
    lib, H, (N, Hq) = cuda_lib, 1, FORMS[form]
    lens = [2300, 700]
    pg = Paged(lib, 2, H, d, 16, 144, seed=7)
    if form == "one_tile":                                      # a table with room: the kernel of long chunks
        pg.bt = torch.cat([pg.bt, torch.full((2, 1 << 14), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    g = torch.Generator().manual_seed(int(margin * 10) + d)
    L = max(lens)
    k = torch.randn((2, H, L, d), generator=g) * 0.3
    v = 1.0 + 0.3 * torch.randn((2, H, L, d), generator=g)
    q = torch.randn((2, Hq, N, d), generator=g)
    q[..., 0] = 16.0
    k[..., 0] = 0.0
    k[:, :, ::every, 0] = margin * math.sqrt(d) / 16.0
    v[:, :, ::every] *= sink
    q = q.to(dt).to(DEV)
    lib.kv4_append(pg.cache, k.to(dt).to(DEV), v.to(dt).to(DEV), pg.bt, ints(lens), new_lens=ints(lens), check=True)
    o, lse = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), causal=N > 1, check=True)
    check_rows(o, lse, q, pg, lens, N > 1, (0, 1, N // 2, N - 1))


@pytest.mark.parametrize("form", FORMS)
def test_maximum_far_along_the_row(cuda_lib, form):
    """Scores that rise along the keys in steps on both sides of the threshold at which the running maximum moves,
    and fall again: P stays inside f16 and nothing of what came before is lost."""
    lib, d, (N, Hq) = cuda_lib, 128, FORMS[form]
    for step in (0.9, 4.9, 5.1, 7.0, 9.9, 10.6, 30.0):                     # in natural units, every 160 keys
        lens = [1300]
        pg = Paged(lib, 1, 1, d, 16, 82, seed=3)
        if form == "one_tile":
            pg.bt = torch.cat([pg.bt, torch.full((1, 1 << 14), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
        g = torch.Generator().manual_seed(int(step * 10))
        k, v = torch.randn((1, 1, 1300, d), generator=g) * 0.3, torch.randn((1, 1, 1300, d), generator=g)
        level = (torch.arange(1300) // 160).float()
        level = torch.where(level > 5, 10 - level, level)
        k[..., 0] = step * level * math.sqrt(d) / 16.0
        q = torch.randn((1, Hq, N, d), generator=g)
        q[..., 0] = 16.0
        q = q.to(torch.bfloat16).to(DEV)
        lib.kv4_append(pg.cache, k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), pg.bt, ints(lens),
                       new_lens=ints(lens), check=True)
        o, lse = lib.forward_kv4(q, pg.cache, pg.bt, ints(lens), causal=N > 1, check=True)
        check_rows(o, lse, q, pg, lens, N > 1, (0, 1, N // 2, N - 1))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,Hq,roomy", [(1, 4, False), (6, 4, False), (6, 8, False), (20, 8, True), (100, 4, False), (100, 4, True),
                                        (300, 2, True)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_goes_where_the_formula_takes_it(cuda_lib, d, N, Hq, roomy, which):
    """A NaN key: every channel and the LSE of the rows that see it. A NaN value: the 16 channels of its block in the
    rows that see it, and not the LSE. Everything else is bit for bit what it is without the NaN, wherever the key
    lies: in front of all queries' positions, among them (some rows see it, some do not), or last."""
    lib, H, L = cuda_lib, 2, 700
    per = -(-L // 16)
    g = torch.Generator().manual_seed(d + N)
    k, v = (torch.randn((1, H, L, d), generator=g).to(torch.bfloat16) for _ in range(2))
    q = make_q(1, Hq, N, d, torch.bfloat16, 5)
    spots = {5, L - N - 1, L - N, L - N // 2 - 1, L - 2, L - 1}
    for causal in (True, False):
        for spot in sorted(spots):
            outs = []
            for bad in (False, True):
                pg = Paged(lib, 1, H, d, 16, per, seed=1)
                if roomy:
                    pg.bt = torch.cat([pg.bt, torch.full((1, 1 << 14), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
                lib.kv4_append(pg.cache, k.to(DEV), v.to(DEV), pg.bt, ints([L]), check=True)
                sf = pg.cache.k_sf if which == "k" else pg.cache.v_sf
                at = (int(pg.bt[0, spot // 16]), 1, spot % 16)                 # of the second cached head
                if bad:
                    sf[at + (1,)] = 0x7F
                    sf[at + (d // 16 - 1,)] = 0xFF                            # either sign is a NaN
                outs.append(lib.forward_kv4(q, pg.cache, pg.bt, ints([L]), causal=causal, check=True))
            (o0, l0), (o1, l1) = outs
            assert torch.isfinite(o0).all() and torch.isfinite(l0).all()
            i = torch.arange(N, device=DEV)
            sees = (L - N + i >= spot) if causal else torch.ones_like(i, dtype=torch.bool)
            row = torch.zeros((1, Hq, N), dtype=torch.bool, device=DEV)
            row[:, Hq // 2:] = sees                                            # heads of the second cached head
            ch = torch.zeros(d, dtype=torch.bool, device=DEV)
            ch[16:32] = ch[d - 16:] = True
            want = row[..., None] & (ch if which == "v" else torch.ones_like(ch))
            assert torch.equal(torch.isnan(o1), want), (causal, spot)
            assert torch.equal(o1[~want], o0[~want])
            lost = row if which == "k" else torch.zeros_like(row)
            assert torch.equal(torch.isnan(l1), lost) and torch.equal(l1[~lost], l0[~lost])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_append_keeps_the_sign_of_zeros(cuda_lib, d, dt):
    """Codes and scale bytes bit for bit where quotients round to zero: zeros of both signs, values far below
    their block's maximum, on either side of the first border."""
    g = torch.Generator().manual_seed(d)
    N = 96
    x = torch.randn((1, 2, N, d), generator=g)
    small = torch.exp2(-torch.randint(1, 40, (1, 2, N, d), generator=g).float())
    x = torch.where(torch.rand((1, 2, N, d), generator=g) < 0.6, x * small, x)
    x = torch.where(torch.rand((1, 2, N, d), generator=g) < 0.1, torch.copysign(torch.zeros(()), x), x)
    x[0, 0, 0], x[0, 0, 1], x[0, 1, 0] = 0.0, -0.0, -float(torch.finfo(dt).tiny)
    x[0, 1, 1, ::2], x[0, 1, 2] = -0.0, -torch.finfo(dt).smallest_normal / 4
    x = x.to(dt)
    pg = Paged(cuda_lib, 1, 2, d, 16, N // 16, k_exp=-3, v_exp=2)
    cuda_lib.kv4_append(pg.cache, x.to(DEV), (-x).to(DEV), pg.bt, ints([N]), check=True)
    bt = pg.bt[0].cpu().numpy()
    negative_zeros = 0
    for sign, codes, sf, e in ((1, pg.cache.k_codes, pg.cache.k_sf, -3), (-1, pg.cache.v_codes, pg.cache.v_sf, 2)):
        c, s = kv4_quantize(n64(sign * x[0]), e)
        assert (kv4_rows(sf.cpu().numpy(), bt, 16, 0, N) == s).all()
        assert (kv4_rows(codes.cpu().numpy(), bt, 16, 0, N) == c).all()
        negative_zeros += int(((c & 15) == 8).sum() + ((c >> 4) == 8).sum())
    assert negative_zeros > 1000
    k, _ = cuda_lib.kv4_read(pg.cache, pg.bt, ints([N]), N, dtype=dt, check=True)
    assert torch.equal(torch.signbit(k.cpu()), torch.signbit(x))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
def test_infinite_and_nan_queries(cuda_lib, form, what):
    """A query row that holds an infinity or NaN has no finite softmax: its O is NaN where it sees a key (whatever the
    signs of the keys it meets), zero where it sees none, and the other rows are right. (Not bit for bit what they
    are beside a finite row: rows of a block move the value they subtract together.)"""
    lib, d, (N, Hq) = cuda_lib, 128, FORMS[form]
    for L, causal in ((40, True), (40, False), (1, True), (700, True)):
        pg = Paged(lib, 1, 1, d, 16, 44, seed=2)
        if form == "one_tile":
            pg.bt = torch.cat([pg.bt, torch.full((1, 1 << 14), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
        g = torch.Generator().manual_seed(L)
        k, v = (torch.randn((1, 1, L, d), generator=g) for _ in range(2))
        k[..., 7] = k[..., 7].abs() + 1.0                                   # one channel of one sign, and not zero
        lib.kv4_append(pg.cache, k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), pg.bt, ints([L]), check=True)
        q = make_q(1, Hq, N, d, torch.bfloat16, 3)
        bad = torch.zeros((1, Hq, N), dtype=torch.bool, device=DEV)
        bad[0, 1, N - 1] = bad[0, Hq - 1, 0] = bad[0, 0, N // 2] = True
        for channel in (7, 50):                                            # scores all of one sign, and of both
            qb = q.clone()
            qb[..., channel] = torch.where(bad, what, q[..., channel])
            o1, l1 = lib.forward_kv4(qb, pg.cache, pg.bt, ints([L]), causal=causal, check=True)
            sees = (L - N + torch.arange(N, device=DEV) >= 0) | (not causal)
            lost = bad & sees
            assert torch.equal(torch.isnan(o1), lost[..., None].expand_as(o1)), (L, causal, channel)
            check_rows(o1, l1, q, pg, [L], causal, sorted({0, 1, N // 2, N - 1}), skip=lost)
