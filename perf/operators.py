"""The 4-bit key/value cache and the attention over it: cases, plain forms and 64-bit definitions.

Three operators:
  append     quantise new keys and values into a paged cache (then read the written rows back)
  read       dequantise a range of positions of the cache
  attention  attention of queries over the cache: single tokens, a few tokens, long chunks

Cache format: per (token, head), blocks of 16 consecutive values along the head width share
one E4M3 scale s (a byte); each value is an E2M1 code (4 bits, low nibble first); a value
reads back as code * s * 2^e with one integer e per tensor. Pages hold `page` tokens:
codes [pages, heads, page, width / 2], scale bytes [pages, heads, page, width / 16]; the page
of a sequence's position p is block_table[b, p // page].
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, B, heads_q, heads_kv, d, N, L, page, dtype, ragged, causal, k_exp=0, v_exp=0):
    return dict(name=name, op=op, B=B, heads_q=heads_q, heads_kv=heads_kv, d=d, N=N, L=L, page=page, dtype=dtype,
                ragged=ragged, causal=causal, k_exp=k_exp, v_exp=v_exp)


def listed():
    return [
        # one new token of eight running sequences joins the cache: the smallest write of a decoding step
        _case("append_token", "append", 8, 32, 8, 128, 1, 1500, 16, "bf16", True, False),
        # the keys and values of a prompt batch at the training length are written at once
        _case("append_prompt", "append", 4, 32, 8, 128, 4096, 4096, 16, "bf16", False, False),
        # prompts of uneven length, narrow heads, small values (the tensor's exponent is below zero)
        _case("append_ragged", "append", 7, 12, 12, 64, 331, 1003, 32, "fp16", True, False, -3, -5),
        # a long cached prefix is read back (to move it, or to hand it to the dense kernels)
        _case("read_long", "read", 1, 32, 8, 128, 32768, 32768, 16, "bf16", False, False),
        # the last part of uneven sequences is read back in fp16
        _case("read_ragged", "read", 7, 12, 4, 64, 777, 4001, 64, "fp16", True, False, 2, 1),
        # one sequence decodes over a short cache: latency alone
        _case("decode_short", "attention", 1, 32, 8, 128, 1, 509, 16, "bf16", False, False),
        # a batch of uneven sequences decodes: the ordinary serving step
        _case("decode_batch", "attention", 16, 32, 8, 128, 1, 4096, 16, "bf16", True, False),
        # a large batch over long caches: the cache's bytes are all that counts
        _case("decode_large", "attention", 32, 32, 8, 128, 1, 32768, 64, "fp16", False, False),
        # narrow heads without grouping, odd lengths
        _case("decode_narrow", "attention", 6, 12, 12, 64, 1, 2047, 32, "fp16", True, False, -1, 0),
        # a few drafted tokens are verified together, eight query heads to a key head
        _case("verify_draft", "attention", 8, 32, 4, 128, 4, 8192, 16, "bf16", True, True),
        # a chunk of a long prompt attends over what is cached before it
        _case("chunk_long", "attention", 1, 32, 8, 128, 2048, 32768, 16, "bf16", False, True),
        # chunks of uneven prompts, some nearly done
        _case("chunk_ragged", "attention", 4, 28, 4, 128, 512, 4096, 32, "fp16", True, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice((64, 128, 128))
    heads_kv = rng.choice((1, 2, 4, 5, 8, 12))
    group = rng.choice((1, 2, 3, 4, 6, 7, 8))
    B = _log(rng, 1, 32)
    page = rng.choice((16, 16, 32, 64, 128))
    dtype = rng.choice(("bf16", "fp16"))
    ragged = rng.random() < 0.7
    k_exp, v_exp = rng.choice(((0, 0), (0, 0), (1, -2), (-4, 0)))
    op = rng.choice(("append", "read", "attention", "attention", "attention"))
    if op != "attention":
        N = _log(rng, 1, max(1, min(32768, 2 ** 25 // (B * heads_kv * d))))
        return _case("", op, B, heads_kv * group, heads_kv, d, N, N + rng.randrange(0, 2000), page, dtype, ragged,
                     False, k_exp, v_exp) | {"name": "drawn"}
    L = _log(rng, 40, max(41, min(32768, 2 ** 29 // (B * heads_kv * d))))
    N = rng.choice((1, 1, 1, _log(rng, 2, 16), _log(rng, 16, 2048)))
    N = max(1, min(N, L, 2 ** 29 // (B * heads_kv * group * L)))
    return _case("", op, B, heads_kv * group, heads_kv, d, N, L, page, dtype, ragged, N > 1 and rng.random() < 0.8,
                 k_exp, v_exp) | {"name": "drawn"}


def _lens(case):
    """Lengths of the sequences after this call, and how many new tokens each has."""
    B, L, N = case["B"], case["L"], case["N"]
    if not case["ragged"]:
        return [L] * B, [N] * B
    new = [max(1, N - (b * 5 * N) // (7 * B)) for b in range(B)]
    lens = [max(new[b], L - (b * 11 * L) // (17 * B)) for b in range(B)]
    return lens, new


# ---------------------------------------------------------------- plain forms (32 bits)
def _quantize(x, e):
    """(codes [..., d], scale bytes [..., d / 16]) of x in 32 bits; codes one to a byte."""
    y = (x.float() * 2.0 ** -e).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1) / 6.0).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    q = y / s.float().unsqueeze(-1)
    a = q.abs()
    # E2M1 by its rounding borders; a value on a border goes to the even code
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = code + 8 * (q < 0).int()
    return code.flatten(-2).to(torch.uint8), s.view(torch.uint8)


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _dequantize(codes, sf, e):
    """Values in 32 bits of packed codes and scale bytes."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = table[c.int()].unflatten(-1, (-1, 16))
    return (v * (sf.view(torch.float8_e4m3fn).float() * 2.0 ** e).unsqueeze(-1)).flatten(-2)


def _rows(st, first, n):
    """(page [B, n], slot [B, n], inside [B, n]) of the n positions from first[b] on."""
    pos = first.long().unsqueeze(1) + torch.arange(n, device=first.device)
    inside = (pos >= 0) & (pos < st["seq_lens"].long().unsqueeze(1))
    pos = pos.clamp(0, st["block_table"].shape[1] * st["page"] - 1)
    return st["block_table"].long().gather(1, pos // st["page"]), pos % st["page"], inside


def _gather(st, first, n, which):
    """Values [B, heads, n, d] in 32 bits of n positions from first[b] on (zero outside the sequence)."""
    page, slot, inside = _rows(st, first, n)
    codes = st[which + "_codes"][page, :, slot]            # [B, n, heads, d / 2]
    sf = st[which + "_sf"][page, :, slot]
    v = _dequantize(codes, sf, st[which + "_exp"])
    return (v * inside[..., None, None]).transpose(1, 2)


def _append_plain(st):
    n = st["k"].shape[2]
    first = st["seq_lens"] - st["new_lens"]
    page, slot, inside = _rows(st, first, n)
    for_row = inside & (torch.arange(n, device=page.device) < st["new_lens"].unsqueeze(1))
    for_row = for_row.nonzero(as_tuple=True)
    p, s = page[for_row], slot[for_row]

    def put(which):
        code, sf = _quantize(st[which].transpose(1, 2)[for_row], st[which + "_exp"])
        st[which + "_codes"][p, :, s] = _pack(code)
        st[which + "_sf"][p, :, s] = sf
    put("k")
    put("v")


def _attention_plain(st):
    q = st["q"].float()
    B, Hq, N, d = q.shape
    L = st["block_table"].shape[1] * st["page"]
    zero = torch.zeros_like(st["seq_lens"])
    k, v = _gather(st, zero, L, "k"), _gather(st, zero, L, "v")
    Hkv = k.shape[1]
    s = (q.reshape(B, Hkv, -1, d) @ k.transpose(2, 3)).view(B, Hq, N, L) * (1.0 / math.sqrt(d))
    j = torch.arange(L, device=q.device)
    i = torch.arange(N, device=q.device)
    lens, new = st["seq_lens"].long().unsqueeze(1), st["new_lens"].long().unsqueeze(1)
    last = torch.where(torch.tensor(st["causal"], device=q.device), lens - new + i, lens - 1)     # [B, N]
    s = s.masked_fill(j > last[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    den = p.sum(-1, keepdim=True)
    o = ((p / den).view(B, Hkv, -1, L) @ v).view(B, Hq, N, d)
    lse = (m + torch.log(den)).squeeze(-1)
    live = (i < new)[:, None, :]                                                                   # padded query rows stay zero
    return (o * live.unsqueeze(-1)).to(st["q"].dtype), lse * live


# ---------------------------------------------------------------- the measured calls
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    B, Hq, Hkv, d, N, L, page = (case[x] for x in ("B", "heads_q", "heads_kv", "d", "N", "L", "page"))
    dt = DTYPES[case["dtype"]]
    lens, new = _lens(case)
    per = -(-L // page)
    pages = B * per + 3
    st = dict(page=page, causal=case["causal"], k_exp=case["k_exp"], v_exp=case["v_exp"], N=N, dtype=dt)
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["new_lens"] = torch.tensor(new, dtype=torch.int32, device=DEV)
    st["starts"] = st["seq_lens"] - st["new_lens"]
    # the pages of a sequence lie anywhere in the cache, as after some time of serving
    st["block_table"] = torch.randperm(pages, generator=g, device=DEV)[:B * per].view(B, per).to(torch.int32)
    k_std, v_std = 1.0 * 2.0 ** case["k_exp"], 0.7 * 2.0 ** case["v_exp"]

    def values(shape, std, spread):
        # normal values, some channels larger than the others as keys have them, and rare outliers
        x = torch.randn(shape, generator=g, device=DEV)
        channel = torch.exp(spread * torch.randn(shape[-1], generator=g, device=DEV))
        x = x * channel * std
        return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.001, 8.0 * x, x)

    for which, std, spread in (("k", k_std, 0.4), ("v", v_std, 0.1)):
        code, sf = _quantize(values((pages, Hkv, page, d), std, spread), case[which + "_exp"])
        st[which + "_codes"], st[which + "_sf"] = _pack(code), sf
        del code
    if case["op"] == "append":
        st["k"] = values((B, Hkv, N, d), k_std, 0.4).to(dt)
        st["v"] = values((B, Hkv, N, d), v_std, 0.1).to(dt)
    elif case["op"] == "read":
        st["starts"] = st["seq_lens"] - N
        st["starts"].clamp_(min=0)
    else:
        st["q"] = torch.randn((B, Hq, N, d), generator=g, device=DEV).to(dt)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((B, Hq, N), device=DEV)
    st["op"] = case["op"]
    return st


def run(st):
    if own:
        import exact_attention_forward_11_b200 as attn
        if "cache" not in st:      # the handle of the cache's tensors, kept as a server keeps it
            st["cache"] = attn.KV4Cache(st["k_codes"], st["k_sf"], st["v_codes"], st["v_sf"], st["k_exp"], st["v_exp"])
        c, bt, lens, new = st["cache"], st["block_table"], st["seq_lens"], st["new_lens"]
        if st["op"] == "append":
            attn.kv4_append(c, st["k"], st["v"], bt, lens, new_lens=new)
        if st["op"] != "attention":
            return attn.kv4_read(c, bt, lens, st["N"], starts=st["starts"], dtype=st["dtype"])
        return attn.forward_kv4(st["q"], c, bt, lens, q_lens=new, causal=st["causal"], out=st["out"], lse=st["lse"])
    if st["op"] == "append":
        _append_plain(st)
    if st["op"] != "attention":
        return tuple(_gather(st, st["starts"], st["N"], w).to(st["dtype"]) for w in ("k", "v"))
    return _attention_plain(st)


def work(case):
    lens, new = _lens(case)
    Hq, Hkv, d, N = case["heads_q"], case["heads_kv"], case["d"], case["N"]
    packed = 2 * Hkv * d * 9 / 16                  # bytes of one token's keys and values in the cache
    if case["op"] == "append":
        t = sum(new)
        # the 16-bit rows are read, the cache rows written, read again and written out in 16 bits
        return {"bytes": t * (2 * Hkv * d * 2 + 2 * packed + 2 * Hkv * d * 2), "flops": t * 2 * Hkv * d * 4}
    if case["op"] == "read":
        t = sum(min(N, x) for x in lens)
        return {"bytes": t * (packed + 2 * Hkv * d * 2), "flops": t * 2 * Hkv * d * 2}
    pairs = sum((n * (x - n) + n * (n + 1) // 2) if case["causal"] else n * x for x, n in zip(lens, new))
    return {"bytes": sum(lens) * packed + sum(new) * Hq * (2 * d * 2 + 4), "flops": 4 * pairs * Hq * d}


# ---------------------------------------------------------------- 64 bits, from the definitions
def _e4m3_values():
    byte = np.arange(127)
    ex, man = byte >> 3, byte & 7
    return np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))


def _nearest(x, values):
    """The index of the nearest of the sorted `values` (a tie goes to the even index), on the GPU in 64 bits."""
    t = torch.tensor(values, dtype=torch.float64, device=x.device)
    mid = (t[1:] + t[:-1]) / 2
    lo = torch.searchsorted(mid, x.contiguous(), right=False)
    on_border = (lo < len(values) - 1) & (x == mid[lo.clamp(max=len(values) - 2)])
    return lo + (on_border & (lo % 2 == 1)).long()


def _stored64(x, e):
    """What the cache holds for x, as values in 64 bits."""
    scales = _e4m3_values()
    st, lv = (torch.tensor(v, dtype=torch.float64, device=x.device) for v in (scales, E2M1))
    y = x.double().reshape(*x.shape[:-1], -1, 16) / 2.0 ** e
    byte = _nearest(y.abs().max(-1).values / 6, scales).clamp(min=1)
    s = st[byte].unsqueeze(-1)
    return (torch.sign(y) * lv[_nearest((y / s).abs(), E2M1)] * s * 2.0 ** e).reshape(x.shape)


def _cached64(st, b, first, last, which):
    """Positions [first, last) of sequence b: values [heads, n, d] in 64 bits."""
    page = st["page"]
    ids = st["block_table"][b, first // page:-(-last // page)].long()
    codes, sf = (st[which + x][ids].transpose(0, 1).flatten(1, 2) for x in ("_codes", "_sf"))
    at = first % page
    codes, sf = codes[:, at:at + last - first].long(), sf[:, at:at + last - first].long()
    lv = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    scales = torch.tensor(_e4m3_values(), device=codes.device)
    out = torch.empty(*codes.shape[:2], 2 * codes.shape[2], dtype=torch.float64, device=codes.device)
    for half, c in ((0, codes % 16), (1, codes // 16)):
        out[..., half::2] = lv[c % 8] * (1 - 2 * (c // 8))
    return out * scales[sf].repeat_interleave(16, -1) * 2.0 ** st[which + "_exp"]


def exact(case, seed):
    lens, new = _lens(case)
    B, Hq, Hkv, d, N = (case[x] for x in ("B", "heads_q", "heads_kv", "d", "N"))
    if sum(lens) * Hkv * d > 2 ** 28 or sum(n * x for n, x in zip(new, lens)) * Hq > 2 ** 32:
        return None
    st = prepare(case, seed)
    if case["op"] != "attention":
        outs = []
        for w in ("k", "v"):
            o = torch.zeros((B, Hkv, N, d), dtype=torch.float64, device=DEV)
            for b in range(B):
                if case["op"] == "append":
                    o[b, :, :new[b]] = _stored64(st[w][b, :, :new[b]], case[w + "_exp"])
                else:
                    n = min(N, lens[b])
                    o[b, :, :n] = _cached64(st, b, lens[b] - n, lens[b], w)
            outs.append(o)
        return tuple(outs)
    out = torch.zeros((B, Hq, N, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, Hq, N), dtype=torch.float64, device=DEV)
    for b in range(B):
        k, v = _cached64(st, b, 0, lens[b], "k"), _cached64(st, b, 0, lens[b], "v")
        seen = torch.arange(lens[b], device=DEV) <= (lens[b] - new[b] + torch.arange(new[b], device=DEV)).unsqueeze(1)
        for h in range(Hq):
            q = st["q"][b, h, :new[b]].double()
            z = (q @ k[h * Hkv // Hq].T) / math.sqrt(d)
            if case["causal"]:
                z = torch.where(seen, z, -math.inf)
            w = torch.logsumexp(z, -1)
            out[b, h, :new[b]] = torch.exp(z - w.unsqueeze(1)) @ v[h * Hkv // Hq]
            lse[b, h, :new[b]] = w
    return out, lse
