"""The 4-bit cache calls refuse bad arguments on the host, before any CUDA call (CPU)."""
import pytest
import torch

import exact_attention_forward_11_b200 as attn

FAKE = 0x100000


@pytest.fixture(scope="module")
def lib():
    from exact_attention_forward_11_b200 import build
    build.build()
    return attn


MOVE = dict(a=FAKE, b=FAKE, c=FAKE, d_=FAKE, e=FAKE, f=FAKE, g=FAKE, h=FAKE, i=None, B=1, Hkv=2, N=3, d=128, pages=4,
            page=16, maxp=2, ke=0, ve=0, dtype=0, stream=None)
FWD = dict(q=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, ql=None, o=FAKE, lse=None, ws=FAKE,
           wsb=1 << 40, B=1, Hq=4, Hkv=2, N=3, d=128, pages=4, page=16, maxp=2, ke=0, ve=0, scale=0.0, causal=0,
           dtype=0, stream=None)
# (changed arguments, status) that all three calls share
SHARED = [(dict(B=0), 1), (dict(Hkv=0), 1), (dict(N=-1), 1), (dict(pages=0), 1), (dict(maxp=0), 1), (dict(page=0), 1),
          (dict(page=24), 2), (dict(page=8), 2), (dict(page=1 << 17), 2), (dict(d=96), 2), (dict(d=256), 2), (dict(dtype=2), 2),
          (dict(ke=33), 1), (dict(ve=-33), 1), (dict(page=65536, maxp=1 << 15), 1),
          (dict(pages=1 << 30, page=16), 1)]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(a=None), 1), (dict(c=None), 1), (dict(g=None), 1), (dict(h=None), 1), (dict(a=FAKE + 8), 3),
    (dict(c=FAKE + 2), 3), (dict(i=FAKE + 2), 3), (dict(B=1 << 16, N=1 << 15), 1)])
def test_append_and_read_refuse(lib, change, status):
    args = list(dict(MOVE, **change).values())
    assert lib.attn_kv4_append(*args) == status                # k, v, caches, tables, new_lens, ...
    order = args[2:8] + [args[8], args[0], args[1]] + args[9:]  # caches, tables, starts, k, v, ...
    assert lib.attn_kv4_read(*order) == status


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(q=None), 1), (dict(o=None), 1), (dict(kc=None), 1), (dict(vs=None), 1), (dict(bt=None), 1), (dict(sl=None), 1),
    (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(causal=2), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(q=FAKE + 4), 3), (dict(lse=FAKE + 4), 3), (dict(ql=FAKE + 1), 3), (dict(vs=FAKE + 8), 3), (dict(ws=FAKE + 8), 3),
    (dict(B=1 << 16, N=1 << 15), 1)])
def test_forward_refuses(lib, change, status):
    assert lib.attn_fwd_kv4(*dict(FWD, **change).values()) == status


def test_workspace_bytes_and_a_small_workspace(lib):
    wsb = lib.attn_fwd_kv4_workspace_bytes
    for bad in ((0, 4, 2, 1, 128, 16, 64), (1, 3, 2, 1, 128, 16, 64), (1, 4, 2, 1, 96, 16, 64), (1, 4, 2, 0, 128, 16, 64),
                (1, 4, 2, 1, 128, 24, 64), (1, 4, 2, 1, 128, 16, 0)):
        assert wsb(*bad) == 0
    need = wsb(1, 4, 2, 3, 128, 16, 2)
    if need:
        assert lib.attn_fwd_kv4(*dict(FWD, wsb=need - 1).values()) == 1
        assert lib.attn_fwd_kv4(*dict(FWD, ws=None).values()) == 1


def test_binding_refuses_tensors():
    """The handle and the calls check shapes, types and devices before the library is reached."""
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)                                # noqa: E731
    with pytest.raises(ValueError):
        attn.KV4Cache(u(4, 2, 16, 64), u(4, 2, 16, 8), u(4, 2, 16, 64), u(4, 2, 16, 8))    # host tensors
    with pytest.raises(ValueError):
        attn.KV4Cache(u(4, 2, 24, 64), u(4, 2, 24, 8), u(4, 2, 24, 64), u(4, 2, 24, 8))    # page size
    with pytest.raises(ValueError):
        attn.KV4Cache(u(4, 2, 16, 48), u(4, 2, 16, 6), u(4, 2, 16, 48), u(4, 2, 16, 6))    # width


@pytest.mark.gpu
def test_binding_refuses_tensors_gpu(cuda_lib):
    lib, dev = cuda_lib, torch.device("cuda:0")
    c = lib.KV4Cache.allocate(4, 2, 16, 128)
    bt, sl = torch.zeros(2, 3, dtype=torch.int32, device=dev), torch.ones(2, dtype=torch.int32, device=dev)
    q = torch.zeros(2, 4, 1, 128, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(2, 2, 1, 128, dtype=torch.bfloat16, device=dev)
    bad = [lambda: lib.forward_kv4(q.float(), c, bt, sl), lambda: lib.forward_kv4(q[..., :64].contiguous(), c, bt, sl),
           lambda: lib.forward_kv4(q, c, bt.long(), sl), lambda: lib.forward_kv4(q, c, bt[:1], sl),
           lambda: lib.forward_kv4(q, c, bt, sl[:1]), lambda: lib.forward_kv4(q, c, bt, sl.cpu()),
           lambda: lib.forward_kv4(q, c, bt, sl, q_lens=sl[:1]), lambda: lib.forward_kv4(q, c, bt, sl, out=q.half()),
           lambda: lib.forward_kv4(q, c, bt, sl, lse=q.float()),
           lambda: lib.forward_kv4(q.expand(2, 4, 2, 128), c, bt, sl),
           lambda: lib.kv4_append(c, q, q, bt, sl), lambda: lib.kv4_append(c, k, k.half(), bt, sl),
           lambda: lib.kv4_append(c, k.cpu(), k, bt, sl), lambda: lib.kv4_append(c, k, k, bt, sl, new_lens=bt),
           lambda: lib.kv4_read(c, bt, sl, 4, dtype=torch.float32), lambda: lib.kv4_read(c, bt, sl, 4, k=q),
           lambda: lib.KV4Cache(c.k_codes, c.k_sf, c.v_codes, c.v_sf[:2])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"case {i} was accepted")
    with pytest.raises(lib.AttnError):
        lib.forward_kv4(q[:, :3].contiguous(), c, bt, sl)                       # 3 query heads over 2
    with pytest.raises(lib.AttnError):
        lib.forward_kv4(q, c, bt, sl, scale=-1.0)
    with pytest.raises(lib.AttnError):
        lib.kv4_append(lib.KV4Cache(c.k_codes, c.k_sf, c.v_codes, c.v_sf, k_exp=40), k, k, bt, sl)
    torch.cuda.synchronize()
    assert lib.attn_get_device_status(None) == lib.ATTN_OK
