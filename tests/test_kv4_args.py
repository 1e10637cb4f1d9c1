"""The 4-bit cache calls refuse bad arguments on the host, before any CUDA call (CPU)."""
import ctypes

import pytest
import torch

import exact_attention_forward_11_b200 as attn

FAKE = 0x100000


@pytest.fixture(scope="module")
def lib():
    from exact_attention_forward_11_b200 import build
    build.build()
    return attn


CACHE = dict(k_codes=FAKE, k_sf=FAKE, v_codes=FAKE, v_sf=FAKE, num_pages=4, page_size=16, Hkv=2, d=128, k_exp=0, v_exp=0)
MOVE = dict(k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, first=None, B=1, N=3, maxp=2, dtype=0, stream=None)
FWD = dict(q=FAKE, bt=FAKE, sl=FAKE, ql=None, o=2 * FAKE, lse=None, ws=FAKE, wsb=1 << 40, B=1, Hq=4, N=3, maxp=2, scale=0.0,
           causal=0, dtype=0, stream=None)


def split(args, change):
    """(address of a cache struct, the other arguments by name) with the changes of either made."""
    struct = attn.attn_kv4_cache(**{k: change.get(k, v) for k, v in CACHE.items()})
    split.kept = struct                                        # alive during the call
    addr = None if "cache" in change else ctypes.addressof(struct)
    return addr, {k: change.get(k, v) for k, v in args.items()}


# (changed arguments, status) that all three calls share
SHARED = [(dict(cache=None), 1), (dict(k_codes=None), 1), (dict(v_sf=None), 1), (dict(bt=None), 1), (dict(sl=None), 1),
          (dict(B=0), 1), (dict(Hkv=0), 1), (dict(N=-1), 1), (dict(num_pages=0), 1), (dict(maxp=0), 1),
          (dict(page_size=0), 1), (dict(page_size=24), 2), (dict(page_size=8), 2), (dict(page_size=1 << 17), 2),
          (dict(d=96), 2), (dict(d=256), 2), (dict(dtype=2), 2), (dict(k_exp=33), 1), (dict(v_exp=-33), 1),
          (dict(page_size=65536, maxp=(1 << 14) + 1), 1), (dict(num_pages=1 << 30), 1), (dict(B=1 << 16, N=1 << 15), 1),
          (dict(k_codes=FAKE + 2), 3), (dict(v_sf=FAKE + 8), 3), (dict(bt=FAKE + 2), 3), (dict(sl=FAKE + 1), 3)]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 3), (dict(first=FAKE + 2), 3)])
def test_append_and_read_refuse(lib, change, status):
    addr, a = split(MOVE, change)
    rest = (a["B"], a["N"], a["maxp"], a["dtype"], a["stream"])
    assert lib.attn_kv4_append(addr, a["k"], a["v"], a["bt"], a["sl"], a["first"], *rest) == status
    assert lib.attn_kv4_read(addr, a["bt"], a["sl"], a["first"], a["k"], a["v"], *rest) == status


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(q=None), 1), (dict(o=None), 1), (dict(o=FAKE), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(causal=2), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(q=FAKE + 4), 3), (dict(lse=FAKE + 4), 3), (dict(ql=FAKE + 1), 3),
    (dict(ws=FAKE + 8), 3)])
def test_forward_refuses(lib, change, status):
    addr, a = split(FWD, change)
    assert lib.attn_fwd_kv4(addr, *a.values()) == status


def test_timeout_hook_refuses(lib):
    addr, a = split(FWD, {})
    *rest, stream = a.values()
    assert lib.attn_fwd_kv4_inject_timeout(addr, *rest, -1, 1 << 22, stream) == 1
    assert lib.attn_fwd_kv4_inject_timeout(addr, *rest, 0, 100, stream) == 1
    assert lib.attn_fwd_kv4_inject_timeout(None, *rest, 0, 1 << 22, stream) == 1


def test_workspace_bytes_and_a_small_workspace(lib):
    wsb = lib.attn_fwd_kv4_workspace_bytes
    for bad in ((0, 4, 2, 1, 128, 16, 64), (1, 3, 2, 1, 128, 16, 64), (1, 4, 2, 1, 96, 16, 64), (1, 4, 2, 0, 128, 16, 64),
                (1, 4, 2, 1, 128, 24, 64), (1, 4, 2, 1, 128, 16, 0)):
        assert wsb(*bad) == 0
    need = wsb(1, 4, 2, 3, 128, 16, 2)
    for change in (dict(wsb=need - 1), dict(ws=None)):
        addr, a = split(FWD, change)
        assert lib.attn_fwd_kv4(addr, *a.values()) == 1


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


def test_too_many_tiles_are_refused(lib):
    wsb = lib.attn_fwd_kv4_workspace_bytes
    tiles = (1 << 30) // 256                                   # of the longest table
    assert wsb(1, 511, 511, 1, 128, 65536, 1 << 14) > 0        # 511 (tiles + 2) < 2^31
    assert wsb(1, 512, 512, 1, 128, 65536, 1 << 14) == 0 and 512 * tiles == 1 << 31
    addr, a = split(FWD, dict(page_size=65536, maxp=1 << 14, num_pages=1, Hkv=512, Hq=512, N=1))
    assert lib.attn_fwd_kv4(addr, *a.values()) == 1


@pytest.mark.gpu
def test_handle_is_fixed_and_streams_of_another_device_are_refused(cuda_lib):
    lib, dev = cuda_lib, torch.device("cuda:0")
    c = lib.KV4Cache.allocate(4, 2, 16, 128, k_exp=-1)
    for name, value in (("k_exp", 2), ("v_codes", c.k_codes), ("heads", 1)):
        with pytest.raises(AttributeError):
            setattr(c, name, value)
    assert c.k_exp == -1 and c.heads == 2
    with pytest.raises(TypeError):
        lib.KV4Cache(c.k_codes, c.k_sf, c.v_codes, c.v_sf, k_exp=0.5)

    class Elsewhere:                                           # stands for a stream of a second GPU
        device = torch.device("cuda:1")
        cuda_stream = 0

    bt, sl = torch.zeros(2, 3, dtype=torch.int32, device=dev), torch.ones(2, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        lib.kv4_read(c, bt, sl, 4, stream=Elsewhere())
    torch.cuda.synchronize()


def test_overlapping_arrays_are_refused(lib):
    """Outputs that overlap one another, or the queries, would be written by CTAs in no order."""
    row = 2 * 3 * 128 * 2                                          # bytes of k: [1, 2, 3, 128]
    for v in (FAKE, FAKE + 16, FAKE - 16, FAKE + row - 16, FAKE - row + 16):
        addr, a = split(MOVE, dict(v=v))
        assert lib.attn_kv4_read(addr, a["bt"], a["sl"], a["first"], a["k"], a["v"], a["B"], a["N"], a["maxp"], a["dtype"],
                                 a["stream"]) == 1
    for o in (FAKE, FAKE + 16, FAKE - 2 * row + 16, FAKE + 2 * row - 16):    # q: [1, 4, 3, 128]
        addr, a = split(FWD, dict(o=o))
        assert lib.attn_fwd_kv4(addr, *a.values()) == 1


@pytest.mark.parametrize("exps", [((1 << 32) + 1, 0), (0, -(1 << 32)), (1 << 31, 0)])
def test_exponents_that_a_c_int_would_wrap(monkeypatch, exps):
    monkeypatch.setattr(attn, "_expect", lambda *a: None)          # (host tensors stand in for the cache's)
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)                                # noqa: E731
    tensors = u(4, 2, 16, 64), u(4, 2, 16, 8), u(4, 2, 16, 64), u(4, 2, 16, 8)
    assert attn.KV4Cache(*tensors, k_exp=-3, v_exp=32).k_exp == -3
    with pytest.raises(ValueError):
        attn.KV4Cache(*tensors, *exps)


@pytest.mark.parametrize("d", [64, 128])
def test_kernel_of_short_chunks(lib, d):
    """Above 32 rows the decode kernel runs up to 1600 units of 16 rows (both kernels are measured around it in
    csrc/kv4_api.cuh): its workspace has blocks of 16 rows, the chunk kernel's of 256."""
    def blocks_of_16(B, N, keys):                                  # 32 query heads on 8
        pages = -(-keys // 16)
        rows, tiles = 4 * N, -(-pages * 16 // 256)
        assert rows > 32
        small = lib.attn_fwd_kv4_workspace_bytes(B, 32, 8, N, d, 16, pages) < 2 * 148 * 17 * (4 * d + 8)
        return small, (tiles + 2) * B * 8 * -(-rows // 16)
    assert blocks_of_16(6, 12, 1000) == (True, 864)
    assert blocks_of_16(9, 12, 1000) == (True, 1296)
    assert blocks_of_16(16, 10, 300) == (True, 1536)
    assert blocks_of_16(3, 25, 2000) == (False, 1680)
    assert blocks_of_16(4, 25, 2000) == (False, 2240)
