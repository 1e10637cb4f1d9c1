"""The 4-bit cache kernels may start while the kernel before them in the stream still runs, and wait for
it themselves. The first test reads their sources (CPU); the second runs calls back to back, each reading what the
one before it wrote, and compares bit for bit with the same calls one at a time."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_forward_11_b200", "csrc")
KERNELS = ("kv4_cache_kernel.cuh", "kv4_attn_kernel.cuh", "kv4_chunk_kernel.cuh")
DEV = torch.device("cuda:0")


def code_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", KERNELS)
def test_nothing_is_read_through_the_read_only_path(name):
    """ld.global.nc asks for memory that nothing writes while the kernel lives: these kernels read what the
    one before them may still be writing. A restrict pointer would let the compiler choose that path, and an
    intrinsic without a memory clobber would let it move a load in front of the wait."""
    code = code_of(name)
    for word in (r"__ldg\b", r"__ldcg\b", r"__ldca\b", r"__ldcs\b", r"__ldlu\b", r"\.nc\b", r"__restrict"):
        assert not re.search(word, code), word


@pytest.mark.parametrize("name", KERNELS)
def test_every_kernel_waits_before_it_touches_memory(name):
    code = code_of(name)
    starts = [m.end() for m in re.finditer(r"__global__", code)]
    assert starts
    for at in starts:
        body = code[code.index("{", at):]
        before = body[:body.index("kv4_grid_wait()")]
        for word in (r"\bp\.c\.(codes|sf|seq_lens|block_table)\b", r"\bp\.(q|q_lens|o|lse|part_o|part_ml|heads)\b",
                     r"\bp\.(in|out|first)\b", r"tmem_alloc", r"__global__"):
            assert not re.search(word, before), (name, word)


@pytest.mark.gpu
@pytest.mark.parametrize("N,Hq,L", [(1, 4, 700), (5, 8, 300), (48, 4, 200), (150, 4, 400)])
@pytest.mark.parametrize("graph", [False, True])
def test_calls_back_to_back(cuda_lib, N, Hq, L, graph):
    """copies -> append -> read -> attention -> append -> ..., nothing between them but the stream's order."""
    lib, B, H, d, page = cuda_lib, 2, 2, 128, 16
    g = torch.Generator().manual_seed(N)
    per = -(-L // page)
    bt = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).to(DEV)
    sl = torch.full((B,), L, dtype=torch.int32, device=DEV)
    ks, vs = (torch.randn((4, B, H, L, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    qs = torch.randn((4, B, Hq, N, d), generator=g).to(torch.bfloat16).to(DEV)
    k, v, q = ks[0].clone(), vs[0].clone(), qs[0].clone()
    lens, table = sl.clone(), bt.clone()
    cache = lib.KV4Cache.allocate(B * per, H, page, d)

    def round_of(i, wait):
        def after():
            if wait:
                torch.cuda.synchronize()
        for dst, src in ((k, ks[i]), (v, vs[i]), (q, qs[i]), (lens, sl), (table, bt)):
            dst.zero_()
            dst.copy_(src)
            after()
        lib.kv4_append(cache, k, v, table, lens)
        after()
        rk, rv = lib.kv4_read(cache, table, lens, L)
        after()
        o, lse = lib.forward_kv4(q, cache, table, lens, causal=True)
        after()
        return rk, rv, o, lse

    want = [round_of(i, True) for i in range(4)]
    if graph:
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            got = [round_of(i % 4, False) for i in range(12)]
        for _ in range(5):
            gph.replay()
        torch.cuda.synchronize()
    else:
        got = [round_of(i % 4, False) for i in range(100)]
        torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i % 4])), i
    assert lib.attn_get_device_status(None) == lib.ATTN_OK
