"""One split-K W4A16 workspace for calls of different shapes, as the projections of a layer use it.

Every call counts on tickets that it finds zero, so no call may leave a partial where another
call's tickets lie. The first test checks the layout on the host (needs nvcc, no GPU); the others run it.
Tolerance of the products: tests/test_w4a16_gpu.py.
"""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import workloads
from oracle.w4a16 import dequantize_weights, w4a16_gemm_fp64

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
DEV = torch.device("cuda:0")


@pytest.mark.skipif(not os.path.exists(NVCC), reason="nvcc not found")
def test_splitk_workspace_layout(tmp_path):
    exe = tmp_path / "w4_workspace_check"
    subprocess.run([NVCC, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a",
                    f"-I{ROOT}/include", f"-I{ROOT}/exact_attention_forward_11_b200/csrc",
                    "-o", str(exe), os.path.join(HERE, "native", "w4_workspace_check.cu")],
                   check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok")


class Product:
    def __init__(self, M, K, N, seed):
        self.host = workloads.make_w4a16(M, N, K, seed=seed)
        self.x, *self.w = (t.to(DEV) for t in self.host)
        xn, qn, sn, zn = (t.numpy() for t in self.host)
        self.want = w4a16_gemm_fp64(xn, qn, sn, zn)
        w = dequantize_weights(qn, sn, zn).astype(np.float64)
        self.bound = 2.0 ** -11 * np.abs(self.want) + 2.0 ** -16 * (np.abs(xn.astype(np.float64)) @ np.abs(w)) + 1e-7

    def check(self, y):
        y = y.float().cpu().numpy()
        assert np.isfinite(y).all(), "NaN/inf in Y (unwritten element?)"
        assert (np.abs(y - self.want) <= self.bound).all()


# (M, K, N), each after the others: a small ticket area and then a larger one, wide and narrow, few and many tokens
RUN = [(16, 2048, 4096), (16, 2048, 6144), (16, 2048, 4096), (1, 4096, 1024), (16, 2048, 6144), (128, 1280, 2048),
       (3, 2176, 1152), (40, 384, 12800), (16, 2048, 6144)]


@pytest.mark.gpu
@pytest.mark.parametrize("own", [False, True], ids=["cached", "given"])
def test_one_workspace_for_products_of_different_widths(cuda_lib, own):
    lib = cuda_lib
    made = {s: Product(*s, seed=i) for i, s in enumerate(dict.fromkeys(RUN))}
    ws = None
    if own:
        ws = torch.zeros(max(lib.w4a16_gemm_splitk_workspace_bytes(M, N, K) for M, K, N in RUN), dtype=torch.uint8,
                         device=DEV)
    first = {}
    for _ in range(2):
        for s in RUN:
            p = made[s]
            y = torch.full((s[0], s[2]), float("nan"), dtype=torch.float16, device=DEV)
            lib.w4a16_matmul(p.x, *p.w, out=y, workspace=ws, check=True)
            p.check(y)
            assert torch.equal(y, first.setdefault(s, y))                # bit-identical whatever ran before
    if own:
        assert not ws[:4864].any()                                        # the tickets are zero again


@pytest.mark.gpu
def test_layer_of_projections_of_different_widths(cuda_lib):
    """Tokens through the projections of a layer (qkv, output, wide, narrow) again and again, one cached workspace."""
    lib, D, M = cuda_lib, 1024, 4
    widths = [(D, 3 * D + 512), (D, D), (D, 8 * D), (8 * D, D)]
    layer = [Product(M, K, N, seed=7 * i) for i, (K, N) in enumerate(widths)]
    for _ in range(5):
        ys = [lib.w4a16_matmul(p.x, *p.w) for p in layer]
        for p, y in zip(layer, ys):
            p.check(y)
    assert lib.attn_get_device_status(None) == lib.ATTN_OK


@pytest.mark.gpu
def test_captured_products_have_workspaces_of_their_own(cuda_lib):
    """Graphs captured on a stream whose cached workspace exists: replayed on two streams at once, between eager
    calls on the capture stream, and after a larger product has replaced the cached workspace."""
    lib = cuda_lib
    small, wide, big = Product(8, 4096, 1024, 1), Product(16, 2048, 6144, 2), Product(128, 4096, 8192, 3)
    side, streams = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = [lib.w4a16_matmul(p.x, *p.w, check=True) for p in (small, wide)]
    for p, y in zip((small, wide), want):
        p.check(y)
    graphs, outs = [], []
    for p in (small, wide):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            first = lib.w4a16_matmul(p.x, *p.w)
            second = lib.w4a16_matmul(small.x, *small.w)
        graphs.append(g)
        outs.append((first, second))
    cached = lib._W4_WORKSPACES[(0, side.cuda_stream)]
    before = cached.data_ptr()
    for round_ in range(4):
        for pair in outs:
            for y in pair:
                y.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(10):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
            with torch.cuda.stream(side):
                eager = lib.w4a16_matmul(wide.x, *wide.w)
        torch.cuda.synchronize()
        assert torch.equal(eager, want[1])
        for (first, second), w in zip(outs, want):
            assert torch.equal(first, w) and torch.equal(second, want[0])
        if round_ == 1:                                                    # a larger one replaces the cached workspace
            big.check(lib.w4a16_matmul(big.x, *big.w, stream=side, check=True))
            assert lib._W4_WORKSPACES[(0, side.cuda_stream)].data_ptr() != before
            del cached
            torch.cuda.empty_cache()
    assert lib.attn_get_device_status(None) == lib.ATTN_OK


@pytest.mark.gpu
def test_capture_without_an_eager_call_first(cuda_lib):
    """On a stream that has no cached workspace yet, with a fork to a second stream inside the capture."""
    lib = cuda_lib
    a, b = Product(4, 2048, 4096, 5), Product(16, 2048, 6144, 6)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        ya = lib.w4a16_matmul(a.x, *a.w)
        yb = torch.empty((16, 6144), dtype=torch.float16, device=DEV)
        lib.w4a16_matmul(b.x, *b.w, out=yb, stream=side)
        main.wait_stream(side)
        yc = lib.w4a16_matmul(b.x, *b.w)
    for _ in range(3):
        for y in (ya, yb, yc):
            y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        a.check(ya)
        b.check(yb)
        assert torch.equal(yb, yc)
    assert lib.attn_get_device_status(None) == lib.ATTN_OK
