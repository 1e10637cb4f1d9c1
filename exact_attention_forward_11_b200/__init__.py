"""B200 (sm_100a) fused attention forward: Python binding of the C ABI.

The entry points below have the names and arguments of the headers in include/ and
only marshal arguments: every step of the computation runs in the CUDA kernels
of libattn_b200.so. There is no CPU fallback; if the library is missing the
calls raise. `forward`, `forward_from_host`, `quantize_fp8`, `forward_fp8`, `quantize_mxfp8`, `forward_mxfp8`,
`backward`, `w4a16_matmul`, `kv4_append`, `kv4_read` and `forward_kv4` are torch conveniences
that allocate outputs with torch (PyTorch serves only for device memory and
streams) and call the same entry points.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
RELEASE_LIB_PATH = os.path.join(_HERE, "libattn_b200.so")
# the debug build (device-side index checks, ATTN_ERR_BOUNDS): ATTN_B200_DEBUG=1
DEBUG_LIB_PATH = os.path.join(_HERE, "libattn_b200_debug.so")
LIB_PATH = DEBUG_LIB_PATH if os.environ.get("ATTN_B200_DEBUG", "0") not in ("", "0") else RELEASE_LIB_PATH

(ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_MISALIGNED, ATTN_ERR_CUDA, ATTN_ERR_TIMEOUT,
 ATTN_ERR_BOUNDS) = range(7)
ATTN_BF16, ATTN_FP16 = 0, 1
TILE = 128

_lib = None

# (name, restype, argtypes) for every symbol the header declares
_P, _I, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _I, _P]),
    "attn_quantize_fp8": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "attn_fwd_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]),
    "attn_quantize_mxfp8": (_I, [_P, _P, _P, _I, _I, _I, _I, _P]),
    "attn_fwd_mxfp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]),
    "attn_get_device_status": (_I, [_P]),
    "attn_fwd_inject_timeout": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _I, ctypes.c_ulonglong, _P]),
    "attn_fwd_one_tile_inject_timeout": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _I, ctypes.c_ulonglong, _P]),
    "attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _I, _I, _I, _I, _F, _I, _P]),
    "attn_bwd_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "attn_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]),
    "w4a16_gemm": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "w4a16_gemm_splitk": (_I, [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _I, _I, _I, _P]),
    "w4a16_gemm_splitk_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I]),
    "attn_fwd_mxfp8_inject_timeout": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _I,
                                           ctypes.c_ulonglong, _P]),
    "attn_fwd_debug_row_limit": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, ctypes.c_longlong, _P]),
    "attn_debug_build": (_I, []),
    "attn_debug_last_failure": (_I, [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_longlong), _P]),
    "attn_kv4_append": (_I, [_P] * 6 + [_I] * 4 + [_P]),
    "attn_kv4_read": (_I, [_P] * 6 + [_I] * 4 + [_P]),
    "attn_fwd_kv4": (_I, [_P] * 8 + [ctypes.c_size_t] + [_I] * 4 + [_F, _I, _I, _P]),
    "attn_fwd_kv4_inject_timeout": (_I, [_P] * 8 + [ctypes.c_size_t] + [_I] * 4 + [_F, _I, _I, _I, ctypes.c_ulonglong, _P]),
    "attn_fwd_kv4_workspace_bytes": (ctypes.c_size_t, [_I] * 7),
    "attn_status_string": (ctypes.c_char_p, [_I]),
    "attn_abi_version": (_I, []),
}


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {attn_status_string(status)}")


def load():
    """Load the library at LIB_PATH: libattn_b200.so, or with ATTN_B200_DEBUG=1 its
    debug build libattn_b200_debug.so (both built by exact_attention_forward_11_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m exact_attention_forward_11_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


# ------------------------------------------------------------------ raw C ABI
def attn_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, dtype, stream):
    return load().attn_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, dtype, stream)


def attn_quantize_fp8(x, rot, x8, scales, B, H, N, d, stream):
    return load().attn_quantize_fp8(x, rot, x8, scales, B, H, N, d, stream)


def attn_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, B, H, N, d, scale, causal, stream):
    return load().attn_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, B, H, N, d, scale, causal, stream)


def attn_quantize_mxfp8(x, codes, sf, B, H, N, d, stream):
    return load().attn_quantize_mxfp8(x, codes, sf, B, H, N, d, stream)


def attn_fwd_mxfp8(q8, k8, v8, q_sf, k_sf, v_sf, o, lse, B, H, N, d, scale, causal, stream):
    return load().attn_fwd_mxfp8(q8, k8, v8, q_sf, k_sf, v_sf, o, lse, B, H, N, d, scale, causal, stream)


def attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, B, H, N, d, scale, causal, stream):
    return load().attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, B, H, N, d, scale,
                           causal, stream)


def attn_bwd_workspace_bytes(B, H, N, d):
    return load().attn_bwd_workspace_bytes(B, H, N, d)


def w4a16_gemm(x, qweight, scales, zeros, y, M, N, K, stream):
    return load().w4a16_gemm(x, qweight, scales, zeros, y, M, N, K, stream)


def w4a16_gemm_splitk(x, qweight, scales, zeros, y, workspace, workspace_bytes, M, N, K, stream):
    return load().w4a16_gemm_splitk(x, qweight, scales, zeros, y, workspace, workspace_bytes, M, N, K, stream)


def w4a16_gemm_splitk_workspace_bytes(M, N, K):
    return load().w4a16_gemm_splitk_workspace_bytes(M, N, K)


def attn_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal, stream):
    """attn_bwd with its scratch in a fixed array inside the library, for callers
    that cannot allocate device memory (include/attn_b200.h)."""
    return load().attn_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, scale, causal, stream)


ATTN_BWD_NOALLOC_MAX_ROWS = 1 << 21


def attn_fwd_inject_timeout(q, k, v, o, lse, B, H, N, d, scale, causal, fault_unit, wait_limit_cycles, stream):
    """Testing hook (include/attn_b200_testing.h): attn_fwd with one K tile withheld."""
    return load().attn_fwd_inject_timeout(q, k, v, o, lse, B, H, N, d, scale, causal, fault_unit,
                                          wait_limit_cycles, stream)


def attn_fwd_one_tile_inject_timeout(q, k, v, o, lse, B, H, N, d, scale, causal, fault_unit, wait_limit_cycles,
                                     stream):
    """Testing hook (include/attn_b200_testing.h): the one-Q-tile schedule with one K tile withheld."""
    return load().attn_fwd_one_tile_inject_timeout(q, k, v, o, lse, B, H, N, d, scale, causal, fault_unit,
                                                   wait_limit_cycles, stream)


def attn_fwd_mxfp8_inject_timeout(q8, k8, v8, q_sf, k_sf, v_sf, o, lse, B, H, N, d, scale, causal, fault_unit,
                                  wait_limit_cycles, stream):
    """Testing hook (include/attn_b200_testing.h): attn_fwd_mxfp8 with one K tile withheld."""
    return load().attn_fwd_mxfp8_inject_timeout(q8, k8, v8, q_sf, k_sf, v_sf, o, lse, B, H, N, d, scale, causal,
                                                fault_unit, wait_limit_cycles, stream)


def attn_fwd_debug_row_limit(q, k, v, o, lse, B, H, N, d, scale, causal, row_limit, stream):
    """Testing hook of the debug build (include/attn_b200_testing.h): attn_fwd told
    that O / LSE hold only `row_limit` rows."""
    return load().attn_fwd_debug_row_limit(q, k, v, o, lse, B, H, N, d, scale, causal, row_limit, stream)


def attn_debug_build():
    return load().attn_debug_build()


def attn_debug_last_failure(stream):
    """(site, index) of the first debug check that failed since the last call; site 0: none."""
    site, index = ctypes.c_int(0), ctypes.c_longlong(0)
    st = load().attn_debug_last_failure(ctypes.byref(site), ctypes.byref(index), stream)
    if st != ATTN_OK:
        raise AttnError(st, "attn_debug_last_failure")
    return site.value, index.value


class attn_kv4_cache(ctypes.Structure):
    """The cache struct of include/kv4_b200.h; the calls take its address (ctypes.addressof)."""
    _fields_ = [(n, _P) for n in ("k_codes", "k_sf", "v_codes", "v_sf")] + \
               [(n, _I) for n in ("num_pages", "page_size", "Hkv", "d", "k_exp", "v_exp")]


def attn_kv4_append(cache, k, v, block_table, seq_lens, new_lens, B, N, max_pages, dtype, stream):
    return load().attn_kv4_append(cache, k, v, block_table, seq_lens, new_lens, B, N, max_pages, dtype, stream)


def attn_kv4_read(cache, block_table, seq_lens, starts, k, v, B, N, max_pages, dtype, stream):
    return load().attn_kv4_read(cache, block_table, seq_lens, starts, k, v, B, N, max_pages, dtype, stream)


def attn_fwd_kv4(cache, q, block_table, seq_lens, q_lens, o, lse, workspace, workspace_bytes, B, Hq, N, max_pages,
                 scale, causal, dtype, stream):
    return load().attn_fwd_kv4(cache, q, block_table, seq_lens, q_lens, o, lse, workspace, workspace_bytes, B, Hq, N,
                               max_pages, scale, causal, dtype, stream)


def attn_fwd_kv4_inject_timeout(cache, q, block_table, seq_lens, q_lens, o, lse, workspace, workspace_bytes, B, Hq, N,
                                max_pages, scale, causal, dtype, fault_cta, wait_limit_cycles, stream):
    """Testing hook (include/attn_b200_testing.h): the chunk kernel with one CTA's first key tile withheld."""
    return load().attn_fwd_kv4_inject_timeout(cache, q, block_table, seq_lens, q_lens, o, lse, workspace, workspace_bytes,
                                              B, Hq, N, max_pages, scale, causal, dtype, fault_cta, wait_limit_cycles,
                                              stream)


def attn_fwd_kv4_workspace_bytes(B, Hq, Hkv, N, d, page_size, max_pages):
    return load().attn_fwd_kv4_workspace_bytes(B, Hq, Hkv, N, d, page_size, max_pages)


def use_library(path):
    """Switch the binding to another build of the library (e.g. DEBUG_LIB_PATH);
    later calls go to it. Returns the previous path."""
    global _lib, LIB_PATH
    prev = LIB_PATH
    LIB_PATH = path
    _lib = None
    return prev


def attn_get_device_status(stream):
    st = load().attn_get_device_status(stream)
    if st != ATTN_OK and _W4_WORKSPACES:
        _reset_w4_workspaces()
    return st


def attn_status_string(status):
    return load().attn_status_string(int(status)).decode()


def attn_abi_version():
    return load().attn_abi_version()


# ------------------------------------------------------------------ torch helpers
def _stream_ptr(t, stream):
    import torch
    s = torch.cuda.current_stream(t.device) if stream is None else stream
    return s.cuda_stream


def _check(status, where):
    if status != ATTN_OK:
        raise AttnError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _shape4(q):
    if q.dim() != 4 or not q.is_contiguous() or not q.is_cuda:
        raise ValueError("expected a contiguous CUDA tensor [B, H, N, d]")
    return tuple(q.shape)


def _expect(t, name, shape, dtype, device):
    """Every tensor handed to the library must be a contiguous CUDA tensor of the
    exact shape and dtype, on the same device as the first input (the kernels
    read and write through raw device pointers)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def _check_device(check, stream_ptr, where):
    """With check=True, wait for the launch and read the library's device status
    word (one per device, shared by every stream and thread: a timeout of any
    earlier launch is reported here too)."""
    if check:
        _check(attn_get_device_status(stream_ptr), where + " (device status)")


def forward(q, k, v, causal=False, scale=None, out=None, lse=None, with_lse=True, stream=None, check=False):
    """O, LSE = attention(q, k, v) for bf16 CUDA tensors [B, H, N, d].

    The call is asynchronous. The outputs are valid once the launch has finished
    AND attn_get_device_status() reports ATTN_OK (a pipeline wait that timed out
    leaves them undefined); check=True does both before returning. `scale`
    None selects 1/sqrt(d); a negative scale raises AttnError."""
    import torch
    B, H, N, d = _shape4(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _expect(t, name, (B, H, N, d), torch.bfloat16, q.device)
    if out is None:
        out = torch.empty_like(q)
    _expect(out, "out", (B, H, N, d), torch.bfloat16, q.device)
    if lse is None and with_lse:
        lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    if lse is not None:
        _expect(lse, "lse", (B, H, N), torch.float32, q.device)
    sc = 0.0 if scale is None else float(scale)
    sp = _stream_ptr(q, stream)
    _check(attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(lse), B, H, N, d, sc,
                    int(bool(causal)), ATTN_BF16, sp), "attn_fwd")
    _check_device(check, sp, "attn_fwd")
    return out, lse


_HOST_STREAMS = {}


def forward_from_host(q, k, v, causal=False, scale=None, out=None, lse=None, device=None, chunks=8):
    """O, LSE of attention for HOST tensors: bf16 [B, H, N, d] in (pinned) CPU
    memory in, O bf16 [B, H, N, d] and LSE fp32 [B, H, N] in (pinned) CPU memory
    out, for callers whose inputs arrive on the host.

    The B*H heads are cut into `chunks` contiguous groups (the heads are
    independent). Three streams overlap the copies with the kernels: group c+1
    is copied in while attn_fwd runs on group c (pointer offsets into the device
    buffers) and group c-1 is copied out, so the two PCIe directions and the GPU
    work at the same time. Returns once O and LSE are in host memory and the
    device status word reads ATTN_OK (raises AttnError otherwise). The results
    are the same bytes as forward() on the same inputs."""
    import torch

    from .sharded import head_range
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.is_cuda or t.dim() != 4 or not t.is_contiguous() or t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be a contiguous bf16 CPU tensor [B, H, N, d]")
    B, H, N, d = q.shape
    if k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v shapes differ")
    BH = B * H
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if out is None:
        out = torch.empty((B, H, N, d), dtype=torch.bfloat16).pin_memory()
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32).pin_memory()
    if out.is_cuda or tuple(out.shape) != (B, H, N, d) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 CPU tensor [B, H, N, d]")
    if lse.is_cuda or tuple(lse.shape) != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 CPU tensor [B, H, N]")
    chunks = max(1, min(int(chunks), BH))
    key = dev.index
    if key not in _HOST_STREAMS:
        _HOST_STREAMS[key] = tuple(torch.cuda.Stream(dev) for _ in range(3))
    s_in, s_run, s_out = _HOST_STREAMS[key]
    flat = [t.view(BH, N, d) for t in (q, k, v)]
    o_flat, l_flat = out.view(BH, N, d), lse.view(BH, N)
    dq, dk, dv, do = (torch.empty((BH, N, d), dtype=torch.bfloat16, device=dev) for _ in range(4))
    # one LSE buffer per group: an offset of h0 * N floats into a shared one is
    # 16-byte aligned only when h0 * N is a multiple of 4
    dls = [torch.empty((head_range(BH, chunks, c)[1], N), dtype=torch.float32, device=dev) for c in range(chunks)]
    # the device buffers are allocated on the current stream; the three streams
    # start after it
    start = torch.cuda.Event()
    start.record(torch.cuda.current_stream(dev))
    for st in (s_in, s_run, s_out):
        st.wait_event(start)
    sc = 0.0 if scale is None else float(scale)
    elem = 2 * N * d
    for c in range(chunks):
        h0, cnt = head_range(BH, chunks, c)
        if cnt == 0:
            continue
        sl = slice(h0, h0 + cnt)
        with torch.cuda.stream(s_in):
            for dst, src in zip((dq, dk, dv), flat):
                dst[sl].copy_(src[sl], non_blocking=True)
            ready = torch.cuda.Event()
            ready.record(s_in)
        s_run.wait_event(ready)
        off = h0 * elem
        _check(attn_fwd(dq.data_ptr() + off, dk.data_ptr() + off, dv.data_ptr() + off, do.data_ptr() + off,
                        dls[c].data_ptr(), 1, cnt, N, d, sc, int(bool(causal)), ATTN_BF16,
                        s_run.cuda_stream), "attn_fwd")
        done = torch.cuda.Event()
        done.record(s_run)
        s_out.wait_event(done)
        with torch.cuda.stream(s_out):
            o_flat[sl].copy_(do[sl], non_blocking=True)
            l_flat[sl].copy_(dls[c], non_blocking=True)
    # every copy and launch above has finished once the copy-out stream has (it
    # waited on each group's kernel, which waited on that group's copies in), so
    # the device buffers can go back to the allocator when this returns
    s_out.synchronize()
    _check(attn_get_device_status(s_run.cuda_stream), "forward_from_host (device status)")
    return out, lse


def quantize_fp8(x, rot=None, stream=None):
    """(codes uint8 [B,H,N,d], scales fp32 [B,H,ceil(N/128)]) of a bf16 tensor."""
    import torch
    B, H, N, d = _shape4(x)
    _expect(x, "x", (B, H, N, d), torch.bfloat16, x.device)
    if rot is not None:
        _expect(rot, "rot", (d, d), torch.bfloat16, x.device)
    x8 = torch.empty((B, H, N, d), device=x.device, dtype=torch.uint8)
    scales = torch.empty((B, H, (N + TILE - 1) // TILE), device=x.device, dtype=torch.float32)
    _check(attn_quantize_fp8(x.data_ptr(), _ptr(rot), x8.data_ptr(), scales.data_ptr(), B, H, N, d,
                             _stream_ptr(x, stream)), "attn_quantize_fp8")
    return x8, scales


def forward_fp8(q8, k8, v8, q_scale, k_scale, v_scale, causal=False, scale=None, out=None, lse=None,
                with_lse=True, stream=None, check=False):
    """O (bf16), LSE from E4M3 codes and their per-tile scales (finite, >= 0).

    Asynchronous like forward(): the outputs are valid once the launch has
    finished and attn_get_device_status() reports ATTN_OK; check=True does both."""
    import torch
    B, H, N, d = _shape4(q8)
    T = (N + TILE - 1) // TILE
    for name, t in (("q8", q8), ("k8", k8), ("v8", v8)):
        _expect(t, name, (B, H, N, d), torch.uint8, q8.device)
    for name, t in (("q_scale", q_scale), ("k_scale", k_scale), ("v_scale", v_scale)):
        _expect(t, name, (B, H, T), torch.float32, q8.device)
    if out is None:
        out = torch.empty((B, H, N, d), device=q8.device, dtype=torch.bfloat16)
    _expect(out, "out", (B, H, N, d), torch.bfloat16, q8.device)
    if lse is None and with_lse:
        lse = torch.empty((B, H, N), device=q8.device, dtype=torch.float32)
    if lse is not None:
        _expect(lse, "lse", (B, H, N), torch.float32, q8.device)
    sc = 0.0 if scale is None else float(scale)
    sp = _stream_ptr(q8, stream)
    _check(attn_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), q_scale.data_ptr(), k_scale.data_ptr(),
                        v_scale.data_ptr(), out.data_ptr(), _ptr(lse), B, H, N, d, sc, int(bool(causal)), sp),
           "attn_fwd_fp8")
    _check_device(check, sp, "attn_fwd_fp8")
    return out, lse


def quantize_mxfp8(x, stream=None):
    """(codes uint8 [B,H,N,d], scale bytes uint8 [B,H,N,d/32]) of a bf16 tensor:
    MXFP8, one E8M0 scale per 32 consecutive values of a row."""
    import torch
    B, H, N, d = _shape4(x)
    _expect(x, "x", (B, H, N, d), torch.bfloat16, x.device)
    codes = torch.empty((B, H, N, d), device=x.device, dtype=torch.uint8)
    # the scale array is padded to 16 bytes so that its base stays 16-byte aligned
    nsf = B * H * N * (d // 32)
    sf = torch.empty(((nsf + 15) // 16) * 16, device=x.device, dtype=torch.uint8)[:nsf].view(B, H, N, d // 32)
    _check(attn_quantize_mxfp8(x.data_ptr(), codes.data_ptr(), sf.data_ptr(), B, H, N, d, _stream_ptr(x, stream)),
           "attn_quantize_mxfp8")
    return codes, sf


def forward_mxfp8(q8, k8, v8, q_sf, k_sf, v_sf, causal=False, scale=None, out=None, lse=None, with_lse=True,
                  stream=None, check=False):
    """O (bf16), LSE from MXFP8 codes [B,H,N,d] and their scale bytes [B,H,N,d/32].

    Asynchronous like forward(): the outputs are valid once the launch has
    finished and attn_get_device_status() reports ATTN_OK; check=True does both."""
    import torch
    B, H, N, d = _shape4(q8)
    for name, t in (("q8", q8), ("k8", k8), ("v8", v8)):
        _expect(t, name, (B, H, N, d), torch.uint8, q8.device)
    if d % 32:
        raise ValueError("d must be a multiple of 32")
    for name, t in (("q_sf", q_sf), ("k_sf", k_sf), ("v_sf", v_sf)):
        _expect(t, name, (B, H, N, d // 32), torch.uint8, q8.device)
    if out is None:
        out = torch.empty((B, H, N, d), device=q8.device, dtype=torch.bfloat16)
    _expect(out, "out", (B, H, N, d), torch.bfloat16, q8.device)
    if lse is None and with_lse:
        lse = torch.empty((B, H, N), device=q8.device, dtype=torch.float32)
    if lse is not None:
        _expect(lse, "lse", (B, H, N), torch.float32, q8.device)
    sc = 0.0 if scale is None else float(scale)
    sp = _stream_ptr(q8, stream)
    _check(attn_fwd_mxfp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), q_sf.data_ptr(), k_sf.data_ptr(),
                          v_sf.data_ptr(), out.data_ptr(), _ptr(lse), B, H, N, d, sc, int(bool(causal)), sp),
           "attn_fwd_mxfp8")
    _check_device(check, sp, "attn_fwd_mxfp8")
    return out, lse


def backward(q, k, v, o, lse, dout, causal=False, scale=None, dq=None, dk=None, dv=None, workspace=None,
             stream=None, check=False):
    """dQ, dK, dV of attention for bf16 CUDA tensors [B, H, N, d], given the
    forward's O and LSE and dout = dL/dO. The workspace (D_i per row) is
    allocated with torch unless given. Asynchronous like forward()."""
    import torch
    B, H, N, d = _shape4(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _expect(t, name, (B, H, N, d), torch.bfloat16, q.device)
    _expect(lse, "lse", (B, H, N), torch.float32, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _expect(t, name, (B, H, N, d), torch.bfloat16, q.device)
    need = attn_bwd_workspace_bytes(B, H, N, d)
    if need == 0:
        raise AttnError(ATTN_ERR_UNSUPPORTED, "attn_bwd_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if not workspace.is_cuda or workspace.device != q.device or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA buffer of at least {need} bytes on {q.device}")
    sc = 0.0 if scale is None else float(scale)
    sp = _stream_ptr(q, stream)
    _check(attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                    dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
                    workspace.numel() * workspace.element_size(), B, H, N, d, sc, int(bool(causal)), sp),
           "attn_bwd")
    _check_device(check, sp, "attn_bwd")
    return dq, dk, dv


# split-K workspaces of w4a16_matmul, one per (device, stream): zeroed when
# allocated; every call leaves the tickets, its first bytes, zero again
_W4_WORKSPACES = {}
_W4_TICKET_BYTES = 4864


def _reset_w4_workspaces():
    """After a device status other than ATTN_OK a split-K call may have left
    tickets set: wait for the device and zero every cached workspace."""
    import torch
    torch.cuda.synchronize()
    for t in _W4_WORKSPACES.values():
        t.zero_()
    torch.cuda.synchronize()


def _w4_workspace(device, stream, stream_ptr, nbytes):
    import torch
    if stream is not None or torch.cuda.current_device() != device.index:
        with torch.cuda.device(device), torch.cuda.stream(stream):  # (a stream of None changes nothing)
            return _w4_workspace(device, None, stream_ptr, nbytes)
    if torch.cuda.is_current_stream_capturing():
        # a graph has its own, zeroed in every replay: it may be replayed on any stream, next to any other
        # call, and after the cached one has been replaced by a larger one
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        ws[:_W4_TICKET_BYTES].zero_()
        return ws
    key = (device.index, stream_ptr)
    ws = _W4_WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        if ws is not None:
            torch.cuda.synchronize(device)        # the old one may still be read by a launch
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        torch.cuda.current_stream(device).synchronize()   # zeroed before any stream uses it
        _W4_WORKSPACES[key] = ws
    return ws


def w4a16_matmul(x, qweight, scales, zeros, out=None, stream=None, check=False, split_k=True, workspace=None):
    """Y = X W for fp16 X [M, K] and W given as packed int4 (int32 [K/8, N]), fp16
    scales [K/128, N] and uint8 zero points [K/128, N] (include/w4a16_b200.h).

    split_k=True (default) runs w4a16_gemm_splitk, which balances the K slices over
    every SM; its workspace is `workspace` (a zeroed uint8 CUDA tensor of at least
    w4a16_gemm_splitk_workspace_bytes(M, N, K) bytes) or one cached per device and
    stream (inside a graph capture: the graph's own). split_k=False runs w4a16_gemm (one CTA per 128 output columns)."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    _expect(x, "x", (M, K), torch.float16, x.device)
    N = qweight.shape[1] if qweight.dim() == 2 else -1
    _expect(qweight, "qweight", (K // 8, N), torch.int32, x.device)
    _expect(scales, "scales", (K // 128, N), torch.float16, x.device)
    _expect(zeros, "zeros", (K // 128, N), torch.uint8, x.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=x.device)
    _expect(out, "out", (M, N), torch.float16, x.device)
    sp = _stream_ptr(x, stream)
    if not split_k:
        _check(w4a16_gemm(x.data_ptr(), qweight.data_ptr(), scales.data_ptr(), zeros.data_ptr(), out.data_ptr(),
                          M, N, K, sp), "w4a16_gemm")
        _check_device(check, sp, "w4a16_gemm")
        return out
    need = w4a16_gemm_splitk_workspace_bytes(M, N, K)
    if need == 0:
        raise AttnError(ATTN_ERR_UNSUPPORTED, "w4a16_gemm_splitk_workspace_bytes")
    if workspace is None:
        workspace = _w4_workspace(x.device, stream, sp, need)
    elif workspace.device != x.device or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a contiguous tensor of at least {need} bytes on {x.device}")
    _check(w4a16_gemm_splitk(x.data_ptr(), qweight.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                             out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                             M, N, K, sp), "w4a16_gemm_splitk")
    _check_device(check, sp, "w4a16_gemm_splitk")
    return out


class KV4Cache:
    """The tensors of a 4-bit key/value cache (format: include/kv4_b200.h) and their
    exponents: k_codes, v_codes uint8 [num_pages, Hkv, page_size, d / 2], k_sf, v_sf uint8
    [num_pages, Hkv, page_size, d / 16]. The handle checks them once and keeps them (its
    attributes cannot be set); KV4Cache.allocate makes new ones. A value reads back as code * scale * 2^exp:
    exponents other than 0 suit tensors whose values are mostly below about 0.1 or
    above 2000."""

    __slots__ = ("k_codes", "k_sf", "v_codes", "v_sf", "k_exp", "v_exp", "num_pages", "heads", "page_size", "d",
                 "device", "_index", "_struct", "_addr", "_need")

    def __init__(self, k_codes, k_sf, v_codes, v_sf, k_exp=0, v_exp=0):
        global torch     # the cache calls below run at the rate of decoding steps: no import in each
        import torch
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [num_pages, Hkv, page_size, d / 2]")
        P, H, S, half = k_codes.shape
        if half not in (32, 64) or S < 16 or S & (S - 1):
            raise ValueError("d must be 64 or 128 and page_size a power of two, 16 or more")
        for name, t, width in (("k_codes", k_codes, half), ("v_codes", v_codes, half), ("k_sf", k_sf, half // 8),
                               ("v_sf", v_sf, half // 8)):
            _expect(t, name, (P, H, S, width), torch.uint8, k_codes.device)
        struct = attn_kv4_cache(*(t.data_ptr() for t in (k_codes, k_sf, v_codes, v_sf)), P, S, H, 2 * half,
                                operator.index(k_exp), operator.index(v_exp))
        if (struct.k_exp, struct.v_exp) != (k_exp, v_exp):      # a C int would wrap
            raise ValueError("k_exp and v_exp must lie in [-32, 32]")
        for name, value in dict(k_codes=k_codes, k_sf=k_sf, v_codes=v_codes, v_sf=v_sf, k_exp=struct.k_exp,
                                v_exp=struct.v_exp, num_pages=P, heads=H, page_size=S, d=2 * half,
                                device=k_codes.device, _index=k_codes.get_device(), _struct=struct,
                                _addr=ctypes.addressof(struct),
                                _need={}).items():     # _need: workspace bytes of forward_kv4 by (B, Hq, N, max_pages)
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError("a KV4Cache is fixed: make another handle")

    @classmethod
    def allocate(cls, num_pages, heads, page_size, d, k_exp=0, v_exp=0, device="cuda"):
        """A cache of num_pages empty pages (their slots hold nothing until written)."""
        import torch
        shape = (num_pages, heads, page_size)
        new = [torch.empty((*shape, w), dtype=torch.uint8, device=device) for w in (d // 2, d // 16, d // 2, d // 16)]
        return cls(*new, k_exp=k_exp, v_exp=v_exp)


def _kv4_int32(t, name, shape, cache):
    if t.shape != shape or t.dtype is not torch.int32 or t.get_device() != cache._index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on {cache.device}")
    return t.data_ptr()


def _kv4_rows(t, name, cache):
    """Shape, element type and its code of a 16-bit [B, H, N, d] argument of the cache calls."""
    dtype, shape = t.dtype, t.shape
    dt = ATTN_BF16 if dtype is torch.bfloat16 else ATTN_FP16
    if len(shape) != 4 or t.get_device() != cache._index or not t.is_contiguous() or \
            (dt == ATTN_FP16 and dtype is not torch.float16):
        raise ValueError(f"{name} must be a contiguous bf16 or fp16 tensor [B, H, N, d] on {cache.device}")
    if shape[3] != cache.d:
        raise ValueError(f"{name} has heads of width {shape[3]}: the cache has {cache.d}")
    return shape, dtype, dt


def _kv4_like(t, name, shape, dtype, cache):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != cache._index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {cache.device}")
    return t.data_ptr()


def _kv4_table(t, B, cache):
    shape = t.shape
    if len(shape) != 2 or shape[0] != B or t.dtype is not torch.int32 or t.get_device() != cache._index or \
            not t.is_contiguous():
        raise ValueError(f"block_table must be a contiguous int32 tensor [{B}, max_pages] on {cache.device}")
    return t.data_ptr(), shape[1]


class _kv4_place:
    """Runs a launch with the tensors' device current and, for torch allocations, the
    launch's stream current (a buffer made here then belongs to that stream)."""

    __slots__ = ("ctx", "sp")

    def __init__(self, device, stream):
        self.ctx = [torch.cuda.device(device)]
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream must be a stream of {device}")
            self.ctx.append(torch.cuda.stream(stream))
        for c in self.ctx:
            c.__enter__()
        self.sp = torch.cuda.current_stream(device).cuda_stream

    def leave(self):
        for c in reversed(self.ctx):
            c.__exit__(None, None, None)


def _kv4_stream(cache, stream):
    """(raw stream, place to leave or None): nothing to switch in the usual case, the
    current stream of the current device."""
    index = cache._index
    if stream is None and index == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(index), None
    place = _kv4_place(cache.device, stream)
    return place.sp, place


def kv4_append(cache, k, v, block_table, seq_lens, new_lens=None, stream=None, check=False):
    """Quantises new tokens k, v (bf16 or fp16 [B, Hkv, N, d]) into the cache.

    seq_lens (int32 [B]) are the lengths AFTER the call: token i < new_lens[b] (None: N
    of each) goes to position seq_lens[b] - new_lens[b] + i, whose page is
    block_table[b, position // page_size]. Asynchronous; a page number or length outside
    the cache skips the write and is reported by attn_get_device_status()
    (check=True waits and raises). Returns the cache."""
    shape, dtype, dt = _kv4_rows(k, "k", cache)
    B, H, N, _ = shape
    if H != cache.heads:
        raise ValueError(f"k has {H} heads: the cache has {cache.heads}")
    vp = _kv4_like(v, "v", shape, dtype, cache)
    bt, max_pages = _kv4_table(block_table, B, cache)
    sl = _kv4_int32(seq_lens, "seq_lens", (B,), cache)
    nl = None if new_lens is None else _kv4_int32(new_lens, "new_lens", (B,), cache)
    sp, place = _kv4_stream(cache, stream)
    try:
        st = load().attn_kv4_append(cache._addr, k.data_ptr(), vp, bt, sl, nl, B, N, max_pages, dt, sp)
        if st or check:
            _check(st, "attn_kv4_append")
            _check_device(check, sp, "attn_kv4_append")
    finally:
        if place is not None:
            place.leave()
    return cache


def kv4_read(cache, block_table, seq_lens, N, starts=None, dtype=None, k=None, v=None, stream=None, check=False):
    """K, V (bf16 or fp16 [B, Hkv, N, d]) read back from the cache: row i holds position
    starts[b] + i (None: i); rows at or behind seq_lens[b] are zero. Asynchronous;
    bad page numbers and lengths as in kv4_append."""
    B = seq_lens.shape[0]
    bt, max_pages = _kv4_table(block_table, B, cache)
    sl = _kv4_int32(seq_lens, "seq_lens", (B,), cache)
    first = None if starts is None else _kv4_int32(starts, "starts", (B,), cache)
    sp, place = _kv4_stream(cache, stream)
    try:
        if k is None:
            k = torch.empty(B, cache.heads, N, cache.d, dtype=torch.bfloat16 if dtype is None else dtype,
                            device=cache.device)
        shape, kdtype, dt = _kv4_rows(k, "k", cache)
        if shape[0] != B or shape[2] != N or shape[1] != cache.heads or (dtype is not None and kdtype is not dtype):
            raise ValueError(f"k must be [{B}, {cache.heads}, {N}, {cache.d}]" + ("" if dtype is None else f" of {dtype}"))
        if v is None:
            v = torch.empty_like(k)
            vp = v.data_ptr()
        else:
            vp = _kv4_like(v, "v", shape, kdtype, cache)
        st = load().attn_kv4_read(cache._addr, bt, sl, first, k.data_ptr(), vp, B, N, max_pages, dt, sp)
        if st or check:
            _check(st, "attn_kv4_read")
            _check_device(check, sp, "attn_kv4_read")
    finally:
        if place is not None:
            place.leave()
    return k, v


# workspaces of forward_kv4, one per (device, stream) of each host thread: launches of one stream run in order, but
# a call is two launches, between which another thread's may come
_KV4_WORKSPACES = threading.local()


def _kv4_workspace(cache, sp, need):
    if torch._C._cuda_isCurrentStreamCapturing():
        # a graph has its own: it may be replayed on any stream, next to any other call
        return torch.empty(need, dtype=torch.uint8, device=cache.device)
    kept = _KV4_WORKSPACES.__dict__
    key = (cache._index, sp)
    ws = kept.get(key)
    if ws is None or ws.shape[0] < need:
        # (made with that stream current: the memory of the old one goes back to its pool)
        ws = kept[key] = torch.empty(need, dtype=torch.uint8, device=cache.device)
    return ws


def forward_kv4(q, cache, block_table, seq_lens, q_lens=None, causal=False, scale=None, out=None, lse=None,
                with_lse=True, workspace=None, stream=None, check=False):
    """O, LSE = attention of q (bf16 or fp16 [B, Hq, N, d]) over the 4-bit cache.

    Hq is a multiple of the cache's heads (query head h reads cache head
    h // (Hq / Hkv)). Query i < q_lens[b] (None: N of each) is the token at position
    seq_lens[b] - q_lens[b] + i (append its key and value first, with the same
    seq_lens); it sees every cached position, with causal=True only those up to its
    own. N = 1 is a decoding step. Rows behind q_lens[b] are left as they were in out
    and lse (zero where those are allocated here); a row that sees no key gets O = 0,
    LSE = -inf. `workspace`: a uint8 tensor of at least attn_fwd_kv4_workspace_bytes(...);
    None: one kept per thread, device and stream (inside a graph capture: the graph's own).
    Asynchronous like forward(); bad page numbers and lengths as in kv4_append."""
    shape, dtype, dt = _kv4_rows(q, "q", cache)
    B, Hq, N, _ = shape
    bt, max_pages = _kv4_table(block_table, B, cache)
    sl = _kv4_int32(seq_lens, "seq_lens", (B,), cache)
    ql = None if q_lens is None else _kv4_int32(q_lens, "q_lens", (B,), cache)
    sp, place = _kv4_stream(cache, stream)
    try:
        if out is None:
            out = torch.empty_like(q) if q_lens is None else torch.zeros_like(q)
            o = out.data_ptr()
        else:
            o = _kv4_like(out, "out", shape, dtype, cache)
        if lse is not None:
            lp = _kv4_like(lse, "lse", (B, Hq, N), torch.float32, cache)
        elif with_lse:
            lse = (torch.empty if q_lens is None else torch.zeros)(B, Hq, N, dtype=torch.float32, device=cache.device)
            lp = lse.data_ptr()
        else:
            lp = None
        sizes = (B, Hq, N, max_pages)
        need = cache._need.get(sizes)
        if need is None:
            need = cache._need[sizes] = attn_fwd_kv4_workspace_bytes(B, Hq, cache.heads, N, cache.d, cache.page_size,
                                                                     max_pages)
        if workspace is None:
            # (a shape the library refuses needs none: the call below says why)
            workspace = _kv4_workspace(cache, sp, need) if need else None
        elif workspace.get_device() != cache._index or workspace.dtype is not torch.uint8 or \
                not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {need} bytes on {cache.device}")
        st = load().attn_fwd_kv4(cache._addr, q.data_ptr(), bt, sl, ql, o, lp,
                                 None if workspace is None else workspace.data_ptr(),
                                 0 if workspace is None else workspace.numel(), B, Hq, N, max_pages,
                                 0.0 if scale is None else float(scale), 1 if causal else 0, dt, sp)
        if st or check:
            _check(st, "attn_fwd_kv4")
            _check_device(check, sp, "attn_fwd_kv4")
    finally:
        if place is not None:
            place.leave()
    return out, lse


def flops(B, H, N, d, causal):
    """Algorithmic FLOPs of one forward: 4 B H N^2 d, halved for causal."""
    f = 4.0 * B * H * N * N * d
    return f / 2 if causal else f


def default_scale(d):
    return 1.0 / math.sqrt(d)
