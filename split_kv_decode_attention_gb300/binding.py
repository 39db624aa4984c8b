"""Thin ctypes binding of libdecode_attn.so (C ABI in include/decode_attn.h).

Argument marshalling only: torch tensors supply device memory and streams,
every step of the computation runs in the library's CUDA kernels.  The names
mirror the C entry points.  There is no fallback: if the library is missing or
no GPU is present, the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libdecode_attn.so")

HEAD_DIM = 128
MAX_ROWS = 128
TOKEN_TILE = 16

DA_OK = 0
DA_STATUS_BAD_PAGE = 1
DA_STATUS_SEQ_LEN = 2
DA_STATUS_SHORT_CAUSAL = 4
DA_STATUS_TIMEOUT = 8
DA_STATUS_POSITION = 16
DA_CACHE_BF16 = 0
DA_CACHE_FP8_E4M3 = 1
DA_CACHE_FP4_E2M1 = 2
DA_FLAG_TWO_PASS = 1
DA_FLAG_KV_FP8_E4M3 = 2
DA_FLAG_TEST_WITHHOLD_COPY = 0x100
DA_ERR_UNSUPPORTED = -12

EXPORTED_SYMBOLS = (
    "decode_attn_params_init", "decode_attn_plan", "decode_attn_plan_slots", "decode_attn_chunk_len",
    "decode_attn_workspace_bytes", "decode_attn", "decode_attn_split", "decode_attn_combine",
    "decode_attn_status_string", "decode_attn_launch_count", "decode_attn_static_workspace",
    "decode_attn_host_workspace_bytes", "decode_attn_host", "decode_attn_device_plan",
    "decode_attn_cached", "decode_attn_cached_workspace_bytes", "decode_attn_rope_table",
    "decode_attn_rope_append", "decode_attn_block_digest", "decode_attn_block_select",
    "decode_attn_block_select_workspace_bytes", "decode_attn_sparse",
    "decode_attn_sparse_workspace_bytes",
)
DA_ERR_STATIC_WORKSPACE_LIMIT = -11
STATIC_WORKSPACE_BYTES = 16 << 20


class DecodeAttnParams(ctypes.Structure):
    """Mirror of `decode_attn_params` (same field order and types)."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("q_len", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32), ("causal", ctypes.c_int32),
        ("scale", ctypes.c_float), ("flags", ctypes.c_int32),
        ("q_stride_batch", ctypes.c_int64), ("q_stride_token", ctypes.c_int64),
        ("q_stride_head", ctypes.c_int64), ("o_stride_batch", ctypes.c_int64),
        ("o_stride_token", ctypes.c_int64), ("o_stride_head", ctypes.c_int64),
        ("kv_stride_page", ctypes.c_int64), ("kv_stride_token", ctypes.c_int64),
        ("kv_stride_head", ctypes.c_int64), ("block_table_stride", ctypes.c_int64),
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
    ]


class DecodeAttnCache(ctypes.Structure):
    """Mirror of `decode_attn_cache`."""

    _fields_ = [
        ("type", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_block_scale", ctypes.c_void_p), ("v_block_scale", ctypes.c_void_p),
        ("bs_stride_page", ctypes.c_int64), ("bs_stride_head", ctypes.c_int64),
    ]


class DecodeAttnRope(ctypes.Structure):
    """Mirror of `decode_attn_rope`."""

    _fields_ = [
        ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("table_positions", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("k_stride_batch", ctypes.c_int64), ("k_stride_token", ctypes.c_int64),
        ("k_stride_head", ctypes.c_int64), ("v_stride_batch", ctypes.c_int64),
        ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
    ]


class DecodeAttnSelect(ctypes.Structure):
    """Mirror of `decode_attn_select`."""

    _fields_ = [("top_k", ctypes.c_int32), ("sink", ctypes.c_int32),
                ("local", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class DecodeAttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where} failed: {decode_attn_status_string(code)} (code {code})")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(DecodeAttnParams)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        pi32 = ctypes.POINTER(ctypes.c_int32)
        L.decode_attn_params_init.argtypes = [P] + [i32] * 10
        L.decode_attn_params_init.restype = None
        L.decode_attn_plan.argtypes = [P, vp, pi32, pi32]
        L.decode_attn_plan_slots.argtypes = [P, vp, ctypes.c_int64, pi32, pi32]
        L.decode_attn_chunk_len.argtypes = [P, i32, pi32]
        L.decode_attn_workspace_bytes.argtypes = [P, i32, ctypes.POINTER(sz)]
        L.decode_attn.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp, vp]
        L.decode_attn_split.argtypes = L.decode_attn.argtypes
        L.decode_attn_static_workspace.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp]
        L.decode_attn_combine.argtypes = [P, vp, i32, i32, vp, sz, vp, vp, vp]
        L.decode_attn_status_string.argtypes = [ctypes.c_int]
        L.decode_attn_status_string.restype = ctypes.c_char_p
        L.decode_attn_launch_count.argtypes = [P, i32]
        L.decode_attn_host_workspace_bytes.argtypes = [P, i32, ctypes.POINTER(sz)]
        L.decode_attn_host.argtypes = L.decode_attn.argtypes
        L.decode_attn_device_plan.argtypes = [P, vp, vp, sz, vp, vp]
        C, R, S = (ctypes.POINTER(t) for t in (DecodeAttnCache, DecodeAttnRope, DecodeAttnSelect))
        i64, psz = ctypes.c_int64, ctypes.POINTER(sz)
        L.decode_attn_cached_workspace_bytes.argtypes = [P, C, i32, psz]
        L.decode_attn_cached.argtypes = [P, C, vp, vp, vp, vp, vp, i32, vp, sz, vp, vp]
        L.decode_attn_rope_table.argtypes = [vp, i32, i64, i64, ctypes.c_double, vp, vp]
        L.decode_attn_rope_append.argtypes = [P, C, R] + [vp] * 11
        L.decode_attn_block_digest.argtypes = [P, C, vp, vp, i32, vp, vp, vp, vp]
        L.decode_attn_block_select_workspace_bytes.argtypes = [P, S, psz]
        L.decode_attn_block_select.argtypes = [P, S] + [vp] * 9 + [sz, vp, vp]
        L.decode_attn_sparse_workspace_bytes.argtypes = [P, C, S, psz]
        L.decode_attn_sparse.argtypes = [P, C, S] + [vp] * 9 + [sz, vp, vp]
        for f in ("decode_attn_plan", "decode_attn_plan_slots", "decode_attn_chunk_len",
                  "decode_attn_workspace_bytes",
                  "decode_attn", "decode_attn_split", "decode_attn_combine",
                  "decode_attn_launch_count", "decode_attn_static_workspace",
                  "decode_attn_host_workspace_bytes", "decode_attn_host",
                  "decode_attn_device_plan", "decode_attn_cached",
                  "decode_attn_cached_workspace_bytes", "decode_attn_rope_table",
                  "decode_attn_rope_append", "decode_attn_block_digest",
                  "decode_attn_block_select", "decode_attn_block_select_workspace_bytes",
                  "decode_attn_sparse", "decode_attn_sparse_workspace_bytes"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def decode_attn_status_string(code: int) -> str:
    return lib().decode_attn_status_string(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != DA_OK:
        raise DecodeAttnError(code, where)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def decode_attn_params_init(batch: int, q_len: int, num_q_heads: int, num_kv_heads: int,
                            head_dim: int = HEAD_DIM, page_size: int = 0,
                            max_pages_per_seq: int = 0, num_pages: int = 0,
                            max_seq_len: int = 0, causal: bool = False) -> DecodeAttnParams:
    p = DecodeAttnParams()
    lib().decode_attn_params_init(ctypes.byref(p), batch, q_len, num_q_heads, num_kv_heads,
                                  head_dim, page_size, max_pages_per_seq, num_pages,
                                  max_seq_len, 1 if causal else 0)
    return p


def params_from_tensors(q, k_cache, block_table=None, *, max_seq_len: int,
                        causal: bool = False, scale: Optional[float] = None,
                        out=None, two_pass: bool = False, k_scale: float = 1.0,
                        v_scale: float = 1.0) -> DecodeAttnParams:
    """Describe torch tensors: q/out [B, q_len, Hq, D]; k_cache paged
    [P, page_size, Hkv, D] (block_table [B, max_pages] given) or contiguous
    [B, S, Hkv, D].  Strides are taken from the tensors.  A one-byte cache
    (uint8 or float8_e4m3fn) is an FP8 E4M3 cache with the given scales."""
    B, T, Hq, D = q.shape
    n0, n1, Hkv, D2 = k_cache.shape
    if D2 != D:
        raise ValueError("head_dim of q and k_cache differ")
    p = DecodeAttnParams()
    p.batch, p.q_len, p.num_q_heads, p.num_kv_heads, p.head_dim = B, T, Hq, Hkv, D
    p.max_seq_len = int(max_seq_len)
    p.causal = 1 if causal else 0
    p.flags = DA_FLAG_TWO_PASS if two_pass else 0
    if k_cache.element_size() == 1:
        p.flags |= DA_FLAG_KV_FP8_E4M3
    p.k_scale, p.v_scale = float(k_scale), float(v_scale)
    p.scale = float(scale if scale is not None else 1.0 / math.sqrt(D))
    p.q_stride_batch, p.q_stride_token, p.q_stride_head = (int(s) for s in q.stride()[:3])
    o = out if out is not None else q
    p.o_stride_batch, p.o_stride_token, p.o_stride_head = (int(s) for s in o.stride()[:3])
    p.kv_stride_page, p.kv_stride_token, p.kv_stride_head = (int(s) for s in k_cache.stride()[:3])
    if block_table is not None:
        p.page_size = n1
        p.num_pages = n0
        p.max_pages_per_seq = block_table.shape[1]
        p.block_table_stride = int(block_table.stride(0))
    return p


def decode_attn_plan(p: DecodeAttnParams, host_seq_lens=None) -> Tuple[int, int]:
    import numpy as np
    ns, cl = ctypes.c_int32(), ctypes.c_int32()
    arr = None
    if host_seq_lens is not None:
        arr = np.ascontiguousarray(host_seq_lens, dtype=np.int32)
    _check(lib().decode_attn_plan(ctypes.byref(p),
                                  None if arr is None else arr.ctypes.data,
                                  ctypes.byref(ns), ctypes.byref(cl)), "decode_attn_plan")
    return ns.value, cl.value


def decode_attn_plan_slots(p: DecodeAttnParams, host_seq_lens, resident_ctas: int) -> Tuple[int, int]:
    """The planner for an explicit number of resident split CTAs (host only)."""
    import numpy as np
    ns, cl = ctypes.c_int32(), ctypes.c_int32()
    arr = None
    if host_seq_lens is not None:
        arr = np.ascontiguousarray(host_seq_lens, dtype=np.int32)
    _check(lib().decode_attn_plan_slots(ctypes.byref(p),
                                        None if arr is None else arr.ctypes.data,
                                        int(resident_ctas), ctypes.byref(ns), ctypes.byref(cl)),
           "decode_attn_plan_slots")
    return ns.value, cl.value


def decode_attn_chunk_len(p: DecodeAttnParams, num_splits: int) -> int:
    c = ctypes.c_int32()
    _check(lib().decode_attn_chunk_len(ctypes.byref(p), int(num_splits), ctypes.byref(c)),
           "decode_attn_chunk_len")
    return c.value


def decode_attn_workspace_bytes(p: DecodeAttnParams, num_splits: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().decode_attn_workspace_bytes(ctypes.byref(p), int(num_splits), ctypes.byref(n)),
           "decode_attn_workspace_bytes")
    return n.value


def decode_attn_launch_count(p: DecodeAttnParams, num_splits: int) -> int:
    n = lib().decode_attn_launch_count(ctypes.byref(p), int(num_splits))
    if n < 0:
        raise DecodeAttnError(n, "decode_attn_launch_count")
    return n


def decode_attn(q, k_cache, v_cache, block_table, seq_lens, *, max_seq_len: int,
                causal: bool = False, scale: Optional[float] = None, num_splits: int = 0,
                out=None, lse=None, workspace=None, status=None, stream=None,
                params: Optional[DecodeAttnParams] = None, two_pass: bool = False,
                k_scale: float = 1.0, v_scale: float = 1.0, k_sf=None, v_sf=None):
    """Run decode attention; returns (out bf16 [B, q_len, Hq, D], lse fp32
    [B, q_len, Hq]).  Output, LSE and workspace tensors are allocated with
    torch when not given; `num_splits <= 0` lets the library's planner choose
    (on the device, from the lengths in `seq_lens`, for two or more requests).
    With block scales `k_sf`, `v_sf` (uint8 E4M3 [P, Hkv, page_size, 8], or [B,
    Hkv, S, 8]) the caches hold 4 bits per value: uint8 [P, page_size, Hkv, 64]
    (or [B, S, Hkv, 64])."""
    import torch

    if k_sf is not None or v_sf is not None:
        return _decode_attn_fp4(q, k_cache, v_cache, k_sf, v_sf, block_table, seq_lens,
                                max_seq_len, causal, scale, num_splits, out, lse, workspace,
                                status, stream, params, two_pass, k_scale, v_scale)
    B, T, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
    p = params if params is not None else params_from_tensors(
        q, k_cache, block_table, max_seq_len=max_seq_len, causal=causal, scale=scale, out=out,
        two_pass=two_pass, k_scale=k_scale, v_scale=v_scale)
    num_splits = max(0, int(num_splits))
    need = decode_attn_workspace_bytes(p, num_splits)
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty((need + 15) // 16 * 4, dtype=torch.float32, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().decode_attn(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                             _ptr(block_table), _ptr(seq_lens), _ptr(out), _ptr(lse),
                             int(num_splits), _ptr(workspace) if need > 0 else None, ws_bytes,
                             _ptr(status), _stream_handle(stream)), "decode_attn")
    return out, lse


def decode_attn_host_workspace_bytes(p: DecodeAttnParams, num_splits: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().decode_attn_host_workspace_bytes(ctypes.byref(p), int(num_splits),
                                                  ctypes.byref(n)),
           "decode_attn_host_workspace_bytes")
    return n.value


def decode_attn_host(q_host, k_cache, v_cache, block_table_host, seq_lens_host, *,
                     max_seq_len: int, causal: bool = False, scale: Optional[float] = None,
                     num_splits: int = 0, out_host=None, lse_host=None, workspace=None,
                     stream=None, params: Optional[DecodeAttnParams] = None,
                     two_pass: bool = False, k_scale: float = 1.0, v_scale: float = 1.0):
    """decode_attn with q, block table and seq_lens in host memory (torch CPU
    tensors, ideally pinned) and out / lse returned to host memory; the K/V
    cache stays on the device.  One C call: with pinned buffers the kernels
    read and write them in place, otherwise copies in and out; the stream is
    synchronised.  Returns (out_host, lse_host, status bits)."""
    import numpy as np
    import torch

    B, T, Hq, D = q_host.shape
    if out_host is None:
        out_host = torch.empty((B, T, Hq, D), dtype=torch.bfloat16).pin_memory()
    if lse_host is None:
        lse_host = torch.empty((B, T, Hq), dtype=torch.float32).pin_memory()
    p = params if params is not None else params_from_tensors(
        q_host, k_cache, block_table_host, max_seq_len=max_seq_len, causal=causal, scale=scale,
        out=out_host, two_pass=two_pass, k_scale=k_scale, v_scale=v_scale)
    if workspace is None:   # (a given workspace is checked by the C call itself)
        if num_splits <= 0:  # the library's planner, with the actual lengths
            num_splits, _ = decode_attn_plan(p, np.asarray(seq_lens_host, dtype=np.int32))
        need = decode_attn_host_workspace_bytes(p, num_splits)
        workspace = torch.empty((need + 15) // 16 * 4, dtype=torch.float32, device=k_cache.device)
    global _host_status
    if _host_status is None:   # a page-locked word: the kernels write it in place
        _host_status = torch.zeros(1, dtype=torch.int32).pin_memory()
    status_ptr = _host_status.data_ptr()
    _check(lib().decode_attn_host(ctypes.byref(p), _ptr(q_host), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(block_table_host), _ptr(seq_lens_host), _ptr(out_host),
                                  _ptr(lse_host), int(num_splits), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  status_ptr, _stream_handle(stream)),
           "decode_attn_host")
    return out_host, lse_host, ctypes.c_int32.from_address(status_ptr).value


_host_status = None


def decode_attn_device_plan(p: DecodeAttnParams, seq_lens, workspace, status=None, stream=None):
    """Run the device planner alone (the first launch of a device-planned
    decode_attn call) into `workspace`; read the plan back with
    device_plan_view()."""
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().decode_attn_device_plan(ctypes.byref(p), _ptr(seq_lens), _ptr(workspace),
                                         ws_bytes, _ptr(status), _stream_handle(stream)),
           "decode_attn_device_plan")


def device_plan_view(workspace, p: DecodeAttnParams):
    """(plan int32[4] = chunk_len, items, chunks of the longest request,
    capacity; pre int32[B + 1]; items int32[capacity, 4] = (b, kv head, chunk,
    length)) views of a device-planned call's workspace, per the layout in the
    header."""
    import torch
    b = workspace.view(-1).view(torch.int32)

    def r256(x):
        return (x + 255) // 256 * 256

    plan = b[:4]
    off = 256
    pre = b[off // 4: off // 4 + p.batch + 1]
    off = r256(off + (p.batch + 1) * 4)
    cap = int(plan[3].item())
    items = b[off // 4: off // 4 + 4 * cap].view(cap, 4)
    return plan, pre, items


def decode_attn_combine(p: DecodeAttnParams, seq_lens, num_splits: int, chunk_len: int,
                        workspace, out, lse, stream=None):
    """Merge the partials held in `workspace` into out/lse (rows of requests
    spanning two or more chunks); num_splits <= 0 after a device-planned
    split pass."""
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().decode_attn_combine(ctypes.byref(p), _ptr(seq_lens), int(num_splits),
                                     int(chunk_len), _ptr(workspace), ws_bytes, _ptr(out),
                                     _ptr(lse), _stream_handle(stream)), "decode_attn_combine")
    return out, lse


def workspace_views(workspace, p: DecodeAttnParams, num_splits: int):
    """(part_o [B, q_len, Hq, S, D], part_lse [B, q_len, Hq, S]) views of a
    workspace tensor, per the layout documented for decode_attn_workspace_bytes."""
    S = num_splits
    rows = p.batch * p.q_len * p.num_q_heads
    f = workspace.view(-1)[: rows * S * (HEAD_DIM + 1)]
    po = f[: rows * S * HEAD_DIM].view(p.batch, p.q_len, p.num_q_heads, S, HEAD_DIM)
    pl = f[rows * S * HEAD_DIM:].view(p.batch, p.q_len, p.num_q_heads, S)
    return po, pl


def decode_attn_split(p: DecodeAttnParams, q, k_cache, v_cache, block_table, seq_lens, out,
                      lse, num_splits: int, workspace=None, status=None, stream=None):
    """The split pass alone (same arguments as the C entry point): final
    out/lse for requests that fit one chunk, partials in `workspace` for the
    rest; decode_attn_combine() with the same num_splits finishes them."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().decode_attn_split(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(block_table), _ptr(seq_lens), _ptr(out), _ptr(lse),
                                   int(num_splits), _ptr(workspace), ws_bytes, _ptr(status),
                                   _stream_handle(stream)), "decode_attn_split")
    return out, lse


def decode_attn_static_workspace(p: DecodeAttnParams, q, k_cache, v_cache, block_table,
                                 seq_lens, out, lse, num_splits: int = 0, status=None,
                                 stream=None):
    """decode_attn() without a caller workspace, for callers that cannot
    allocate device memory: the partials live in the library's fixed 16 MiB
    device array (shared by all calls on a device; overlapping calls race).
    Raises DecodeAttnError(-11) when a call needs more than that."""
    _check(lib().decode_attn_static_workspace(
        ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(seq_lens), _ptr(out), _ptr(lse), int(num_splits), _ptr(status),
        _stream_handle(stream)), "decode_attn_static_workspace")
    return out, lse


# ---------------------------------------------------------------------------
# The operators around the cache

def _dtype(t, want, name):
    if t.dtype not in want:
        raise ValueError(f"{name} is {t.dtype}; expected {' or '.join(str(w) for w in want)}")


def _on_current_device(*tensors):
    """Every given tensor lies on the current CUDA device (the one whose stream
    the call takes and whose planner it asks)."""
    import torch
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"a tensor is on {t.device}, the current CUDA device is {cur}")


def _cache_args(k_cache, v_cache, k_sf, v_sf, block_table):
    """(DecodeAttnCache, groups, tokens, kv heads) of cache tensors."""
    import torch
    if k_sf is not None or v_sf is not None:
        ctype, width = DA_CACHE_FP4_E2M1, HEAD_DIM // 2
        if k_sf is None or (v_cache is not None and v_sf is None):
            raise ValueError("a 4-bit cache needs the block scales of K and of V")
        _dtype(k_cache, (torch.uint8,), "k_cache")
    elif k_cache.element_size() == 1:
        ctype, width = DA_CACHE_FP8_E4M3, HEAD_DIM
        _dtype(k_cache, (torch.uint8, torch.float8_e4m3fn), "k_cache")
    else:
        ctype, width = DA_CACHE_BF16, HEAD_DIM
        _dtype(k_cache, (torch.bfloat16,), "k_cache")
    if k_cache.dim() != 4 or k_cache.shape[3] != width or k_cache.stride(3) != 1:
        raise ValueError(f"k_cache must be [groups, tokens, heads, {width}], its last dimension dense")
    if v_cache is not None and (v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride()
                                or v_cache.dtype != k_cache.dtype):
        raise ValueError("k_cache and v_cache differ in shape, strides or type")
    groups, tokens, heads, _ = k_cache.shape
    c = DecodeAttnCache()
    c.type = ctype
    c.k, c.v = _ptr(k_cache), _ptr(v_cache)
    if ctype == DA_CACHE_FP4_E2M1:
        for t, name in ((k_sf, "k_sf"), (v_sf, "v_sf")):
            if t is None:
                continue
            _dtype(t, (torch.uint8, torch.float8_e4m3fn), name)
            if t.shape != (groups, heads, tokens, 8) or t.stride()[2:] != (8, 1):
                raise ValueError(f"{name} must be [{groups}, {heads}, {tokens}, 8] with dense tokens")
        if v_sf is not None and v_sf.stride() != k_sf.stride():
            raise ValueError("k_sf and v_sf differ in strides")
        c.k_block_scale, c.v_block_scale = _ptr(k_sf), _ptr(v_sf)
        c.bs_stride_page, c.bs_stride_head = k_sf.stride(0), k_sf.stride(1)
    _dtype_int(block_table, "block_table")
    return c, groups, tokens, heads


def _dtype_int(t, name):
    import torch
    if t is not None:
        _dtype(t, (torch.int32,), name)
        if t.dim() > 0 and t.numel() > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must be dense in its last dimension")


def _cache_params(B, T, Hq, k_cache, block_table, max_seq_len, causal, scale, k_scale, v_scale,
                  flags=0):
    groups, tokens, heads, _ = k_cache.shape
    p = DecodeAttnParams()
    p.batch, p.q_len, p.num_q_heads, p.num_kv_heads, p.head_dim = B, T, Hq, heads, HEAD_DIM
    p.max_seq_len, p.causal, p.flags = int(max_seq_len), 1 if causal else 0, flags
    p.scale = float(scale if scale is not None else 1.0 / math.sqrt(HEAD_DIM))
    p.kv_stride_page, p.kv_stride_token, p.kv_stride_head = k_cache.stride()[:3]
    p.k_scale, p.v_scale = float(k_scale), float(v_scale)
    if block_table is not None:
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [batch, pages]")
        p.page_size, p.num_pages = tokens, groups
        p.max_pages_per_seq, p.block_table_stride = block_table.shape[1], block_table.stride(0)
    elif groups != B or tokens < max_seq_len:
        raise ValueError("a contiguous cache holds max_seq_len tokens of every request")
    return p


def _q_strides(p, q, out):
    p.q_stride_batch, p.q_stride_token, p.q_stride_head = q.stride()[:3]
    p.o_stride_batch, p.o_stride_token, p.o_stride_head = out.stride()[:3]


def _heads_tensor(t, B, T, name):
    import torch
    _dtype(t, (torch.bfloat16,), name)
    if t.dim() != 4 or t.shape[0] != B or t.shape[1] != T or t.shape[3] != HEAD_DIM or t.stride(3) != 1:
        raise ValueError(f"{name} must be [{B}, {T}, heads, {HEAD_DIM}], its last dimension dense")


def _lens_tensor(t, B, name="seq_lens"):
    _dtype_int(t, name)
    if t.shape != (B,):
        raise ValueError(f"{name} must be [{B}]")


def _outputs(q, out, lse):
    import torch
    B, T, Hq, D = q.shape
    if out is None:
        out = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=q.device)
    else:
        _heads_tensor(out, B, T, "out")
        if out.shape[2] != Hq:
            raise ValueError("out and q differ in heads")
    if lse is None:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
    else:
        _dtype(lse, (torch.float32,), "lse")
        if lse.shape != (B, T, Hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be dense [{B}, {T}, {Hq}]")
    return out, lse


def _workspace(given, need, device):
    import torch
    if need == 0:
        return given
    if given is None or given.numel() * given.element_size() < need:
        return torch.empty((need + 15) // 16 * 4, dtype=torch.float32, device=device)
    return given


def _status_word(status):
    import torch
    if status is not None:
        _dtype(status, (torch.int32,), "status")
    return _ptr(status)


def _decode_attn_fp4(q, k_cache, v_cache, k_sf, v_sf, block_table, seq_lens, max_seq_len, causal,
                     scale, num_splits, out, lse, workspace, status, stream, params, two_pass,
                     k_scale, v_scale):
    B, T, Hq, _ = q.shape
    _heads_tensor(q, B, T, "q")
    _lens_tensor(seq_lens, B)
    c, _, _, heads = _cache_args(k_cache, v_cache, k_sf, v_sf, block_table)
    _on_current_device(q, k_cache, v_cache, k_sf, v_sf, block_table, seq_lens, out, lse, workspace,
                       status)
    out, lse = _outputs(q, out, lse)
    p = params
    if p is None:
        p = _cache_params(B, T, Hq, k_cache, block_table, max_seq_len, causal, scale, k_scale,
                          v_scale, DA_FLAG_TWO_PASS if two_pass else 0)
        _q_strides(p, q, out)
    num_splits = max(0, int(num_splits))
    n = ctypes.c_size_t()
    _check(lib().decode_attn_cached_workspace_bytes(ctypes.byref(p), ctypes.byref(c), num_splits,
                                                    ctypes.byref(n)),
           "decode_attn_cached_workspace_bytes")
    workspace = _workspace(workspace, n.value, q.device)
    _check(lib().decode_attn_cached(
        ctypes.byref(p), ctypes.byref(c), _ptr(q), _ptr(block_table), _ptr(seq_lens), _ptr(out),
        _ptr(lse), num_splits, _ptr(workspace), 0 if workspace is None else
        workspace.numel() * workspace.element_size(), _status_word(status),
        _stream_handle(stream)), "decode_attn_cached")
    return out, lse


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
                     factor: float = 1.0, original_positions: int = 8192, low: float = 1.0,
                     high: float = 4.0, beta_slow: float = 1.0, beta_fast: float = 32.0):
    """(inv_freq float64 [rotary_dim / 2] on the CPU, amplitude) for rope_table():
    base^(-2i / rotary_dim), scaled for contexts `factor` times longer than the
    `original_positions` a model was trained on.

      None        as they are
      "linear"    every frequency divided by factor
      "ntk"       the base raised to base * factor^(rotary_dim / (rotary_dim - 2)),
                  which divides the slowest frequency by factor and leaves the fastest
      "by_parts"  frequencies that turn at least `high` times over the original
                  positions as they are, at most `low` times divided by factor, a
                  linear ramp (in turns) between
      "yarn"      a linear ramp in i between the pairs that turn beta_fast and
                  beta_slow times over the original positions (rounded outwards),
                  and the amplitude 0.1 ln(factor) + 1"""
    import torch
    if rotary_dim < 2 or rotary_dim % 2 or rotary_dim > HEAD_DIM:
        raise ValueError(f"rotary_dim must be even, 2 .. {HEAD_DIM}")
    if not base > 1.0 or not factor > 0.0 or original_positions < 1:
        raise ValueError("base > 1, factor > 0 and original_positions >= 1 are needed")
    n = rotary_dim // 2
    i = torch.arange(n, dtype=torch.float64)
    if scaling == "ntk":
        if rotary_dim == 2:
            raise ValueError('"ntk" needs rotary_dim of 4 or more')
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-i / n)
    amplitude = 1.0
    if scaling is None or scaling == "ntk":
        pass
    elif scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        if not high > low:
            raise ValueError("high must exceed low")
        turns = original_positions * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (keep + (1 - keep) / factor)
    elif scaling == "yarn":
        def pair_at(turns):  # the (real) pair index that turns this often
            return n * math.log(original_positions / (turns * 2 * math.pi)) / math.log(base)
        first = max(math.floor(pair_at(beta_fast)), 0)
        last = min(math.ceil(pair_at(beta_slow)), rotary_dim - 1)
        ramp = ((i - first) / max(last - first, 0.001)).clamp(0.0, 1.0)
        f = f * (1 - ramp + ramp / factor)
        amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    else:
        raise ValueError(f"unknown scaling {scaling!r}")
    return f, amplitude


def rope_table(inv_freq, max_pos: int, *, amplitude: float = 1.0, first: int = 0, out=None,
               stream=None):
    """fp32 [max_pos, 2 n]: amplitude * cos, then sin, of (first + row) * inv_freq,
    for inv_freq float64 [n] in device memory (rope_frequencies() gives it)."""
    import torch
    _dtype(inv_freq, (torch.float64,), "inv_freq")
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a dense vector")
    _on_current_device(inv_freq, out)
    n = inv_freq.shape[0]
    if out is None:
        out = torch.empty((max_pos, 2 * n), dtype=torch.float32, device=inv_freq.device)
    else:
        _dtype(out, (torch.float32,), "out")
        if out.shape != (max_pos, 2 * n) or not out.is_contiguous():
            raise ValueError(f"out must be dense [{max_pos}, {2 * n}]")
    _check(lib().decode_attn_rope_table(_ptr(inv_freq), n, int(first), int(max_pos),
                                        float(amplitude), _ptr(out), _stream_handle(stream)),
           "decode_attn_rope_table")
    return out


def rope_append(q, k, v, table, k_cache, v_cache, block_table, seq_lens, *, max_seq_len: int,
                interleaved: bool = False, positions=None, new_lens=None, k_scale: float = 1.0,
                v_scale: float = 1.0, k_sf=None, v_sf=None, q_out=None, status=None, stream=None):
    """Rotate the new tokens' q and k (bf16 [B, q_len, heads, 128]) and write k and
    v into the caches at the last q_len (or new_lens[b]) of each request's
    seq_lens[b] tokens; returns q_out.  `table` is rope_table()'s [positions,
    rotary_dim] (None: no rotation), `positions` int32 [B, q_len] overrides the
    cache positions as angles.  k and v None: only q is rotated; q None: only
    the caches are written.  q_out may be q."""
    import torch
    lead = q if q is not None else k
    if lead is None or (k is None) != (v is None):
        raise ValueError("q, or k and v, or all three are needed")
    B, T = lead.shape[:2]
    c, _, _, heads = _cache_args(k_cache, v_cache, k_sf, v_sf, block_table)
    if c.type == DA_CACHE_FP4_E2M1 and v_sf is None:
        raise ValueError("a 4-bit cache needs the block scales of K and of V")
    _lens_tensor(seq_lens, B)
    r = DecodeAttnRope()
    if table is not None:
        _dtype(table, (torch.float32,), "table")
        if table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be dense [positions, rotary_dim]")
        r.table_positions, r.rotary_dim = table.shape
    r.interleaved = 1 if interleaved else 0
    if k is not None:
        for t, name in ((k, "k"), (v, "v")):
            _heads_tensor(t, B, T, name)
            if t.shape[2] != heads:
                raise ValueError(f"{name} has {t.shape[2]} heads, the cache {heads}")
        r.k_stride_batch, r.k_stride_token, r.k_stride_head = k.stride()[:3]
        r.v_stride_batch, r.v_stride_token, r.v_stride_head = v.stride()[:3]
    p = _cache_params(B, T, heads, k_cache, block_table, max_seq_len, False, 1.0, k_scale, v_scale)
    if q is not None:
        _heads_tensor(q, B, T, "q")
        if q.shape[2] % heads:
            raise ValueError(f"{q.shape[2]} query heads are no multiple of {heads}")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        else:
            _heads_tensor(q_out, B, T, "q_out")
            if q_out.shape != q.shape:
                raise ValueError("q_out and q differ in shape")
        p.num_q_heads = q.shape[2]
        _q_strides(p, q, q_out)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if positions is not None:
        _dtype_int(positions, "positions")
        if positions.shape != (B, T) or not positions.is_contiguous():
            raise ValueError(f"positions must be dense [{B}, {T}]")
    if new_lens is not None:
        _lens_tensor(new_lens, B, "new_lens")
    _on_current_device(q, k, v, table, k_cache, v_cache, k_sf, v_sf, block_table, seq_lens, q_out,
                       positions, new_lens, status)
    _check(lib().decode_attn_rope_append(
        ctypes.byref(p), ctypes.byref(c), ctypes.byref(r), _ptr(q), _ptr(k), _ptr(v), _ptr(table),
        _ptr(positions), _ptr(new_lens), _ptr(block_table), _ptr(seq_lens), _ptr(q_out),
        _status_word(status), _stream_handle(stream)), "decode_attn_rope_append")
    return q_out


def _digest_tensors(digest, digest_scale, pages, heads):
    import torch
    _dtype(digest, (torch.int8,), "digest")
    _dtype(digest_scale, (torch.float32,), "digest_scale")
    if digest.shape != (pages, heads, 2, HEAD_DIM) or not digest.is_contiguous():
        raise ValueError(f"digest must be dense [{pages}, {heads}, 2, {HEAD_DIM}]")
    if digest_scale.shape != (pages, heads) or not digest_scale.is_contiguous():
        raise ValueError(f"digest_scale must be dense [{pages}, {heads}]")


def block_digest(k_cache, block_table, seq_lens, digest=None, digest_scale=None, *,
                 max_seq_len: int, max_new: int = 0, k_sf=None, status=None, stream=None):
    """Digest the pages of a paged K cache for decode_attn_sparse(): (digest int8
    [P, Hkv, 2, 128], digest_scale fp32 [P, Hkv]), allocated (zero) when not
    given.  max_new > 0 digests only the pages that hold each request's last
    max_new tokens: what a decode step has changed."""
    import torch
    if block_table is None:
        raise ValueError("digests are per page: a block_table is needed")
    B = block_table.shape[0]
    c, pages, _, heads = _cache_args(k_cache, None, k_sf, None, block_table)
    _lens_tensor(seq_lens, B)
    if digest is None:
        digest = torch.zeros((pages, heads, 2, HEAD_DIM), dtype=torch.int8, device=k_cache.device)
    if digest_scale is None:
        digest_scale = torch.zeros((pages, heads), dtype=torch.float32, device=k_cache.device)
    _digest_tensors(digest, digest_scale, pages, heads)
    p = _cache_params(B, 1, heads, k_cache, block_table, max_seq_len, False, 1.0, 1.0, 1.0)
    _on_current_device(k_cache, k_sf, block_table, seq_lens, digest, digest_scale, status)
    _check(lib().decode_attn_block_digest(
        ctypes.byref(p), ctypes.byref(c), _ptr(block_table), _ptr(seq_lens), int(max_new),
        _ptr(digest), _ptr(digest_scale), _status_word(status), _stream_handle(stream)),
        "decode_attn_block_digest")
    return digest, digest_scale


def _select_args(top_k, sink, local):
    s = DecodeAttnSelect()
    s.top_k, s.sink, s.local = int(top_k), int(sink), int(local)
    return s


def _blocks_tensor(blocks, shape):
    import torch
    _dtype(blocks, (torch.int32,), "blocks")
    if blocks.shape != shape or not blocks.is_contiguous():
        raise ValueError(f"blocks must be dense {list(shape)}")


def block_select(q, digest, digest_scale, block_table, seq_lens, *, page_size: int,
                 max_seq_len: int, top_k: int, sink: int = 1, local: int = 1,
                 causal: bool = False, blocks=None, workspace=None, status=None, stream=None):
    """The pages decode_attn_sparse() would read: (blocks int32 [B, q_len, Hkv,
    top_k], the pages' places in each request, ascending, -1 behind the last;
    pages, their ids; tokens int32 [B, q_len, Hkv], how many tokens they hold)."""
    import torch
    B, T, Hq, _ = q.shape
    _heads_tensor(q, B, T, "q")
    _dtype_int(block_table, "block_table")
    _lens_tensor(seq_lens, B)
    pages, heads = digest.shape[:2]
    _digest_tensors(digest, digest_scale, pages, heads)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [batch, pages]")
    p = DecodeAttnParams()
    p.batch, p.q_len, p.num_q_heads, p.num_kv_heads, p.head_dim = B, T, Hq, heads, HEAD_DIM
    p.page_size, p.num_pages, p.max_seq_len = int(page_size), pages, int(max_seq_len)
    p.max_pages_per_seq, p.block_table_stride = block_table.shape[1], block_table.stride(0)
    p.causal, p.scale = 1 if causal else 0, 1.0
    _q_strides(p, q, q)
    s = _select_args(top_k, sink, local)
    n = ctypes.c_size_t()
    _check(lib().decode_attn_block_select_workspace_bytes(ctypes.byref(p), ctypes.byref(s),
                                                          ctypes.byref(n)),
           "decode_attn_block_select_workspace_bytes")
    workspace = _workspace(workspace, n.value, q.device)
    shape = (B, T, heads, s.top_k)
    if blocks is None:
        blocks = torch.empty(shape, dtype=torch.int32, device=q.device)
    _blocks_tensor(blocks, shape)
    ids = torch.empty(shape, dtype=torch.int32, device=q.device)
    tokens = torch.empty(shape[:3], dtype=torch.int32, device=q.device)
    _on_current_device(q, digest, digest_scale, block_table, seq_lens, blocks, workspace, status)
    _check(lib().decode_attn_block_select(
        ctypes.byref(p), ctypes.byref(s), _ptr(q), _ptr(digest), _ptr(digest_scale),
        _ptr(block_table), _ptr(seq_lens), _ptr(blocks), _ptr(ids), _ptr(tokens), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _status_word(status), _stream_handle(stream)), "decode_attn_block_select")
    return blocks, ids, tokens


def decode_attn_sparse(q, k_cache, v_cache, block_table, seq_lens, digest, digest_scale, *,
                       max_seq_len: int, top_k: int, sink: int = 1, local: int = 1,
                       causal: bool = False, scale: Optional[float] = None, k_scale: float = 1.0,
                       v_scale: float = 1.0, k_sf=None, v_sf=None, out=None, lse=None,
                       blocks=None, workspace=None, status=None, stream=None):
    """Decode attention over the top_k pages per (token, KV head) that the digests
    of block_digest() score highest, the first `sink` and last `local` pages
    always among them: (out, lse, blocks).  Any cache type, as decode_attn()."""
    import torch
    B, T, Hq, _ = q.shape
    _heads_tensor(q, B, T, "q")
    _lens_tensor(seq_lens, B)
    if block_table is None:
        raise ValueError("the selection is of pages: a block_table is needed")
    c, pages, _, heads = _cache_args(k_cache, v_cache, k_sf, v_sf, block_table)
    _digest_tensors(digest, digest_scale, pages, heads)
    _on_current_device(q, k_cache, v_cache, k_sf, v_sf, block_table, seq_lens, digest, digest_scale,
                       out, lse, blocks, workspace, status)
    out, lse = _outputs(q, out, lse)
    p = _cache_params(B, T, Hq, k_cache, block_table, max_seq_len, causal, scale, k_scale, v_scale)
    _q_strides(p, q, out)
    s = _select_args(top_k, sink, local)
    shape = (B, T, heads, s.top_k)
    if blocks is None:
        blocks = torch.empty(shape, dtype=torch.int32, device=q.device)
    else:
        _blocks_tensor(blocks, shape)
    n = ctypes.c_size_t()
    _check(lib().decode_attn_sparse_workspace_bytes(ctypes.byref(p), ctypes.byref(c),
                                                    ctypes.byref(s), ctypes.byref(n)),
           "decode_attn_sparse_workspace_bytes")
    workspace = _workspace(workspace, n.value, q.device)
    _check(lib().decode_attn_sparse(
        ctypes.byref(p), ctypes.byref(c), ctypes.byref(s), _ptr(q), _ptr(digest),
        _ptr(digest_scale), _ptr(block_table), _ptr(seq_lens), _ptr(out), _ptr(lse), _ptr(blocks),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _status_word(status), _stream_handle(stream)), "decode_attn_sparse")
    return out, lse, blocks
