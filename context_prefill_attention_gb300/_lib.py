"""ctypes binding of libpcp (include/pcp.h). Argument marshalling only: every
step of the path runs in the library. The binding refuses to work without the
compiled library; there is no fallback of any kind."""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpcp.so")

PCP_OK = 0
PCP_ERR_ARG = -1
PCP_ERR_RANGE = -2
PCP_ERR_UNSUPPORTED = -3
PCP_ERR_ALIGN = -4
PCP_ERR_CUDA = -5
PCP_ERR_TIMEOUT = -6
PCP_ERR_WORKSPACE = -7
PCP_ERR_PAGES = -8

PCP_SPLIT_CONTIGUOUS = 0
PCP_SPLIT_DUAL_CHUNK = 1

PCP_ATTN_SEPARATE_CONTEXT = 1
PCP_ATTN_SPLIT_AT_ROW_START = 2


def PCP_ATTN_KV_SHARDS(n: int) -> int:
    """Flag: compute each prefill row as n partials over n contiguous key shards
    (decode-context-parallel emulation) and merge them by LSE."""
    return (int(n) & 0xFF) << 8


def PCP_ATTN_DECODE_SMS(n: int) -> int:
    """Flag: run the decode rows on n SMs beside the prefill rows (see
    :func:`pcp_decode_sms`)."""
    return (int(n) & 0xFF) << 16

ROW_FIELDS = ("req", "shard", "q_start", "q_len", "ctx_len", "kv_end", "causal_off", "is_decode")
PREFIX_FIELDS = ("q_start", "q_len", "req", "prefix_len")

# every symbol include/pcp.h declares
EXPORTS = ("pcp_build_row_plan", "pcp_mask_slots_for_shard", "pcp_decode_sms", "pcp_kv_cache_write",
           "pcp_kv_cache_write_fp8", "pcp_attn_workspace_size", "pcp_attn_varlen", "pcp_attn_varlen_noalloc",
           "pcp_attn_varlen_fp8kv", "pcp_lse_merge",
           "pcp_attn_window_workspace_size", "pcp_attn_window", "pcp_attn_window_fp8kv",
           "pcp_build_prefix_groups", "pcp_attn_shared_prefix_workspace_size", "pcp_attn_shared_prefix",
           "pcp_attn_shared_prefix_fp8kv", "pcp_kv_pages_workspace_size", "pcp_kv_fork", "pcp_kv_release",
           "pcp_kv_compact",
           "pcp_set_profile_events", "pcp_selftest_bounded_wait",
           "pcp_last_cuda_error", "pcp_status_string")

_lib = None


class PcpError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = "?"
        if _lib is not None:
            msg = _lib.pcp_status_string(code).decode()
        extra = ""
        if code == PCP_ERR_CUDA and _lib is not None:
            extra = f" (cudaError {_lib.pcp_last_cuda_error()})"
        super().__init__(f"{what}: {msg} [{code}]{extra}")
        self.code = code


def load(path: Optional[str] = None):
    """Load libpcp.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with context_prefill_attention_gb300.build.build() "
                           "(nvcc, sm_103a); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.pcp_build_row_plan.argtypes = [i32, P, P, P, i32, i32, i32, i32, P, i32, P, P, P, P]
    lib.pcp_build_row_plan.restype = ctypes.c_int
    lib.pcp_mask_slots_for_shard.argtypes = [P, P, i32, i32, P]
    lib.pcp_mask_slots_for_shard.restype = ctypes.c_int
    lib.pcp_decode_sms.argtypes = [P, i32, i32, i32, i32, i32, i32]
    lib.pcp_decode_sms.restype = i32
    lib.pcp_kv_cache_write.argtypes = [P, P, P, i32, P, P, i64, i32, i32, i32, P, P]
    lib.pcp_kv_cache_write.restype = ctypes.c_int
    lib.pcp_kv_cache_write_fp8.argtypes = [P, P, P, i32, P, P, i64, i32, i32, i32, f32, f32, P, P]
    lib.pcp_kv_cache_write_fp8.restype = ctypes.c_int
    lib.pcp_attn_varlen_fp8kv.argtypes = [P, P, P, P, P, P, i32, i32, i64, i32, P, i32, i32, i32, i32, i32, f32,
                                          P, P, P, sz, i32, P, P]
    lib.pcp_attn_varlen_fp8kv.restype = ctypes.c_int
    lib.pcp_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.pcp_attn_workspace_size.restype = sz
    lib.pcp_attn_varlen.argtypes = [P, P, P, P, i32, i32, i64, i32, P, i32, i32, i32, i32, i32, f32, P, P, P,
                                    sz, i32, P, P]
    lib.pcp_attn_varlen.restype = ctypes.c_int
    lib.pcp_lse_merge.argtypes = [P, P, P, P, P, P, i32, i32, i32, P]
    lib.pcp_lse_merge.restype = ctypes.c_int
    lib.pcp_attn_varlen_noalloc.argtypes = [P, P, P, P, i32, i32, i64, i32, P, i32, i32, i32, i32, i32, f32,
                                            P, P, i32, P, P]
    lib.pcp_attn_varlen_noalloc.restype = ctypes.c_int
    lib.pcp_attn_window_workspace_size.argtypes = [i32] * 9
    lib.pcp_attn_window_workspace_size.restype = sz
    lib.pcp_attn_window.argtypes = [P, P, P, P, i32, i32, i64, i32, P, i32, i32, i32, i32, i32, f32, i32, i32, P, P,
                                    P, sz, P, P]
    lib.pcp_attn_window.restype = ctypes.c_int
    lib.pcp_attn_window_fp8kv.argtypes = [P, P, P, P, P, P, i32, i32, i64, i32, P, i32, i32, i32, i32, i32, f32, i32,
                                          i32, P, P, P, sz, P, P]
    lib.pcp_attn_window_fp8kv.restype = ctypes.c_int
    lib.pcp_build_prefix_groups.argtypes = [P, i32, P, i32, i32, i32, i32, P, i32, P]
    lib.pcp_build_prefix_groups.restype = ctypes.c_int
    lib.pcp_attn_shared_prefix_workspace_size.argtypes = [i32] * 7
    lib.pcp_attn_shared_prefix_workspace_size.restype = sz
    lib.pcp_attn_shared_prefix.argtypes = [P, P, P, P, i32, i32, i64, i32, P, i32, P, i32, i32, i32, i32, i32, f32,
                                           P, P, P, sz, P, P]
    lib.pcp_attn_shared_prefix.restype = ctypes.c_int
    lib.pcp_attn_shared_prefix_fp8kv.argtypes = [P, P, P, P, P, P, i32, i32, i64, i32, P, i32, P, i32, i32, i32, i32,
                                                 i32, f32, P, P, P, sz, P, P]
    lib.pcp_attn_shared_prefix_fp8kv.restype = ctypes.c_int
    lib.pcp_kv_pages_workspace_size.argtypes = [i64]
    lib.pcp_kv_pages_workspace_size.restype = sz
    lib.pcp_kv_fork.argtypes = [P, P, i64, i32, i32, P, i32, i32, P, P, i32, P, P, P, P, sz, P, P]
    lib.pcp_kv_fork.restype = ctypes.c_int
    lib.pcp_kv_release.argtypes = [P, i32, i32, P, P, P, i64, P, P, P, P]
    lib.pcp_kv_release.restype = ctypes.c_int
    lib.pcp_kv_compact.argtypes = [P, P, i64, i32, i32, P, i32, i32, P, P, P, P, P, sz, P, P]
    lib.pcp_kv_compact.restype = ctypes.c_int
    lib.pcp_selftest_bounded_wait.argtypes = [P, ctypes.c_uint32, P]
    lib.pcp_selftest_bounded_wait.restype = ctypes.c_int
    lib.pcp_set_profile_events.argtypes = [P, P, P, P]
    lib.pcp_set_profile_events.restype = ctypes.c_int
    lib.pcp_last_cuda_error.argtypes = []
    lib.pcp_last_cuda_error.restype = ctypes.c_int
    lib.pcp_status_string.argtypes = [ctypes.c_int]
    lib.pcp_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def _t_ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(rc: int, what: str):
    if rc != PCP_OK:
        raise PcpError(rc, what)


BF16 = (torch.bfloat16,)
F32 = (torch.float32,)
I32 = (torch.int32,)
I64 = (torch.int64,)
# an FP8 cache holds one e4m3 code per byte: raw bytes or PyTorch's e4m3 "fn" type
FP8_CACHE = (torch.uint8,) + ((torch.float8_e4m3fn,) if hasattr(torch, "float8_e4m3fn") else ())

PAGE_CACHE = BF16 + FP8_CACHE

def _is_device_tensor(t: torch.Tensor) -> bool:
    return t.device.type == "cuda"


def _dev(t, name: str, dtypes=None, shape=None, device=None) -> torch.Tensor:
    """``t`` checked before its pointer crosses the ABI: a contiguous CUDA tensor
    (the library takes device pointers), of one of ``dtypes``, of ``shape``
    where given (-1 leaves a dimension free) and on ``device`` where given.
    Raises TypeError / ValueError; nothing is launched."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and (t.dim() != len(shape) or
                              any(want != -1 and want != got for want, got in zip(shape, t.shape))):
        want = tuple("*" if x == -1 else x for x in shape)
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {want}")
    if not _is_device_tensor(t):
        raise ValueError(f"{name}: must be a CUDA tensor (the library takes device pointers), got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, the other arguments are on {device}")
    return t


def _status(status, device) -> Optional[torch.Tensor]:
    if status is None:
        return None
    _dev(status, "status", I32, device=device)
    if status.numel() < 1:
        raise ValueError("status: needs one int32 element")
    return status


def _check_write(k, v, slot_mapping, key_cache, value_cache, status, cache_dtypes):
    _dev(key_cache, "key_cache", cache_dtypes, shape=(-1, -1, -1, -1))
    dev = key_cache.device
    nb, bs, hkv, d = (int(x) for x in key_cache.shape)
    _dev(value_cache, "value_cache", cache_dtypes, shape=(nb, bs, hkv, d), device=dev)
    _dev(k, "k", BF16, shape=(-1, hkv, d), device=dev)
    T = int(k.shape[0])
    _dev(v, "v", BF16, shape=(T, hkv, d), device=dev)
    _dev(slot_mapping, "slot_mapping", I64, shape=(T,), device=dev)
    _status(status, dev)
    return T, nb, bs, hkv, d


def _check_attn(q, key_cache, value_cache, block_table, rows, out, lse, workspace, status, cache_dtypes):
    _dev(q, "q", BF16, shape=(-1, -1, -1))
    dev = q.device
    T, hq, d = (int(x) for x in q.shape)
    _dev(key_cache, "key_cache", cache_dtypes, shape=(-1, -1, -1, d), device=dev)
    nb, bs, hkv, _ = (int(x) for x in key_cache.shape)
    _dev(value_cache, "value_cache", cache_dtypes, shape=(nb, bs, hkv, d), device=dev)
    _dev(block_table, "block_table", I32, shape=(-1, -1), device=dev)
    _dev(rows, "rows", I32, shape=(-1, len(ROW_FIELDS)), device=dev)
    if out is not None:
        _dev(out, "out", BF16, shape=(T, hq, d), device=dev)
    if lse is not None:
        _dev(lse, "lse", F32, shape=(hq, T), device=dev)
    if workspace is not None:
        _dev(workspace, "workspace", device=dev)
    _status(status, dev)
    return T, hq, d, nb, bs, hkv


def pcp_build_row_plan(query_len, num_computed, block_table, block_size: int, num_shards: int,
                       split_mode: int = PCP_SPLIT_CONTIGUOUS, rows_capacity: Optional[int] = None):
    """Host row plan and slot mapping. Returns a dict of numpy arrays:
    ``rows`` int32[n, 8], ``cu_q`` int32[n+1], ``slot_mapping`` int64[T],
    ``owner_shard`` int8[T]."""
    lib = load()
    ql = np.ascontiguousarray(np.asarray(query_len, dtype=np.int32))
    nc = np.ascontiguousarray(np.asarray(num_computed, dtype=np.int32))
    bt = block_table.numpy() if isinstance(block_table, torch.Tensor) else block_table
    bt = np.ascontiguousarray(np.asarray(bt, dtype=np.int32))
    R = int(ql.shape[0])
    mb = int(bt.shape[1]) if bt.ndim == 2 else 0
    T = int(ql.sum())
    cap = rows_capacity if rows_capacity is not None else max(1, 2 * num_shards * R)
    rows = np.zeros((max(cap, 1), 8), dtype=np.int32)
    cu = np.zeros(max(cap, 1) + 1, dtype=np.int32)
    slot = np.zeros(max(T, 1), dtype=np.int64)
    owner = np.zeros(max(T, 1), dtype=np.int8)
    n = np.zeros(1, dtype=np.int32)
    rc = lib.pcp_build_row_plan(R, _np_ptr(ql), _np_ptr(nc), _np_ptr(bt), mb, block_size, num_shards,
                                split_mode, _np_ptr(rows), cap, _np_ptr(n), _np_ptr(cu), _np_ptr(slot),
                                _np_ptr(owner))
    _check(rc, "pcp_build_row_plan")
    k = int(n[0])
    return dict(rows=rows[:k], cu_q=cu[:k + 1], slot_mapping=slot[:T], owner_shard=owner[:T])


def pcp_mask_slots_for_shard(slot_mapping: np.ndarray, owner_shard: np.ndarray, shard: int) -> np.ndarray:
    """PAD-masked slot mapping of one shard (host arrays)."""
    lib = load()
    s = np.ascontiguousarray(slot_mapping, dtype=np.int64)
    o = np.ascontiguousarray(owner_shard, dtype=np.int8)
    out = np.empty_like(s)
    _check(lib.pcp_mask_slots_for_shard(_np_ptr(s), _np_ptr(o), int(s.shape[0]), shard, _np_ptr(out)),
           "pcp_mask_slots_for_shard")
    return out


def pcp_decode_sms(rows: np.ndarray, num_q_heads: int, num_kv_heads: int, head_dim: int,
                   kv_cache_fp8: bool, num_sms: int) -> int:
    """SMs for the decode rows of a host row plan (int32 ``[n, 8]``) beside its
    prefill rows, or 0 to run them in sequence (host function, no GPU)."""
    lib = load()
    r = np.ascontiguousarray(rows, dtype=np.int32)
    if r.ndim != 2 or (r.shape[0] and r.shape[1] != 8):
        raise ValueError(f"rows: shape {r.shape}, expected [n, 8]")
    return int(lib.pcp_decode_sms(_np_ptr(r), int(r.shape[0]), int(num_q_heads), int(num_kv_heads),
                                  int(head_dim), 1 if kv_cache_fp8 else 0, int(num_sms)))


def pcp_kv_cache_write(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                       key_cache: torch.Tensor, value_cache: torch.Tensor,
                       status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Scatter new K/V ``[T, Hkv, D]`` into the paged caches ``[num_blocks, bs, Hkv, D]``."""
    lib = load()
    T, nb, bs, hkv, d = _check_write(k, v, slot_mapping, key_cache, value_cache, status, BF16)
    rc = lib.pcp_kv_cache_write(_t_ptr(k), _t_ptr(v), _t_ptr(slot_mapping), T, _t_ptr(key_cache),
                                _t_ptr(value_cache), nb, bs, hkv, d, _t_ptr(status), _stream(stream))
    _check(rc, "pcp_kv_cache_write")


def pcp_kv_cache_write_fp8(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                           key_cache: torch.Tensor, value_cache: torch.Tensor, k_scale: float, v_scale: float,
                           status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Scatter new bf16 K/V ``[T, Hkv, D]`` into FP8 (e4m3) caches ``[num_blocks, bs,
    Hkv, D]`` (uint8) as e4m3(x / k_scale) and e4m3(x / v_scale)."""
    lib = load()
    T, nb, bs, hkv, d = _check_write(k, v, slot_mapping, key_cache, value_cache, status, FP8_CACHE)
    rc = lib.pcp_kv_cache_write_fp8(_t_ptr(k), _t_ptr(v), _t_ptr(slot_mapping), T, _t_ptr(key_cache),
                                    _t_ptr(value_cache), nb, bs, hkv, d, float(k_scale), float(v_scale),
                                    _t_ptr(status), _stream(stream))
    _check(rc, "pcp_kv_cache_write_fp8")


def pcp_attn_workspace_size(num_rows: int, total_q: int, num_q_heads: int, head_dim: int,
                            max_kv_len: int, flags: int = 0) -> int:
    return int(load().pcp_attn_workspace_size(num_rows, total_q, num_q_heads, head_dim, max_kv_len, flags))


def pcp_attn_varlen(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                    block_table: torch.Tensor, rows: torch.Tensor, scale: float,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, flags: int = 0,
                    status: Optional[torch.Tensor] = None, stream=None):
    """Attention of every planned row. ``q`` ``[T, Hq, D]`` bf16; ``rows`` int32
    ``[n, 8]`` on the device; returns ``(out [T, Hq, D] bf16, lse [Hq, T] fp32)``.
    Pass ``out``/``lse``/``workspace`` to avoid allocating per call."""
    lib = load()
    T, hq, d, nb, bs, hkv = _check_attn(q, key_cache, value_cache, block_table, rows, out, lse, workspace, status,
                                        BF16)
    n_rows = int(rows.shape[0])
    mb = int(block_table.shape[1])
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    need = pcp_attn_workspace_size(n_rows, T, hq, d, mb * bs, flags)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = lib.pcp_attn_varlen(_t_ptr(q), _t_ptr(key_cache), _t_ptr(value_cache), _t_ptr(block_table),
                             int(block_table.shape[0]), mb, nb,
                             bs, _t_ptr(rows), n_rows, T, hq, hkv, d, float(scale), _t_ptr(out), _t_ptr(lse),
                             _t_ptr(workspace), int(workspace.numel() * workspace.element_size()), flags,
                             _t_ptr(status), _stream(stream))
    _check(rc, "pcp_attn_varlen")
    return out, lse


def pcp_attn_varlen_fp8kv(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                          k_descale: torch.Tensor, v_descale: torch.Tensor, block_table: torch.Tensor,
                          rows: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          flags: int = 0, status: Optional[torch.Tensor] = None, stream=None):
    """:func:`pcp_attn_varlen` over FP8 (e4m3, uint8) caches with fp32 descales
    ``[num_reqs, Hkv]`` on the device."""
    lib = load()
    T, hq, d, nb, bs, hkv = _check_attn(q, key_cache, value_cache, block_table, rows, out, lse, workspace, status,
                                        FP8_CACHE)
    R = int(block_table.shape[0])
    _dev(k_descale, "k_descale", F32, shape=(R, hkv), device=q.device)
    _dev(v_descale, "v_descale", F32, shape=(R, hkv), device=q.device)
    n_rows = int(rows.shape[0])
    mb = int(block_table.shape[1])
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    need = pcp_attn_workspace_size(n_rows, T, hq, d, mb * bs, flags)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = lib.pcp_attn_varlen_fp8kv(_t_ptr(q), _t_ptr(key_cache), _t_ptr(value_cache), _t_ptr(k_descale),
                                   _t_ptr(v_descale), _t_ptr(block_table), int(block_table.shape[0]), mb, nb, bs,
                                   _t_ptr(rows), n_rows, T, hq, hkv, d, float(scale), _t_ptr(out), _t_ptr(lse),
                                   _t_ptr(workspace), int(workspace.numel() * workspace.element_size()), flags,
                                   _t_ptr(status), _stream(stream))
    _check(rc, "pcp_attn_varlen_fp8kv")
    return out, lse


def pcp_attn_varlen_noalloc(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                            block_table: torch.Tensor, rows: torch.Tensor, scale: float, out: torch.Tensor,
                            lse: torch.Tensor, flags: int = 0, status: Optional[torch.Tensor] = None,
                            stream=None):
    """:func:`pcp_attn_varlen` for callers that cannot allocate device memory:
    the caller passes ``out`` and ``lse``, and the library's own fixed 64 MiB
    scratch array (reserved on each GPU that loads the library) replaces the
    workspace. Calls on one device share that array: keep them on one stream."""
    lib = load()
    if out is None or lse is None:
        raise ValueError("pcp_attn_varlen_noalloc: out and lse are required")
    T, hq, d, nb, bs, hkv = _check_attn(q, key_cache, value_cache, block_table, rows, out, lse, None, status,
                                        BF16)
    rc = lib.pcp_attn_varlen_noalloc(_t_ptr(q), _t_ptr(key_cache), _t_ptr(value_cache), _t_ptr(block_table),
                                     int(block_table.shape[0]), int(block_table.shape[1]), nb, bs, _t_ptr(rows),
                                     int(rows.shape[0]), T, hq, hkv, d, float(scale), _t_ptr(out), _t_ptr(lse),
                                     flags, _t_ptr(status), _stream(stream))
    _check(rc, "pcp_attn_varlen_noalloc")
    return out, lse


def pcp_attn_window_workspace_size(num_rows: int, total_q: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                   max_kv_len: int, block_size: int, window: int, num_sinks: int = 0) -> int:
    return int(load().pcp_attn_window_workspace_size(num_rows, total_q, num_q_heads, num_kv_heads, head_dim,
                                                     max_kv_len, block_size, window, num_sinks))


def pcp_attn_shared_prefix_workspace_size(num_rows: int, num_prefixes: int, total_q: int, num_q_heads: int,
                                          num_kv_heads: int, head_dim: int, max_kv_len: int) -> int:
    return int(load().pcp_attn_shared_prefix_workspace_size(num_rows, num_prefixes, total_q, num_q_heads,
                                                            num_kv_heads, head_dim, max_kv_len))


def _i32_arg(x, name: str) -> int:
    v = int(x)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name}: {v} does not fit in 32 bits")
    return v


def _ready(device: int, *pairs) -> bool:
    """Whether every ``(tensor, dtype)`` is a contiguous CUDA tensor of that type on
    that device (the quick form of :func:`_dev`, which says what is wrong)."""
    kind = torch.Tensor
    for t, dtype in pairs:
        if type(t) is not kind or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
            return False
    return True


def _launch(f, device: int, stream, *args) -> int:
    """``f(*args, stream)`` with the tensors' device current; without a stream, on that
    device's current one."""
    if device < 0:  # not a CUDA device: the library is a stand-in
        return f(*args, _stream(stream))
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(device)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == device:
        return f(*args, s)
    with torch.cuda.device(device):
        return f(*args, s)


def _range_args(q, key_cache, value_cache, descales, block_table, rows, out, lse, workspace, status, cache_dtypes):
    """The checks of :func:`_check_attn` and the descales', quick where every buffer is
    passed. Returns (T, hq, d, nb, bs, hkv, R, mb, n_rows, device index)."""
    dev = q.get_device() if isinstance(q, torch.Tensor) else -1
    if dev >= 0 and out is not None and lse is not None and workspace is not None:
        cache = key_cache.dtype if isinstance(key_cache, torch.Tensor) else None
        pairs = ((q, torch.bfloat16), (key_cache, cache), (value_cache, cache), (block_table, torch.int32),
                 (rows, torch.int32), (out, torch.bfloat16), (lse, torch.float32), (workspace, torch.uint8))
        if cache in cache_dtypes and _ready(dev, *pairs) and (status is None or _ready(dev, (status, torch.int32))) \
                and (not descales or _ready(dev, (descales[0], torch.float32), (descales[1], torch.float32))):
            qs, ks, bts, rs = q.shape, key_cache.shape, block_table.shape, rows.shape
            if len(qs) == 3 and len(ks) == 4 and len(bts) == 2 and len(rs) == 2 and rs[1] == len(ROW_FIELDS):
                T, hq, d = qs
                nb, bs, hkv, kd = ks
                R, mb = bts
                if kd == d and value_cache.shape == ks and out.shape == qs and lse.shape == (hq, T) \
                        and (status is None or status.numel() > 0) \
                        and (not descales or descales[0].shape == descales[1].shape == (R, hkv)):
                    return T, hq, d, nb, bs, hkv, R, mb, rs[0], dev
    T, hq, d, nb, bs, hkv = _check_attn(q, key_cache, value_cache, block_table, rows, out, lse, workspace, status,
                                        cache_dtypes)
    R, mb = (int(x) for x in block_table.shape)
    for t, name in zip(descales, ("k_descale", "v_descale")):
        _dev(t, name, F32, shape=(R, hkv), device=q.device)
    return T, hq, d, nb, bs, hkv, R, mb, int(rows.shape[0]), dev


def _range_buffers(q, hq: int, T: int, out, lse, workspace, need):
    """out, lse and workspace as given, or new ones (``need()``: workspace bytes)."""
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(need(), 256), dtype=torch.uint8, device=q.device)
    return out, lse, workspace


def _attn_window(what, q, key_cache, value_cache, descales, block_table, rows, scale, window, num_sinks, out, lse,
                 workspace, status, stream, cache_dtypes):
    lib = load()
    T, hq, d, nb, bs, hkv, R, mb, n_rows, dev = _range_args(q, key_cache, value_cache, descales, block_table, rows,
                                                            out, lse, workspace, status, cache_dtypes)
    window, num_sinks = _i32_arg(window, "window"), _i32_arg(num_sinks, "num_sinks")
    out, lse, workspace = _range_buffers(
        q, hq, T, out, lse, workspace,
        lambda: pcp_attn_window_workspace_size(n_rows, T, hq, hkv, d, mb * bs, bs, window, num_sinks))
    rc = _launch(getattr(lib, what), dev, stream, q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                 *[x.data_ptr() for x in descales], block_table.data_ptr(), R, mb, nb, bs, rows.data_ptr(), n_rows, T,
                 hq, hkv, d, scale, window, num_sinks, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                 workspace.numel() * workspace.element_size(), None if status is None else status.data_ptr())
    if rc:
        raise PcpError(rc, what)
    return out, lse


def pcp_attn_window(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor, block_table: torch.Tensor,
                    rows: torch.Tensor, scale: float, window: int, num_sinks: int = 0,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """:func:`pcp_attn_varlen` where a query sees the last ``window`` keys up to its
    own and the first ``num_sinks`` keys of its request."""
    return _attn_window("pcp_attn_window", q, key_cache, value_cache, (), block_table, rows, scale, window, num_sinks,
                        out, lse, workspace, status, stream, BF16)


def pcp_attn_window_fp8kv(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                          k_descale: torch.Tensor, v_descale: torch.Tensor, block_table: torch.Tensor,
                          rows: torch.Tensor, scale: float, window: int, num_sinks: int = 0,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                          stream=None):
    """:func:`pcp_attn_window` over FP8 (e4m3, uint8) caches with fp32 descales
    ``[num_reqs, Hkv]`` on the device."""
    return _attn_window("pcp_attn_window_fp8kv", q, key_cache, value_cache, (k_descale, v_descale), block_table, rows,
                        scale, window, num_sinks, out, lse, workspace, status, stream, FP8_CACHE)


def pcp_build_prefix_groups(rows: np.ndarray, block_table, block_size: int, min_prefix_len: int = 1024) -> np.ndarray:
    """Prefix groups int32 ``[n, 4]`` (``PREFIX_FIELDS``) of a host row plan: runs of
    rows whose block tables begin with the same pages (host function, no GPU)."""
    lib = load()
    r = np.ascontiguousarray(rows, dtype=np.int32)
    if r.ndim != 2 or (r.shape[0] and r.shape[1] != len(ROW_FIELDS)):
        raise ValueError(f"rows: shape {r.shape}, expected [n, {len(ROW_FIELDS)}]")
    bt = block_table.numpy() if isinstance(block_table, torch.Tensor) else block_table
    bt = np.ascontiguousarray(np.asarray(bt, dtype=np.int32))
    if bt.ndim != 2:
        raise ValueError(f"block_table: shape {bt.shape}, expected [num_reqs, max_blocks]")
    cap = max(1, r.shape[0] // 2)
    out = np.zeros((cap, len(PREFIX_FIELDS)), dtype=np.int32)
    n = np.zeros(1, dtype=np.int32)
    rc = lib.pcp_build_prefix_groups(_np_ptr(r), int(r.shape[0]), _np_ptr(bt), int(bt.shape[0]), int(bt.shape[1]),
                                     _i32_arg(block_size, "block_size"), _i32_arg(min_prefix_len, "min_prefix_len"),
                                     _np_ptr(out), cap, _np_ptr(n))
    _check(rc, "pcp_build_prefix_groups")
    return out[:int(n[0])]


def _attn_shared(what, q, key_cache, value_cache, descales, block_table, rows, prefixes, scale, out, lse, workspace,
                 status, stream, cache_dtypes):
    lib = load()
    T, hq, d, nb, bs, hkv, R, mb, n_rows, dev = _range_args(q, key_cache, value_cache, descales, block_table, rows,
                                                            out, lse, workspace, status, cache_dtypes)
    _dev(prefixes, "prefixes", I32, shape=(-1, len(PREFIX_FIELDS)), device=q.device)
    ng = prefixes.shape[0]
    out, lse, workspace = _range_buffers(
        q, hq, T, out, lse, workspace,
        lambda: pcp_attn_shared_prefix_workspace_size(n_rows, ng, T, hq, hkv, d, mb * bs))
    rc = _launch(getattr(lib, what), dev, stream, q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                 *[x.data_ptr() for x in descales], block_table.data_ptr(), R, mb, nb, bs, rows.data_ptr(), n_rows,
                 prefixes.data_ptr(), ng, T, hq, hkv, d, scale, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                 workspace.numel() * workspace.element_size(), None if status is None else status.data_ptr())
    if rc:
        raise PcpError(rc, what)
    return out, lse


def pcp_attn_shared_prefix(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                           block_table: torch.Tensor, rows: torch.Tensor, prefixes: torch.Tensor, scale: float,
                           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                           stream=None):
    """:func:`pcp_attn_varlen` of a batch whose token groups share prefixes, each
    prefix attended once for its group. ``prefixes`` int32 ``[n, 4]`` on the device
    (:func:`pcp_build_prefix_groups`)."""
    return _attn_shared("pcp_attn_shared_prefix", q, key_cache, value_cache, (), block_table, rows, prefixes, scale,
                        out, lse, workspace, status, stream, BF16)


def pcp_attn_shared_prefix_fp8kv(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                                 k_descale: torch.Tensor, v_descale: torch.Tensor, block_table: torch.Tensor,
                                 rows: torch.Tensor, prefixes: torch.Tensor, scale: float,
                                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                                 stream=None):
    """:func:`pcp_attn_shared_prefix` over FP8 (e4m3, uint8) caches with fp32 descales
    ``[num_reqs, Hkv]`` on the device (a prefix takes those of its request)."""
    return _attn_shared("pcp_attn_shared_prefix_fp8kv", q, key_cache, value_cache, (k_descale, v_descale), block_table,
                        rows, prefixes, scale, out, lse, workspace, status, stream, FP8_CACHE)


def pcp_kv_pages_workspace_size(num_blocks: int) -> int:
    return int(load().pcp_kv_pages_workspace_size(num_blocks))


def _ints_ready(device: int, *pairs) -> bool:
    """Whether every ``(tensor, shape)`` is a contiguous int32 CUDA tensor of that shape on
    that device (the quick form of :func:`_i32_in`)."""
    if device < 0:
        return False
    i32, kind = torch.int32, torch.Tensor
    for t, shape in pairs:
        if type(t) is not kind or t.dtype is not i32 or t.get_device() != device or t.shape != shape \
                or not t.is_contiguous():
            return False
    return True


def _i32_in(t, name: str, shape, like) -> None:
    """``t`` checked as an int32 input of ``shape`` on the device of ``like``."""
    if not _ints_ready(like.get_device(), (t, shape)):
        _dev(t, name, I32, shape=shape, device=like.device)


def _i32_out(t, name: str, shape, like):
    """``t`` checked as an int32 output of ``shape`` on the device of ``like``, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=torch.int32, device=like.device)
    _i32_in(t, name, shape, like)
    return t


def _status_in(status, like) -> None:
    if status is not None and not _ints_ready(like.get_device(), (status, (1,))):
        _status(status, like.device)


def _check_pages(key_cache, value_cache, block_table, ref_count, status):
    dtype = key_cache.dtype if isinstance(key_cache, torch.Tensor) else None
    dev = key_cache.get_device() if dtype is not None else -1
    if dev < 0 or dtype not in PAGE_CACHE or \
            not _ready(dev, (key_cache, dtype), (value_cache, dtype), (block_table, torch.int32),
                       (ref_count, torch.int32)) or \
            key_cache.dim() != 4 or value_cache.shape != key_cache.shape or block_table.dim() != 2 or \
            ref_count.shape != key_cache.shape[:1]:
        _dev(key_cache, "key_cache", PAGE_CACHE, shape=(-1, -1, -1, -1))
        device = key_cache.device
        _dev(value_cache, "value_cache", (dtype,), shape=tuple(key_cache.shape), device=device)
        _dev(block_table, "block_table", I32, shape=(-1, -1), device=device)
        _dev(ref_count, "ref_count", I32, shape=(int(key_cache.shape[0]),), device=device)
    _status_in(status, key_cache)
    nb, bs, hkv, d = key_cache.shape
    return dev, nb, bs, hkv * d * key_cache.element_size()


def _pages_workspace(workspace, nb: int, like):
    if workspace is None:
        return torch.empty(max(pcp_kv_pages_workspace_size(nb), 256), dtype=torch.uint8, device=like.device)
    if not _ready(like.get_device(), (workspace, torch.uint8)):
        _dev(workspace, "workspace", device=like.device)
    return workspace


def pcp_kv_fork(key_cache: torch.Tensor, value_cache: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor,
                parent: torch.Tensor, ref_count: torch.Tensor, block_table_out: Optional[torch.Tensor] = None,
                ref_count_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, stream=None):
    """Children of requests: child ``i`` shares the full pages of request
    ``parent[i]`` and gets a new page with a copy of the partly filled last one.
    ``kv_len`` int32 ``[num_reqs]``, ``parent`` int32 ``[num_children]`` (-1: empty
    child), ``ref_count`` int32 ``[num_blocks]``. Returns ``(block_table_out
    [num_children, max_blocks], ref_count_out)``."""
    lib = load()
    dev, nb, bs, slot_bytes = _check_pages(key_cache, value_cache, block_table, ref_count, status)
    R, mb = block_table.shape
    N = parent.numel() if isinstance(parent, torch.Tensor) else 0
    if not _ints_ready(dev, (kv_len, (R,)), (parent, (N,)), (block_table_out, (N, mb)), (ref_count_out, (nb,))):
        _i32_in(kv_len, "kv_len", (R,), block_table)
        _i32_in(parent, "parent", (N,), block_table)
        block_table_out = _i32_out(block_table_out, "block_table_out", (N, mb), block_table)
        ref_count_out = _i32_out(ref_count_out, "ref_count_out", (nb,), block_table)
    workspace = _pages_workspace(workspace, nb, block_table)
    rc = _launch(lib.pcp_kv_fork, dev, stream, key_cache.data_ptr(), value_cache.data_ptr(), nb, bs, slot_bytes,
                 block_table.data_ptr(), R, mb, kv_len.data_ptr(), parent.data_ptr(), N, ref_count.data_ptr(),
                 block_table_out.data_ptr(), ref_count_out.data_ptr(), workspace.data_ptr(),
                 workspace.numel() * workspace.element_size(), None if status is None else status.data_ptr())
    if rc:
        raise PcpError(rc, "pcp_kv_fork")
    return block_table_out, ref_count_out


def pcp_kv_release(block_table: torch.Tensor, first_page: torch.Tensor, last_page: torch.Tensor,
                   ref_count: torch.Tensor, block_table_out: Optional[torch.Tensor] = None,
                   ref_count_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Give back one reference of every block-table entry ``[first_page[r],
    last_page[r])`` of each row (int32 ``[num_reqs]``); the entries become -1.
    Returns ``(block_table_out, ref_count_out)``; pass the inputs themselves to
    work in place."""
    lib = load()
    dev = block_table.get_device() if isinstance(block_table, torch.Tensor) else -1
    if dev < 0 or block_table.dim() != 2 or not _ready(dev, (block_table, torch.int32)):
        _dev(block_table, "block_table", I32, shape=(-1, -1))
    R, mb = block_table.shape
    nb = ref_count.numel() if isinstance(ref_count, torch.Tensor) else 0
    if not _ints_ready(dev, (first_page, (R,)), (last_page, (R,)), (ref_count, (nb,)), (block_table_out, (R, mb)),
                       (ref_count_out, (nb,))):
        _i32_in(first_page, "first_page", (R,), block_table)
        _i32_in(last_page, "last_page", (R,), block_table)
        _i32_in(ref_count, "ref_count", (nb,), block_table)
        block_table_out = _i32_out(block_table_out, "block_table_out", (R, mb), block_table)
        ref_count_out = _i32_out(ref_count_out, "ref_count_out", (nb,), block_table)
    _status_in(status, block_table)
    rc = _launch(lib.pcp_kv_release, dev, stream, block_table.data_ptr(), R, mb,
                 first_page.data_ptr(), last_page.data_ptr(), ref_count.data_ptr(), nb, block_table_out.data_ptr(),
                 ref_count_out.data_ptr(), None if status is None else status.data_ptr())
    if rc:
        raise PcpError(rc, "pcp_kv_release")
    return block_table_out, ref_count_out


def pcp_kv_compact(key_cache: torch.Tensor, value_cache: torch.Tensor, block_table: torch.Tensor,
                   ref_count: torch.Tensor, block_table_out: Optional[torch.Tensor] = None,
                   ref_count_out: Optional[torch.Tensor] = None, num_live: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Move the ``n`` live pages to ids ``[0, n)``, in the caches, the counts and the
    table. Returns ``(block_table_out, ref_count_out, num_live)``, ``num_live``
    int32 ``[1]`` on the device."""
    lib = load()
    dev, nb, bs, slot_bytes = _check_pages(key_cache, value_cache, block_table, ref_count, status)
    R, mb = block_table.shape
    if not _ints_ready(dev, (block_table_out, (R, mb)), (ref_count_out, (nb,)), (num_live, (1,))):
        block_table_out = _i32_out(block_table_out, "block_table_out", (R, mb), block_table)
        ref_count_out = _i32_out(ref_count_out, "ref_count_out", (nb,), block_table)
        num_live = _i32_out(num_live, "num_live", (1,), block_table)
    workspace = _pages_workspace(workspace, nb, block_table)
    rc = _launch(lib.pcp_kv_compact, dev, stream, key_cache.data_ptr(), value_cache.data_ptr(), nb, bs, slot_bytes,
                 block_table.data_ptr(), R, mb, ref_count.data_ptr(), block_table_out.data_ptr(),
                 ref_count_out.data_ptr(), num_live.data_ptr(), workspace.data_ptr(),
                 workspace.numel() * workspace.element_size(), None if status is None else status.data_ptr())
    if rc:
        raise PcpError(rc, "pcp_kv_compact")
    return block_table_out, ref_count_out, num_live


def pcp_lse_merge(out_a: torch.Tensor, lse_a: torch.Tensor, out_b: torch.Tensor, lse_b: torch.Tensor,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None):
    """LSE merge of two fp32 partials ``[T, Hq, D]`` / ``[Hq, T]`` into bf16 out and fp32 lse."""
    lib = load()
    _dev(out_a, "out_a", F32, shape=(-1, -1, -1))
    dev = out_a.device
    T, hq, d = (int(x) for x in out_a.shape)
    _dev(out_b, "out_b", F32, shape=(T, hq, d), device=dev)
    _dev(lse_a, "lse_a", F32, shape=(hq, T), device=dev)
    _dev(lse_b, "lse_b", F32, shape=(hq, T), device=dev)
    if out is None:
        out = torch.empty(out_a.shape, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty_like(lse_a)
    _dev(out, "out", BF16, shape=(T, hq, d), device=dev)
    _dev(lse, "lse", F32, shape=(hq, T), device=dev)
    rc = lib.pcp_lse_merge(_t_ptr(out_a), _t_ptr(lse_a), _t_ptr(out_b), _t_ptr(lse_b), _t_ptr(out), _t_ptr(lse),
                           T, hq, d, _stream(stream))
    _check(rc, "pcp_lse_merge")
    return out, lse


def pcp_set_profile_events(prefill_begin=None, prefill_end=None, decode_begin=None, decode_end=None) -> None:
    """Register ``torch.cuda.Event`` objects (already recorded once, so that they
    exist) to be recorded around the prefill and decode kernels of later
    :func:`pcp_attn_varlen` calls in this thread; no arguments unregisters."""
    def h(e):
        return None if e is None else ctypes.c_void_p(int(e.cuda_event))
    load().pcp_set_profile_events(h(prefill_begin), h(prefill_end), h(decode_begin), h(decode_end))
