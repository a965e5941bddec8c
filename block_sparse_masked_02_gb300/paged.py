"""ctypes binding of libfdma's paged key/value cache (include/fdma_paged.h).

`kv_append` writes new tokens' K and V rows into the pages of a cache, `kv_gather` reads sequences
back and `fwd` is the attention of every sequence's newest tokens (one, a few, or a chunk of a
prompt) over its pages.  Like `fdma`, it marshals pointers and strides only: every step runs in the
CUDA kernels of libfdma.so, and there is no CPU path.

One set of plan tensors serves the three of them, all int32 on the cache's device:

  page_table (B, max_pages)  page of each page_size positions of a sequence; entries behind the last
                             page that k_lens needs are not read
  k_lens (B,)                keys of each sequence, its new tokens among them
  cu_q (B + 1,)              where each sequence's new tokens begin in the packed token axis

so new token i of the n of sequence b is at position k_lens[b] - n + i.  Their contents stay on the
device: a captured CUDA graph follows them when they change in place.  Page numbers, lengths or
offsets out of range are left out by the kernels and reported by `fdma.device_error()`.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import fdma as _fdma
from . import inputs as _inputs

FDMA_CACHE_BF16 = 0
FDMA_CACHE_E4M3 = 1

EXPORTED = ("fdma_kv_append", "fdma_kv_gather", "fdma_paged_workspace_size", "fdma_paged_fwd")

_I64x2 = ctypes.c_int64 * 2
_I64x3 = ctypes.c_int64 * 3


class FdmaKvCache(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("cache_type", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("k_stride", _I64x3),
        ("v", ctypes.c_void_p), ("v_stride", _I64x3),
        ("k_exp", ctypes.c_void_p), ("k_exp_stride", _I64x3),
        ("v_exp", ctypes.c_void_p), ("v_exp_stride", _I64x3),
        ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("k_len", ctypes.c_void_p),
    ]


class FdmaPagedArgs(ctypes.Structure):
    _fields_ = [
        ("cache", FdmaKvCache), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("q_stride", _I64x2), ("cu_q", ctypes.c_void_p), ("max_q", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("scale", ctypes.c_float),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


# The same two structs as packed bytes (native alignment): filling them is a good part of a small
# call's time, and one struct.pack takes a quarter of what the ctypes fields take.
_CACHE_FMT = "7iP3qP3qP3qP3qPqP"
_PACK_CACHE = struct.Struct(_CACHE_FMT).pack
_PACK_ARGS = struct.Struct(_CACHE_FMT + "2iP2qP4ifPN").pack
_PACK_WORKSPACE = struct.Struct("PN").pack  # the last two fields

_LIB = None


def load() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        lib = _fdma.load()
        # (structs go as the address of their packed bytes)
        S, P, I = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_int
        lib.fdma_kv_append.argtypes = [S, P, S, P, S, P, I, P]
        lib.fdma_kv_append.restype = I
        lib.fdma_kv_gather.argtypes = [S, P, P, I, P, P, P]
        lib.fdma_kv_gather.restype = I
        lib.fdma_paged_workspace_size.argtypes = [S]
        lib.fdma_paged_workspace_size.restype = ctypes.c_size_t
        lib.fdma_paged_fwd.argtypes = [S, P, P, P]
        lib.fdma_paged_fwd.restype = I
        _LIB = lib
    return _LIB


def _check_device(first, *ts):
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("libfdma takes CUDA tensors only (no CPU path)")
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError("all tensors of a call are on one device")
    return dev


def _check_int(name, t, n):
    if t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be int32 ({n},) and contiguous")


def _on(dev, stream):
    """(guard that makes the device and the launch stream current, or None; stream pointer): what is
    allocated for the call then belongs to the stream that it runs on."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError("the stream belongs to another device than the tensors")
        return torch.cuda.stream(stream), stream.cuda_stream
    guard = None if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
    return guard, torch._C._cuda_getCurrentRawStream(dev.index)


def _check_workspace(ws):
    if ws is not None and not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _cache(k_cache, v_cache, page_table, k_lens, k_exp, v_exp):
    """The fields of fdma_kv_cache, in order."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be (num_pages, page_size, Hkv, d)")
    n, ps, h, d = shape
    dt = k_cache.dtype
    sk, sv = k_cache.stride(), v_cache.stride()
    if d > 1 and (sk[3] != 1 or sv[3] != 1):
        raise ValueError("k_cache and v_cache need a contiguous head dim")
    if page_table.dtype is not torch.int32 or page_table.dim() != 2:
        raise ValueError("page_table must be int32 (B, max_pages)")
    B, mp = page_table.shape
    ts, tc = page_table.stride()
    if mp > 1 and tc != 1:
        raise ValueError("page_table must have a contiguous last dimension")
    _check_int("k_lens", k_lens, B)
    rows = (n, ps, mp, k_cache.data_ptr(), sk[0], sk[1], sk[2], v_cache.data_ptr(), sv[0], sv[1], sv[2])
    if dt is torch.bfloat16 and v_cache.dtype is dt:
        if k_exp is not None or v_exp is not None:
            raise ValueError("k_exp and v_exp belong to float8_e4m3fn caches")
        return (B, h, d, FDMA_CACHE_BF16, *rows, 0, 0, 0, 0, 0, 0, 0, 0, page_table.data_ptr(), ts, k_lens.data_ptr())
    if dt is torch.float8_e4m3fn and v_cache.dtype is dt:
        for name, t in (("k_exp", k_exp), ("v_exp", v_exp)):
            if t is None or t.dtype is not torch.uint8 or t.shape != shape[:3]:
                raise ValueError(f"{name} must be uint8 (num_pages, page_size, Hkv) for a float8_e4m3fn cache")
        return (B, h, d, FDMA_CACHE_E4M3, *rows, k_exp.data_ptr(), *k_exp.stride(), v_exp.data_ptr(), *v_exp.stride(),
                page_table.data_ptr(), ts, k_lens.data_ptr())
    raise ValueError("k_cache and v_cache must both be bfloat16 or both float8_e4m3fn")


def empty_cache(num_pages, page_size, Hkv, d, *, dtype=torch.bfloat16, device="cuda"):
    """An uninitialised cache: (k_cache, v_cache, k_exp, v_exp), the caches (num_pages, page_size, Hkv, d)
    and, for dtype float8_e4m3fn, the scale bytes (num_pages, page_size, Hkv) (else None).  A page's rows
    of one head lie together in memory: attention reads whole pages of one head."""
    def one(dt, *tail):
        x = torch.empty((num_pages, Hkv, page_size) + tail, dtype=dt, device=device)
        return x.transpose(1, 2)
    if dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError("dtype must be torch.bfloat16 or torch.float8_e4m3fn")
    exp = (one(torch.uint8), one(torch.uint8)) if dtype == torch.float8_e4m3fn else (None, None)
    return (one(dtype, d), one(dtype, d)) + exp


_PACK_2Q = struct.Struct("2q").pack


def kv_append(k, v, k_cache, v_cache, page_table, k_lens, cu_q, *, k_exp=None, v_exp=None, stream=None):
    """Write the new tokens' rows k, v (T, Hkv, d) bf16 (contiguous head dim) into the cache, quantised
    (with their scale bytes into k_exp, v_exp) where it is float8_e4m3fn.  Rows behind cu_q[B] are ignored.
    The slots of one call must be distinct, and none may hold a row of k or v itself."""
    dev = _check_device(k, v, k_cache, v_cache, page_table, k_lens, cu_q, k_exp, v_exp)
    c = _cache(k_cache, v_cache, page_table, k_lens, k_exp, v_exp)
    B, Hkv, d = c[:3]
    _check_int("cu_q", cu_q, B + 1)
    sk, sv = k.stride(), v.stride()
    if k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16 or v.shape != k.shape or len(sk) != 3 or \
            k.shape[1] != Hkv or k.shape[2] != d or sk[2] != 1 or sv[2] != 1:
        raise ValueError("k and v must be bf16 (T, Hkv, d) with a contiguous head dim")
    guard, sp = _on(dev, stream)
    args = (_PACK_CACHE(*c), k.data_ptr(), _PACK_2Q(sk[0], sk[1]), v.data_ptr(), _PACK_2Q(sv[0], sv[1]),
            cu_q.data_ptr(), k.shape[0], sp)
    if guard is None:
        st = load().fdma_kv_append(*args)
    else:
        with guard:
            st = load().fdma_kv_append(*args)
    _fdma._raise(st, "fdma_kv_append")


def _launch_norm_rope_append(args, c, q, k, v, q_out, cu_q, sp):
    rows = _inputs._rows
    qr, kr, vr = rows("q", q), rows("k", k), rows("v", v)
    if q_out is None:
        q_out, qor = _inputs._new_rows(q)
    else:
        qor = rows("q_out", q_out, q.shape)
    st = _inputs.load().fdma_norm_rope_append(args, _PACK_CACHE(*c), qr, kr, vr, qor, cu_q.data_ptr(), sp)
    if st:
        _fdma._raise(st, "fdma_norm_rope_append")
    return q_out


def norm_rope_append(q, k, v, k_cache, v_cache, page_table, k_lens, cu_q, *, q_weight=None, k_weight=None, rope=None,
                     positions=None, interleaved=False, norm=True, eps=1e-6, k_exp=None, v_exp=None, q_out=None, stream=None):
    """`inputs.norm_rope` of the packed new tokens q (T, Hq, d) and k (T, Hkv, d), and `kv_append` of the keys with v
    (T, Hkv, d), in one launch: returns q_out (T, Hq, d), which `fwd` takes.  A token's position is its place in its
    sequence, or positions[t] (int32 (T,)) where that is something else.  A float8_e4m3fn cache takes its codes from the
    fp32 values, rounded once.  Rows behind cu_q[B] and tokens at a negative position (padding) are left as they are, in
    q_out (uninitialised where it is allocated here) and in the cache."""
    dev = _inputs._check_device(q, k, v, k_cache, v_cache, page_table, k_lens, cu_q, q_weight, k_weight, rope, positions, k_exp,
                                v_exp, q_out)
    c = _cache(k_cache, v_cache, page_table, k_lens, k_exp, v_exp)
    B, Hkv, d = c[:3]
    _check_int("cu_q", cu_q, B + 1)
    qs = q.shape
    if len(qs) != 3 or qs[2] != d or k.shape != (qs[0], Hkv, d) or v.shape != k.shape:
        raise ValueError("q, k and v must be (T, heads, d) with the kv heads and head dim of the cache")
    if positions is not None:
        _check_int("positions", positions, qs[0])
    args = _inputs._norm_rope_args(q, k, q_weight, k_weight, rope, positions, 0, interleaved, norm, eps)
    guard, sp = _inputs._on(dev, stream)
    return _inputs._run(guard, _launch_norm_rope_append, args, c, q, k, v, q_out, cu_q, sp)


def kv_gather(k_cache, v_cache, page_table, k_lens, cu_k, total, *, first=None, k_exp=None, v_exp=None, k_out=None,
              v_out=None, stream=None):
    """Read positions first[b] + i (first: int32 (B,), default 0) of every sequence into rows cu_k[b] + i of
    (k, v), each (total, Hkv, d) bf16.  Positions outside [0, k_lens[b]) read as zeros, so with cu_k = b * N
    and total = B * N the result views as the (B, N, Hkv, d) that `fdma.fwd` takes.  Rows behind cu_k[B] are
    left as they are (uninitialised where the outputs are allocated here)."""
    dev = _check_device(k_cache, v_cache, page_table, k_lens, cu_k, first, k_exp, v_exp, k_out, v_out)
    c = _cache(k_cache, v_cache, page_table, k_lens, k_exp, v_exp)
    B, Hkv, d = c[:3]
    _check_int("cu_k", cu_k, B + 1)
    if first is not None:
        _check_int("first", first, B)
    shape = (int(total), Hkv, d)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None and (t.dtype is not torch.bfloat16 or t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous bf16 {shape}")
    guard, sp = _on(dev, stream)

    def call():
        ko = torch.empty(shape, dtype=torch.bfloat16, device=dev) if k_out is None else k_out
        vo = torch.empty(shape, dtype=torch.bfloat16, device=dev) if v_out is None else v_out
        return ko, vo, load().fdma_kv_gather(_PACK_CACHE(*c), cu_k.data_ptr(), None if first is None else first.data_ptr(),
                                             shape[0], ko.data_ptr(), vo.data_ptr(), sp)

    if guard is None:
        ko, vo, st = call()
    else:
        with guard:
            ko, vo, st = call()
    _fdma._raise(st, "fdma_kv_gather")
    return ko, vo


def _fields(q, k_cache, v_cache, page_table, k_lens, cu_q, max_q, k_exp, v_exp, causal, window, sinks, scale):
    """The fields of fdma_paged_args up to the workspace, in order."""
    c = _cache(k_cache, v_cache, page_table, k_lens, k_exp, v_exp)
    _check_int("cu_q", cu_q, c[0] + 1)
    sq = q.stride()
    if q.dtype is not torch.bfloat16 or len(sq) != 3 or q.shape[2] != c[2] or sq[2] != 1:
        raise ValueError("q must be bf16 (T, Hq, d) with a contiguous head dim")
    T, Hq, d = q.shape
    return (*c, T, Hq, q.data_ptr(), sq[0], sq[1], cu_q.data_ptr(), int(max_q), 1 if causal else 0, int(window),
            int(sinks), d ** -0.5 if scale is None else float(scale))


def make_args(q, k_cache, v_cache, page_table, k_lens, cu_q, max_q, *, k_exp=None, v_exp=None, causal=True, window=0,
              sinks=0, scale=None, workspace=None) -> FdmaPagedArgs:
    """fdma_paged_args of a call (see `fwd`)."""
    f = _fields(q, k_cache, v_cache, page_table, k_lens, cu_q, max_q, k_exp, v_exp, causal, window, sinks, scale)
    _check_workspace(workspace)
    ws = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return FdmaPagedArgs.from_buffer_copy(_PACK_ARGS(*f, *ws))


def workspace_size(args: FdmaPagedArgs) -> int:
    return int(load().fdma_paged_workspace_size(bytes(args)))


def alloc_workspace(args: FdmaPagedArgs, device) -> torch.Tensor:
    # (the caching allocator's blocks are 512-byte aligned)
    return torch.empty(workspace_size(args), dtype=torch.uint8, device=device)


def _launch_fwd(f, T, Hq, d, dev, sp, ws, out, lse):
    lib = load()
    args = _PACK_ARGS(*f, 0, 0)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(lib.fdma_paged_workspace_size(args), dtype=torch.uint8, device=dev)
    st = lib.fdma_paged_fwd(args[:-16] + _PACK_WORKSPACE(ws.data_ptr(), ws.numel() * ws.element_size()), out.data_ptr(),
                            lse.data_ptr(), sp)
    if st:
        _fdma._raise(st, "fdma_paged_fwd")
    return out, lse


def fwd(q, k_cache, v_cache, page_table, k_lens, cu_q, max_q, *, k_exp=None, v_exp=None, causal=True, window=0, sinks=0,
        scale=None, workspace: Optional[torch.Tensor] = None, out=None, lse=None, stream=None):
    """Attention of the packed new tokens q (T, Hq, d) over the cache: (out (T, Hq, d) bf16, lse (Hq, T) fp32).

    The row at position p sees keys j <= p (all of k_lens[b] with causal=False); with window=W > 0 only those
    with j > p - W or j < sinks.  max_q (a host int) bounds the new tokens of a sequence.  scale defaults to
    d ** -0.5.  A row without keys gets out = 0 and lse = -inf; rows behind cu_q[B] are left as they are
    (uninitialised where out and lse are allocated here).  A workspace passed in serves one call at a time."""
    dev = _check_device(q, k_cache, v_cache, page_table, k_lens, cu_q, k_exp, v_exp, workspace, out, lse)
    f = _fields(q, k_cache, v_cache, page_table, k_lens, cu_q, max_q, k_exp, v_exp, causal, window, sinks, scale)
    T, Hq, d = q.shape
    if out is not None and (out.dtype is not torch.bfloat16 or out.shape != q.shape or not out.is_contiguous()):
        raise ValueError("out must be contiguous bf16 (T, Hq, d)")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (Hq, T) or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 (Hq, T)")
    _check_workspace(workspace)
    guard, sp = _on(dev, stream)
    if guard is None:
        return _launch_fwd(f, T, Hq, d, dev, sp, workspace, out, lse)
    with guard:
        return _launch_fwd(f, T, Hq, d, dev, sp, workspace, out, lse)
