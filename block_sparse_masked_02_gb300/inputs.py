"""ctypes binding of libfdma's operators on what goes into attention (include/fdma_inputs.h).

`norm_rope` divides each head's row of the queries and keys by its root mean square, multiplies it with a
learned weight and turns its pairs by the angles of its position, in one pass; `norm_rope_bwd` gives the gradients
of rows and weights.  `rel_bias` makes the (1, H, Nq, Nk) bias that `fdma.fwd` takes from a learned table by
buckets of the distance between query and key; `rel_bias_bwd` gives the gradient of the table from the dBias of
`fdma.bwd`.  A training step is

  q, k = norm_rope(...);  bias = rel_bias(...).expand(B, -1, -1, -1);  out, lse = fdma.fwd(q, k, v, bias=bias, ...)
  dq, dk, dv, dbias = fdma.bwd(...);  dtable = rel_bias_bwd(dbias, ...);  dq, dk, dqw, dkw = norm_rope_bwd(..., dq, dk, ...)

For serving, `paged.norm_rope_append` does the norm and rotation of new tokens and writes their keys and values into
the cache in one launch.  Like `fdma`, this marshals pointers and strides only: every step runs in the CUDA
kernels of libfdma.so, and there is no CPU path.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import fdma as _fdma

FDMA_FP32 = 0
FDMA_BF16 = 1
MAX_BUCKETS = 256

EXPORTED = ("fdma_norm_rope", "fdma_norm_rope_bwd_workspace_size", "fdma_norm_rope_bwd", "fdma_norm_rope_append",
            "fdma_rel_bias", "fdma_rel_bias_bwd_workspace_size", "fdma_rel_bias_bwd")


class FdmaRows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("stride", ctypes.c_int64 * 3)]


class FdmaNormRopeArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("N", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("d", ctypes.c_int32),
        ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("weight_type", ctypes.c_int32),
        ("q_weight", ctypes.c_void_p), ("q_weight_head", ctypes.c_int64),
        ("k_weight", ctypes.c_void_p), ("k_weight_head", ctypes.c_int64),
        ("rope", ctypes.c_void_p), ("rope_len", ctypes.c_int32), ("rot", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("first", ctypes.c_int32),
        ("positions", ctypes.c_void_p), ("pos_stride", ctypes.c_int64 * 2),
    ]


class FdmaRelArgs(ctypes.Structure):
    _fields_ = [
        ("H", ctypes.c_int32), ("Nq", ctypes.c_int32), ("Nk", ctypes.c_int32), ("num_starts", ctypes.c_int32),
        ("starts", ctypes.c_void_p), ("two_sided", ctypes.c_int32), ("offset", ctypes.c_int32),
    ]


# The structs as packed bytes (native alignment): a quarter of the time that ctypes fields take.
_PACK_NORM_ROPE = struct.Struct("6ifiPqPqP4iP2q").pack
_PACK_ROWS = struct.Struct("P3q").pack
_PACK_REL = struct.Struct("4iP2i").pack
_PACK_2Q = struct.Struct("2q").pack
_PACK_3Q = struct.Struct("3q").pack

_LIB = None


def load() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        lib = _fdma.load()
        # (structs go as the address of their packed bytes)
        S, P, I, N = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.fdma_norm_rope.argtypes = [S, S, S, S, S, P]
        lib.fdma_norm_rope.restype = I
        lib.fdma_norm_rope_bwd_workspace_size.argtypes = [S]
        lib.fdma_norm_rope_bwd_workspace_size.restype = N
        lib.fdma_norm_rope_bwd.argtypes = [S, S, S, S, S, S, S, P, P, P, N, P]
        lib.fdma_norm_rope_bwd.restype = I
        lib.fdma_norm_rope_append.argtypes = [S, S, S, S, S, S, P, P]
        lib.fdma_norm_rope_append.restype = I
        lib.fdma_rel_bias.argtypes = [S, P, I, S, P, S, P]
        lib.fdma_rel_bias.restype = I
        lib.fdma_rel_bias_bwd_workspace_size.argtypes = [S, I]
        lib.fdma_rel_bias_bwd_workspace_size.restype = N
        lib.fdma_rel_bias_bwd.argtypes = [S, I, P, S, I, P, P, N, P]
        lib.fdma_rel_bias_bwd.restype = I
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


def _on(dev, stream):
    """(guard that makes the device and the launch stream current, or None; stream pointer): what is
    allocated for the call then belongs to the stream that it runs on."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError("the stream belongs to another device than the tensors")
        return torch.cuda.stream(stream), stream.cuda_stream
    guard = None if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
    return guard, torch._C._cuda_getCurrentRawStream(dev.index)


def _run(guard, call):
    if guard is None:
        return call()
    with guard:
        return call()


def _rows(name, t, like=None):
    """fdma_rows of (B, N, H, d) or packed (T, H, d) rows, as packed bytes."""
    st = t.stride()
    if t.dtype is not torch.bfloat16 or len(st) not in (3, 4) or (st[-1] != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be bf16 (B, N, H, d) or (T, H, d) with a contiguous head dim")
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name} must have the shape {tuple(like.shape)}")
    return _PACK_ROWS(t.data_ptr(), *st[:3]) if len(st) == 4 else _PACK_ROWS(t.data_ptr(), 0, st[0], st[1])


def _weight(name, w, H, d):
    """(pointer, head stride, type) of a weight (d) or (H, d)."""
    if w is None:
        return 0, 0, None
    dt = FDMA_FP32 if w.dtype is torch.float32 else FDMA_BF16 if w.dtype is torch.bfloat16 else None
    shape = w.shape
    if dt is None or shape not in ((d,), (H, d)) or w.stride(-1) != 1:
        raise ValueError(f"{name} must be fp32 or bf16, ({d},) or ({H}, {d}), with a contiguous last dimension")
    head = 0
    if len(shape) == 2:
        head = w.stride(0)
        if H > 1 and head < d:
            raise ValueError(f"the heads of {name} must not overlap")
        head = max(head, d)
    return w.data_ptr(), head, dt


def _norm_rope_args(q, k, q_weight, k_weight, rope, positions, first, interleaved, norm, eps):
    """fdma_norm_rope_args as packed bytes."""
    shape = q.shape
    if len(shape) == 4:
        B, N, Hq, d = shape
    elif len(shape) == 3:
        (N, Hq, d), B = shape, 1
    else:
        raise ValueError("q must be (B, N, Hq, d) or (T, Hq, d)")
    Hk = 0
    if k is not None:
        Hk = k.shape[-2]
        if k.shape != (*shape[:-2], Hk, d):
            raise ValueError("k must have the tokens and the head dim of q")
    elif k_weight is not None:
        raise ValueError("a weight for keys without keys")
    qw, qh, qt = _weight("q_weight", q_weight, Hq, d)
    kw, kh, kt = _weight("k_weight", k_weight, Hk, d)
    if qt is not None and kt is not None and qt != kt:
        raise ValueError("q_weight and k_weight must have one type")
    wt = qt if qt is not None else kt if kt is not None else FDMA_FP32
    rp = length = rot = 0
    if rope is not None:
        if rope.dtype is not torch.float32 or rope.dim() != 3 or rope.shape[1] != 2 or not rope.is_contiguous():
            raise ValueError("rope must be contiguous fp32 (length, 2, rot / 2)")
        rp, length, rot = rope.data_ptr(), rope.shape[0], 2 * rope.shape[2]
    pp = sb = sn = 0
    if positions is not None:
        ps = positions.shape
        if positions.dtype is not torch.int32 or ps not in ((N,), (B, N)):
            raise ValueError(f"positions must be int32 ({N},) or ({B}, {N})")
        pp, sn = positions.data_ptr(), positions.stride(-1)
        sb = positions.stride(0) if len(ps) == 2 else 0
    return _PACK_NORM_ROPE(B, N, Hq, Hk, d, 1 if norm else 0, eps, wt, qw, qh, kw, kh, rp, length, rot, 1 if interleaved else 0,
                           first, pp, sb, sn)


def _as_given(t, dev):
    """An uninitialised contiguous tensor of t's shape."""
    return torch.empty(t.shape, dtype=torch.bfloat16, device=dev)


def rope_table(length, rot, *, base=10000.0, device="cuda"):
    """The table that `norm_rope` takes: fp32 (length, 2, rot / 2), cosines and sines of p * base ** (-2 i / rot), formed in
    64 bits (in 32, the angles of far positions lose what matters)."""
    f = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(length, dtype=torch.float64, device=device)[:, None] * f
    return torch.stack((a.cos(), a.sin()), 1).float()


def norm_rope(q, k=None, *, q_weight=None, k_weight=None, rope=None, positions=None, first=0, interleaved=False, norm=True,
              eps=1e-6, q_out=None, k_out=None, stream=None):
    """Norm and rotation of q (B, N, Hq, d) and k (B, N, Hk, d) or None, or packed (T, H, d), bf16 with a contiguous head
    dim: (q_out, k_out), k_out None without k.

    Each row is divided by sqrt(mean of its squares + eps) and multiplied with its weight, (d) or (heads, d), fp32 or
    bf16, None for ones (norm=False leaves all of that out).  Then the first rot values are turned: rope is the table
    of `rope_table` (None: no rotation), pairs are (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved.  Token n of each
    sequence is at position first + n, or at positions (int32 (N,) or (B, N)); a token at a negative position is padding
    and its rows are left as they are (uninitialised where the outputs are allocated here).  A position behind the
    table is left out too and reported by `fdma.device_error()`.  q_out and k_out may be q and k themselves."""
    dev = _check_device(q, k, q_weight, k_weight, rope, positions, q_out, k_out)
    args = _norm_rope_args(q, k, q_weight, k_weight, rope, positions, first, interleaved, norm, eps)
    qr, kr = _rows("q", q), None if k is None else _rows("k", k)
    guard, sp = _on(dev, stream)

    def call():
        qo = _as_given(q, dev) if q_out is None else q_out
        ko = None if k is None else _as_given(k, dev) if k_out is None else k_out
        return qo, ko, load().fdma_norm_rope(args, qr, kr, _rows("q_out", qo, q), None if k is None else _rows("k_out", ko, k), sp)

    qo, ko, st = _run(guard, call)
    if st:
        _fdma._raise(st, "fdma_norm_rope")
    return qo, ko


def norm_rope_bwd(q, k, dq_out, dk_out, *, q_weight=None, k_weight=None, rope=None, positions=None, first=0,
                  interleaved=False, norm=True, eps=1e-6, want_dweight=True, grads=None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradients (dq, dk, dq_weight, dk_weight) from those of `norm_rope`'s outputs, given its inputs: dq and dk bf16
    (zero for tokens that were left out), the weights' fp32, (d) or (heads, d) like the weights; None for what is not
    there or, with want_dweight=False, not wanted.  grads=(dq, dk, dq_weight, dk_weight) are written where they are not
    None; dq and dk may be dq_out and dk_out themselves.  A workspace passed in (uint8, `norm_rope_bwd_workspace`)
    serves one call at a time."""
    g = (None,) * 4 if grads is None else tuple(grads)
    if len(g) != 4:
        raise ValueError("grads must be (dq, dk, dq_weight, dk_weight)")
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    dev = _check_device(q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, workspace, *g)
    args = _norm_rope_args(q, k, q_weight, k_weight, rope, positions, first, interleaved, norm, eps)
    rows = (_rows("q", q), None if k is None else _rows("k", k), _rows("dq_out", dq_out, q),
            None if k is None else _rows("dk_out", dk_out, k))
    for name, w, t in (("dq_weight", q_weight, g[2]), ("dk_weight", k_weight, g[3])):
        if t is not None and (w is None or t.dtype is not torch.float32 or t.shape != w.shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous fp32 of its weight's shape")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    guard, sp = _on(dev, stream)

    def call():
        lib = load()
        dq = _as_given(q, dev) if g[0] is None else g[0]
        dk = None if k is None else _as_given(k, dev) if g[1] is None else g[1]
        dw = [None, None]
        if want_dweight:
            dw = [t if t is not None or w is None else torch.empty(w.shape, dtype=torch.float32, device=dev)
                  for w, t in ((q_weight, g[2]), (k_weight, g[3]))]
        ws, n = None, 0
        if dw[0] is not None or dw[1] is not None:
            ws = workspace
            if ws is None:
                ws = torch.empty(lib.fdma_norm_rope_bwd_workspace_size(args), dtype=torch.uint8, device=dev)
            n = ws.numel() * ws.element_size()
        st = lib.fdma_norm_rope_bwd(args, *rows, _rows("dq", dq, q), None if k is None else _rows("dk", dk, k),
                                    _fdma._ptr(dw[0]), _fdma._ptr(dw[1]), _fdma._ptr(ws), n, sp)
        return (dq, dk, dw[0], dw[1]), st

    out, st = _run(guard, call)
    if st:
        _fdma._raise(st, "fdma_norm_rope_bwd")
    return out


def norm_rope_bwd_workspace(q, k=None, *, q_weight=None, k_weight=None):
    """A workspace for `norm_rope_bwd` of these inputs."""
    dev = _check_device(q, k, q_weight, k_weight)
    args = _norm_rope_args(q, k, q_weight, k_weight, None, None, 0, False, True, 1.0)
    return torch.empty(load().fdma_norm_rope_bwd_workspace_size(args), dtype=torch.uint8, device=dev)


def rel_starts(num_buckets, max_distance, *, bidirectional=True):
    """The first distance of each bucket of one side, for the usual division: the first half of a side's buckets hold one
    distance each, the others are as wide as each other in the logarithm up to max_distance, the last one holds
    what is further too.  (bidirectional: the table's num_buckets are those of both sides.)  Borders are found in whole
    numbers."""
    n = num_buckets // 2 if bidirectional else num_buckets
    e = n // 2
    if e < 1 or (bidirectional and num_buckets % 2) or max_distance <= e:
        raise ValueError("at least two buckets a side, an even number of them in all, and max_distance behind the first half")
    m, at = n - e, list(range(e))
    for k in range(m):  # distance a is behind border k where (a / e) ** m >= (max_distance / e) ** k
        lo, hi = e, max_distance
        while lo < hi:
            mid = (lo + hi) // 2
            if mid ** m * e ** k >= max_distance ** k * e ** m:
                hi = mid
            else:
                lo = mid + 1
        at.append(lo)
    return tuple(at)


def _rel_args(H, Nq, Nk, starts, bidirectional, offset):
    """(fdma_rel_args as packed bytes, what they point to)."""
    n = len(starts)
    if not 0 < n <= MAX_BUCKETS:
        raise ValueError(f"1 to {MAX_BUCKETS} buckets a side")
    a = struct.pack("%di" % n, *starts)
    address = ctypes.cast(ctypes.c_char_p(a), ctypes.c_void_p).value
    return _PACK_REL(H, Nq, Nk, n, address, 1 if bidirectional else 0, Nk - Nq if offset is None else offset), a


def rel_bias(table, Nq, Nk, starts, *, bidirectional=True, offset=None, out=None, stream=None):
    """The bias (1, H, Nq, Nk) bf16 of a learned table (buckets, H), fp32 or bf16: table[bucket(j - (i + offset)), h] for
    query row i and key j.  starts holds the first distance of each bucket of one side (`rel_starts`): a distance is in the
    last bucket that begins at it or before.  One-sided, keys behind the query are at distance 0; bidirectional, they
    have the second half of the table.  offset is the position of query row 0 among the keys, by default Nk - Nq (as
    `fdma.fwd`'s causal).  Nk is a multiple of 8.  `expand` it over a batch."""
    dev = _check_device(table, out)
    dt = FDMA_FP32 if table.dtype is torch.float32 else FDMA_BF16 if table.dtype is torch.bfloat16 else None
    if dt is None or table.dim() != 2 or table.shape[0] != (2 if bidirectional else 1) * len(starts):
        raise ValueError("table must be fp32 or bf16 (buckets, H), with len(starts) buckets (twice as many if bidirectional)")
    H = table.shape[1]
    args, keep = _rel_args(H, Nq, Nk, starts, bidirectional, offset)
    if out is not None and (out.dtype is not torch.bfloat16 or out.shape != (1, H, Nq, Nk) or (Nk > 1 and out.stride(3) != 1)):
        raise ValueError("out must be bf16 (1, H, Nq, Nk) with contiguous columns")
    guard, sp = _on(dev, stream)

    def call():
        o = torch.empty((1, H, Nq, Nk), dtype=torch.bfloat16, device=dev) if out is None else out
        return o, load().fdma_rel_bias(args, table.data_ptr(), dt, _PACK_2Q(*table.stride()), o.data_ptr(),
                                       _PACK_2Q(o.stride(1), o.stride(2)), sp)

    o, st = _run(guard, call)
    if st:
        _fdma._raise(st, "fdma_rel_bias")
    return o


def rel_bias_bwd(dbias, starts, *, bidirectional=True, offset=None, causal=False, dtable=None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradient (buckets, H) fp32 of `rel_bias`'s table from dbias (B, H, Nq, Nk) bf16, as `fdma.bwd` returns it, summed
    over the batch too.  With causal=True keys behind the query count as zeros and most are not read.  A workspace
    passed in (uint8, `rel_bias_bwd_workspace`) serves one call at a time."""
    dev = _check_device(dbias, dtable, workspace)
    st = dbias.stride()
    if dbias.dtype is not torch.bfloat16 or len(st) != 4 or (st[3] != 1 and dbias.shape[3] > 1):
        raise ValueError("dbias must be bf16 (B, H, Nq, Nk) with contiguous columns")
    B, H, Nq, Nk = dbias.shape
    args, keep = _rel_args(H, Nq, Nk, starts, bidirectional, offset)
    shape = ((2 if bidirectional else 1) * len(starts), H)
    if dtable is not None and (dtable.dtype is not torch.float32 or dtable.shape != shape or not dtable.is_contiguous()):
        raise ValueError(f"dtable must be contiguous fp32 {shape}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    guard, sp = _on(dev, stream)

    def call():
        lib = load()
        out = torch.empty(shape, dtype=torch.float32, device=dev) if dtable is None else dtable
        ws = workspace
        if ws is None:
            ws = torch.empty(lib.fdma_rel_bias_bwd_workspace_size(args, B), dtype=torch.uint8, device=dev)
        return out, lib.fdma_rel_bias_bwd(args, B, dbias.data_ptr(), _PACK_3Q(*st[:3]), 1 if causal else 0, out.data_ptr(),
                                          ws.data_ptr(), ws.numel() * ws.element_size(), sp)

    out, status = _run(guard, call)
    if status:
        _fdma._raise(status, "fdma_rel_bias_bwd")
    return out


def rel_bias_bwd_workspace(B, H, Nq, Nk, starts, *, bidirectional=True, device="cuda"):
    """A workspace for `rel_bias_bwd` of these sizes."""
    args, keep = _rel_args(H, Nq, Nk, starts, bidirectional, None)
    return torch.empty(load().fdma_rel_bias_bwd_workspace_size(args, B), dtype=torch.uint8, device=device)
