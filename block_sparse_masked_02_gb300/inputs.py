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
        ("two_sided", ctypes.c_int32), ("offset", ctypes.c_int32),
    ]


# The structs as packed bytes (native alignment): a quarter of the time that ctypes fields take.
_PACK_NORM_ROPE = struct.Struct("6ifiPqPqP4iP2q").pack
_PACK_ROWS = struct.Struct("P3q").pack
_PACK_REL = struct.Struct("6i").pack
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
        lib.fdma_rel_bias.argtypes = [S, S, P, I, S, P, S, P]
        lib.fdma_rel_bias.restype = I
        lib.fdma_rel_bias_bwd_workspace_size.argtypes = [S, I]
        lib.fdma_rel_bias_bwd_workspace_size.restype = N
        lib.fdma_rel_bias_bwd.argtypes = [S, S, I, P, S, I, P, P, N, P]
        lib.fdma_rel_bias_bwd.restype = I
        _LIB = lib
    return _LIB


_BF16, _FP32, _I32 = torch.bfloat16, torch.float32, torch.int32
_FP32_MAX = torch.finfo(torch.float32).max
# (a torch built without CUDA has none of these; it can still import this)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# A call's own workspace comes from the caching allocator without a tensor around it, which would cost 3 us (a torch that does
# not have these calls makes the tensor).
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _check_device(first, *ts):
    """The index of the device that all tensors of a call are on."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("libfdma takes CUDA tensors only (no CPU path)")
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors of a call are on one device")
    return dev


def _on(dev, stream):
    """(guard that makes the device and the launch stream current, or None; stream pointer): what is
    allocated for the call then belongs to the stream that it runs on."""
    if stream is None:
        return (None if _current_device() == dev else torch.cuda.device(dev)), _raw_stream(dev)
    if stream.device.index != dev:
        raise ValueError("the stream belongs to another device than the tensors")
    return torch.cuda.stream(stream), stream.cuda_stream


def _workspace(n, dev, sp):
    """(address of n bytes for a call on the stream sp, which is current; the raw block or the tensor that holds them)."""
    if _raw_alloc is None or _raw_delete is None:
        t = torch.empty(n, dtype=torch.uint8, device=dev)
        return t.data_ptr(), t
    p = _raw_alloc(n, sp)
    return p, p


def _release(own):
    """Gives a workspace back: what is allocated next on its stream runs behind the kernels that were launched with it."""
    if type(own) is int and own:
        _raw_delete(own)


def _run(guard, call, *args):
    if guard is None:
        return call(*args)
    with guard:
        return call(*args)


def _rows(name, t, shape=None):
    """fdma_rows of (B, N, H, d) or packed (T, H, d) rows, as packed bytes."""
    st = t.stride()
    n = len(st)
    if t.dtype is not _BF16 or (n != 4 and n != 3) or (st[-1] != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be bf16 (B, N, H, d) or (T, H, d) with a contiguous head dim")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")
    return _PACK_ROWS(t.data_ptr(), st[0], st[1], st[2]) if n == 4 else _PACK_ROWS(t.data_ptr(), 0, st[0], st[1])


def _new_rows(like):
    """An uninitialised contiguous tensor of a tensor's shape, and its fdma_rows."""
    t = torch.empty_like(like, memory_format=torch.contiguous_format)
    shape = t.shape
    hd = shape[-2] * shape[-1]
    return t, _PACK_ROWS(t.data_ptr(), shape[-3] * hd, hd, shape[-1])


def _weight(name, w, H, d):
    """(pointer, head stride, type) of a weight (d) or (H, d)."""
    dt, shape = w.dtype, w.shape
    dt = FDMA_FP32 if dt is _FP32 else FDMA_BF16 if dt is _BF16 else None
    if len(shape) == 1:
        if dt is not None and shape[0] == d and w.stride(0) == 1:
            return w.data_ptr(), 0, dt
    elif dt is not None and shape == (H, d):
        head, one = w.stride()
        if one == 1 and (H == 1 or head >= d):
            return w.data_ptr(), head if H > 1 else d, dt
    raise ValueError(f"{name} must be fp32 or bf16, ({d},) or ({H}, {d}), its heads apart and contiguous")


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
        ks = k.shape
        Hk = ks[-2]
        if ks != ((B, N, Hk, d) if len(shape) == 4 else (N, Hk, d)):
            raise ValueError("k must have the tokens and the head dim of q")
    elif k_weight is not None:
        raise ValueError("a weight for keys without keys")
    qw = qh = kw = kh = 0
    wt = kt = None
    if q_weight is not None:
        qw, qh, wt = _weight("q_weight", q_weight, Hq, d)
    if k_weight is not None:
        kw, kh, kt = _weight("k_weight", k_weight, Hk, d)
        if wt is None:
            wt = kt
        elif wt != kt:
            raise ValueError("q_weight and k_weight must have one type")
    rp = length = rot = 0
    if rope is not None:
        rs = rope.shape
        if rope.dtype is not _FP32 or len(rs) != 3 or rs[1] != 2 or not rope.is_contiguous():
            raise ValueError("rope must be contiguous fp32 (length, 2, rot / 2)")
        rp, length, rot = rope.data_ptr(), rs[0], 2 * rs[2]
    pp = sb = sn = 0
    if positions is not None:
        ps, st = positions.shape, positions.stride()
        if positions.dtype is not _I32 or (ps != (N,) and ps != (B, N)):
            raise ValueError(f"positions must be int32 ({N},) or ({B}, {N})")
        pp, sn = positions.data_ptr(), st[-1]
        sb = st[0] if len(st) == 2 else 0
    try:
        args = _PACK_NORM_ROPE(B, N, Hq, Hk, d, 1 if norm else 0, eps, wt or 0, qw, qh, kw, kh, rp, length, rot,
                               1 if interleaved else 0, first, pp, sb, sn)
    except struct.error:
        args = None
    if args is None or eps > _FP32_MAX:
        raise ValueError("sizes and first must be whole numbers of 32 bits, eps a number that fp32 holds")
    return args


def rope_table(length, rot, *, base=10000.0, device="cuda"):
    """The table that `norm_rope` takes: fp32 (length, 2, rot / 2), cosines and sines of p * base ** (-2 i / rot), formed in
    64 bits (in 32, the angles of far positions lose what matters)."""
    f = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(length, dtype=torch.float64, device=device)[:, None] * f
    return torch.stack((a.cos(), a.sin()), 1).float()


def _launch_norm_rope(args, q, k, q_out, k_out, sp):
    kr = kor = None
    if q_out is None:
        q_out, qor = _new_rows(q)
    else:
        qor = _rows("q_out", q_out, q.shape)
    if k is not None:
        kr = _rows("k", k)
        if k_out is None:
            k_out, kor = _new_rows(k)
        else:
            kor = _rows("k_out", k_out, k.shape)
    st = load().fdma_norm_rope(args, _rows("q", q), kr, qor, kor, sp)
    if st:
        _fdma._raise(st, "fdma_norm_rope")
    return q_out, k_out


def norm_rope(q, k=None, *, q_weight=None, k_weight=None, rope=None, positions=None, first=0, interleaved=False, norm=True,
              eps=1e-6, q_out=None, k_out=None, stream=None):
    """Norm and rotation of q (B, N, Hq, d) and k (B, N, Hk, d) or None, or packed (T, H, d), bf16 with a contiguous head
    dim: (q_out, k_out), k_out None without k.

    Each row is divided by sqrt(mean of its squares + eps) and multiplied with its weight, (d) or (heads, d) (both
    weights of one form), fp32 or bf16, None for ones (norm=False leaves all of that out).  Then the first rot values
    are turned: rope is the table of `rope_table` (None: no rotation), pairs are (i, i + rot / 2), or (2 i, 2 i + 1) if
    interleaved.  Token n of each sequence is at position first + n, or at positions (int32 (N,) or (B, N)); a token
    at a negative position is padding and its rows are left as they are (uninitialised where the outputs are
    allocated here).  A position behind the table is left out too and reported by `fdma.device_error()`.  q_out and
    k_out may be q and k themselves."""
    if k is None and k_out is not None:
        raise ValueError("an output for keys without keys")
    dev = _check_device(q, k, q_weight, k_weight, rope, positions, q_out, k_out)
    args = _norm_rope_args(q, k, q_weight, k_weight, rope, positions, first, interleaved, norm, eps)
    guard, sp = _on(dev, stream)
    return _run(guard, _launch_norm_rope, args, q, k, q_out, k_out, sp)


def _launch_norm_rope_bwd(args, q, k, dq_out, dk_out, weights, grads, want_dweight, ws, sp):
    lib = load()
    dq, dk, *dw = grads
    kr = kg = ko = None
    if dq is None:
        dq, qo = _new_rows(q)
    else:
        qo = _rows("dq", dq, q.shape)
    if k is not None:
        if dk is None:
            dk, ko = _new_rows(k)
        else:
            ko = _rows("dk", dk, k.shape)
        kr, kg = _rows("k", k), _rows("dk_out", dk_out, k.shape)
    n = wp = own = 0
    if want_dweight:
        dw = [torch.empty_like(w, dtype=_FP32, memory_format=torch.contiguous_format) if t is None and w is not None else t
              for w, t in zip(weights, dw)]
        if dw[0] is not None or dw[1] is not None:
            if ws is None:
                n = lib.fdma_norm_rope_bwd_workspace_size(args)
            else:
                wp, n = ws.data_ptr(), ws.numel() * ws.element_size()
    else:
        dw = (None, None)
    rows = (_rows("q", q), kr, _rows("dq_out", dq_out, q.shape), kg, qo, ko)
    if n and ws is None:
        wp, own = _workspace(n, q.device, sp)
    st = lib.fdma_norm_rope_bwd(args, *rows, None if dw[0] is None else dw[0].data_ptr(),
                                None if dw[1] is None else dw[1].data_ptr(), wp, n, sp)
    _release(own)
    if st:
        _fdma._raise(st, "fdma_norm_rope_bwd")
    return dq, dk, dw[0], dw[1]


def norm_rope_bwd(q, k, dq_out, dk_out, *, q_weight=None, k_weight=None, rope=None, positions=None, first=0,
                  interleaved=False, norm=True, eps=1e-6, want_dweight=True, grads=None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradients (dq, dk, dq_weight, dk_weight) from those of `norm_rope`'s outputs, given its inputs: dq and dk bf16
    (zero for tokens that were left out), the weights' fp32, (d) or (heads, d) like the weights; None for what is not
    there or, with want_dweight=False, not wanted.  grads=(dq, dk, dq_weight, dk_weight) are written where they are not
    None (one that the call would not write is refused); dq and dk may be dq_out and dk_out themselves.  A workspace
    passed in (uint8, `norm_rope_bwd_workspace`) serves one call at a time."""
    g = (None,) * 4 if grads is None else tuple(grads)
    if len(g) != 4:
        raise ValueError("grads must be (dq, dk, dq_weight, dk_weight)")
    if not want_dweight and (g[2] is not None or g[3] is not None):
        raise ValueError("grads holds a weight's gradient that want_dweight=False leaves out")
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    if k is None and g[1] is not None:
        raise ValueError("an output for keys without keys")
    dev = _check_device(q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, workspace, *g)
    args = _norm_rope_args(q, k, q_weight, k_weight, rope, positions, first, interleaved, norm, eps)
    for name, w, t in (("dq_weight", q_weight, g[2]), ("dk_weight", k_weight, g[3])):
        if t is not None and (w is None or t.dtype is not _FP32 or t.shape != w.shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous fp32 of its weight's shape")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    guard, sp = _on(dev, stream)
    return _run(guard, _launch_norm_rope_bwd, args, q, k, dq_out, dk_out, (q_weight, k_weight), g, want_dweight, workspace, sp)


def norm_rope_bwd_workspace(q, k=None, *, q_weight=None, k_weight=None, rope=None, interleaved=False):
    """A workspace for `norm_rope_bwd` of these inputs."""
    _check_device(q, k, q_weight, k_weight, rope)
    args = _norm_rope_args(q, k, q_weight, k_weight, rope, None, 0, interleaved, True, 1.0)
    return torch.empty(load().fdma_norm_rope_bwd_workspace_size(args), dtype=torch.uint8, device=q.device)


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
    """(fdma_rel_args, starts) as packed bytes."""
    n = len(starts)
    if not 0 < n <= MAX_BUCKETS:
        raise ValueError(f"1 to {MAX_BUCKETS} buckets a side")
    try:
        return (_PACK_REL(H, Nq, Nk, n, 1 if bidirectional else 0, Nk - Nq if offset is None else offset),
                struct.pack(f"{n}i", *starts))
    except struct.error:
        raise ValueError("sizes, offset and starts must be whole numbers of 32 bits") from None


def _launch_rel_bias(args, first, table, dt, out, shape, sp):
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=table.device)
    ts, os = table.stride(), out.stride()
    st = load().fdma_rel_bias(args, first, table.data_ptr(), dt, _PACK_2Q(ts[0], ts[1]), out.data_ptr(), _PACK_2Q(os[1], os[2]), sp)
    if st:
        _fdma._raise(st, "fdma_rel_bias")
    return out


def rel_bias(table, Nq, Nk, starts, *, bidirectional=True, offset=None, out=None, stream=None):
    """The bias (1, H, Nq, Nk) bf16 of a learned table (buckets, H), fp32 or bf16: table[bucket(j - (i + offset)), h] for
    query row i and key j.  starts holds the first distance of each bucket of one side (`rel_starts`): a distance is in the
    last bucket that begins at it or before.  One-sided, keys behind the query are at distance 0; bidirectional, they
    have the second half of the table.  H is the number of kv heads, as `fdma.fwd` takes a bias (B, Hkv, Nq, Nk) (or 1, to
    be expanded over them; the gradient is then the sum of `rel_bias_bwd`'s columns): query heads that share a kv head share
    its bias.  offset is the position of query row 0 among the keys, by default Nk - Nq (as `fdma.fwd`'s causal).  Nk is a
    multiple of 8.  `expand` it over a batch."""
    dev = _check_device(table, out)
    dt, shape = table.dtype, table.shape
    dt = FDMA_FP32 if dt is _FP32 else FDMA_BF16 if dt is _BF16 else None
    if dt is None or len(shape) != 2 or shape[0] != (2 if bidirectional else 1) * len(starts):
        raise ValueError("table must be fp32 or bf16 (buckets, H), with len(starts) buckets (twice as many if bidirectional)")
    args, first = _rel_args(shape[1], Nq, Nk, starts, bidirectional, offset)
    shape = (1, shape[1], Nq, Nk)
    if out is not None and (out.dtype is not _BF16 or out.shape != shape or (Nk > 1 and out.stride(3) != 1)):
        raise ValueError("out must be bf16 (1, H, Nq, Nk) with contiguous columns")
    guard, sp = _on(dev, stream)
    return _run(guard, _launch_rel_bias, args, first, table, dt, out, shape, sp)


def _launch_rel_bias_bwd(args, first, dbias, causal, dtable, shape, ws, sp):
    lib = load()
    st = dbias.stride()
    if dtable is None:
        dtable = torch.empty(shape, dtype=_FP32, device=dbias.device)
    B, wp, own = dbias.shape[0], 0, 0
    if ws is None:
        n = lib.fdma_rel_bias_bwd_workspace_size(args, B)
        if n:
            wp, own = _workspace(n, dbias.device, sp)
    else:
        wp, n = ws.data_ptr(), ws.numel() * ws.element_size()
    st = lib.fdma_rel_bias_bwd(args, first, B, dbias.data_ptr(), _PACK_3Q(st[0], st[1], st[2]), 1 if causal else 0, dtable.data_ptr(),
                               wp, n, sp)
    _release(own)
    if st:
        _fdma._raise(st, "fdma_rel_bias_bwd")
    return dtable


def rel_bias_bwd(dbias, starts, *, bidirectional=True, offset=None, causal=False, dtable=None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """The gradient (buckets, H) fp32 of `rel_bias`'s table from dbias (B, H, Nq, Nk) bf16, as `fdma.bwd` returns it, summed
    over the batch too.  With causal=True keys behind the query count as zeros and most are not read.  A workspace
    passed in (uint8, `rel_bias_bwd_workspace`) serves one call at a time."""
    dev = _check_device(dbias, dtable, workspace)
    st, ds = dbias.stride(), dbias.shape
    if dbias.dtype is not _BF16 or len(st) != 4 or (st[3] != 1 and ds[3] > 1):
        raise ValueError("dbias must be bf16 (B, H, Nq, Nk) with contiguous columns")
    args, first = _rel_args(ds[1], ds[2], ds[3], starts, bidirectional, offset)
    shape = ((2 if bidirectional else 1) * len(starts), ds[1])
    if dtable is not None and (dtable.dtype is not _FP32 or dtable.shape != shape or not dtable.is_contiguous()):
        raise ValueError(f"dtable must be contiguous fp32 {shape}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    guard, sp = _on(dev, stream)
    return _run(guard, _launch_rel_bias_bwd, args, first, dbias, causal, dtable, shape, workspace, sp)


def rel_bias_bwd_workspace(B, H, Nq, Nk, starts, *, bidirectional=True, device="cuda"):
    """A workspace for `rel_bias_bwd` of these sizes."""
    args, _ = _rel_args(H, Nq, Nk, starts, bidirectional, None)
    return torch.empty(load().fdma_rel_bias_bwd_workspace_size(args, B), dtype=torch.uint8, device=device)
