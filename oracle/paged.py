"""CPU oracle of the paged key/value cache operators (append, gather, attention of new tokens).

TEST INFRASTRUCTURE ONLY.  Only the test suite may import this module; the product path never does.
It shares no code with the CUDA path.

numpy float64, one sequence, head and row block at a time, straight from the definitions:

  position of new token i of n      p = k_len - n + i, in slot (table[p // page], p % page)
  e4m3 row x                        e least with max |x| <= 448 2^e (-126 <= e <= 119), value
                                    round-to-nearest-even of x 2^-e to e4m3, at most 448, times 2^e
  attention of the row at p         over keys j <= p (all, not causal), with a window w only those with
                                    j > p - w or j < sinks; out = softmax(scale q.k) v, lse = log sum exp
"""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 256 values of the e4m3 codes (1 sign, 4 exponent, 3 mantissa bits, bias 7, S.1111.111 = NaN)."""
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            x = np.nan
        out[code] = -x if code & 128 else x
    return out


_VALUES = e4m3_values()
_POS = _VALUES[:127]  # 0 .. 448, increasing


def _round_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest values (ties to the even code), saturating; NaN to code 127."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, np.nan_to_num(a, nan=0.0)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = np.abs(_POS[hi] - a), np.abs(a - _POS[lo])
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(x: np.ndarray):
    """Rows (last axis) of x as (codes uint8, scale bytes uint8)."""
    x = np.asarray(x, np.float64)
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -126, np.int64)
    for i in np.ndindex(*top.shape):
        while e[i] < 119 and 448.0 * 2.0 ** int(e[i]) < top[i]:
            e[i] += 1
    return _round_e4m3(x * np.exp2(-e.astype(np.float64))[..., None]), (e + 127).astype(np.uint8)


def dequantise(code: np.ndarray, byte: np.ndarray) -> np.ndarray:
    return _VALUES[code] * np.exp2(byte.astype(np.float64) - 127)[..., None]


def slots(table_row, page, positions):
    positions = np.asarray(positions, np.int64)
    return np.asarray(table_row)[positions // page], positions % page


def gather(cache, table_row, n):
    """Rows 0 .. n-1 of one sequence: cache (pages, page, Hkv, d) float64."""
    pg, at = slots(table_row, cache.shape[1], np.arange(n))
    return cache[pg, at]


def visible(p, n_keys, causal, window, sinks):
    j = np.arange(n_keys)
    if not causal:
        return np.ones(n_keys, bool)
    keep = j <= p
    if window > 0:
        keep &= (j > p - window) | (j < sinks)
    return keep


def attend(q, K, V, scale, causal=True, window=0, sinks=0):
    """q (n, Hq, d), K, V (keys, Hkv, d) of one sequence.  Returns out (n, Hq, d), lse (n, Hq), and two
    magnitudes that error bounds are made of: A = sum_j P_j |v_j| (n, Hq, d) and
    D = max_j scale * sum_c |q_c k_jc| over the visible keys (n, Hq)."""
    n, Hq, d = q.shape
    nk, Hkv = K.shape[0], K.shape[1]
    out, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    A, D = np.zeros((n, Hq, d)), np.zeros((n, Hq))
    for i in range(n):
        keep = visible(nk - n + i, nk, causal, window, sinks)
        if not keep.any():
            continue
        for h in range(Hq):
            k, v = K[keep, h // (Hq // Hkv)], V[keep, h // (Hq // Hkv)]
            s = scale * (k @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            out[i, h], A[i, h] = (p / p.sum()) @ v, (p / p.sum()) @ np.abs(v)
            lse[i, h] = m + np.log(p.sum())
            D[i, h] = scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, lse, A, D
