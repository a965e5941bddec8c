"""float64 reference of what goes into attention: norm and rotation of rows, and the learned bias by distance."""
import numpy as np


def _pairs(rot, interleaved):
    p = np.arange(rot // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)


def turn(y, cos, sin, interleaved, back=False):
    """Rows y (..., d) with their first 2 * cos.shape[-1] values turned; and the sum of the magnitudes of each value's terms."""
    out, mag = y.copy(), np.abs(y)
    if cos is None:
        return out, mag
    i, j = _pairs(2 * cos.shape[-1], interleaved)
    s = -sin if back else sin
    a, b = y[..., i], y[..., j]
    out[..., i], out[..., j] = a * cos - b * s, b * cos + a * s
    mag[..., i], mag[..., j] = np.abs(a * cos) + np.abs(b * s), np.abs(b * cos) + np.abs(a * s)
    return out, mag


def rms(x, eps):
    return np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def norm_rope(x, w, cos, sin, interleaved, norm, eps):
    """(output, magnitudes of its terms) of rows x (..., H, d); w (d) or (H, d) or None; cos, sin (..., 1, rot / 2) or None."""
    y = x / rms(x, eps) if norm else x
    return turn(y if w is None else y * w, cos, sin, interleaved)


def norm_rope_bwd(x, dout, w, cos, sin, interleaved, norm, eps):
    """(dx, magnitudes of its terms, dw by head, magnitudes of its terms); dw (H, d) summed over all axes but the last two."""
    g, gm = turn(dout, cos, sin, interleaved, back=True)
    if not norm:
        return g, gm, None, None
    r = rms(x, eps)
    xn = x / r
    over = tuple(range(x.ndim - 2))
    dw, dwm = (g * xn).sum(over), (gm * np.abs(xn)).sum(over)
    wv = 1.0 if w is None else w
    dx = (g * wv - xn * (g * wv * xn).mean(-1, keepdims=True)) / r
    aw = np.abs(wv)
    mag = (gm * aw + np.abs(xn) * (gm * aw * np.abs(xn)).mean(-1, keepdims=True)) / r
    return dx, mag, dw, dwm


def buckets(Nq, Nk, starts, two_sided, offset):
    """(Nq, Nk) bucket of each (query, key)."""
    delta = np.arange(Nk)[None, :] - (np.arange(Nq)[:, None] + offset)
    a = np.abs(delta) if two_sided else np.maximum(-delta, 0)
    side = np.zeros(a.shape, dtype=np.int64)
    for s, first in enumerate(starts):  # the last bucket that begins at the distance or before
        side[a >= first] = s
    return side + len(starts) * (delta > 0) if two_sided else side


def rel_bias(table, Nq, Nk, starts, two_sided, offset):
    """(H, Nq, Nk) of a table (buckets, H)."""
    return np.moveaxis(table[buckets(Nq, Nk, starts, two_sided, offset)], -1, 0)


def rel_bias_bwd(dbias, starts, two_sided, offset, causal):
    """(gradient (buckets, H), sum of the magnitudes of its terms) of dbias (B, H, Nq, Nk)."""
    B, H, Nq, Nk = dbias.shape
    at = buckets(Nq, Nk, starts, two_sided, offset)
    x, m = dbias.sum(0), np.abs(dbias).sum(0)
    if causal:
        seen = np.arange(Nk)[None, :] <= np.arange(Nq)[:, None] + offset
        x, m = np.where(seen, x, 0), np.where(seen, m, 0)
    n = len(starts) * (2 if two_sided else 1)
    out, mag = np.zeros((n, H)), np.zeros((n, H))
    for h in range(H):
        out[:, h] = np.bincount(at.ravel(), x[h].ravel(), n)
        mag[:, h] = np.bincount(at.ravel(), m[h].ravel(), n)
    return out, mag
