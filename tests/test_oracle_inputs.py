"""Pins of the oracle of what goes into attention (oracle/inputs.py) against independent computations, on the CPU."""
import math

import numpy as np
import pytest
import torch

from oracle import inputs as orc


def _case(seed, H=3, N=4, d=16, rot=8, per_head=True):
    g = np.random.default_rng(seed)
    x, do = g.standard_normal((N, H, d)), g.standard_normal((N, H, d))
    w = g.standard_normal((H, d) if per_head else (d,))
    a = g.standard_normal((N, 1, rot // 2)) * 3
    return x, do, w, np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_against_a_loop(interleaved):
    x, _, w, c, s = _case(1)
    out, _ = orc.norm_rope(x, w, c, s, interleaved, True, 1e-3)
    for n in range(4):
        for h in range(3):
            r = math.sqrt(sum(v * v for v in x[n, h]) / 16 + 1e-3)
            y = [x[n, h, j] / r * w[h, j] for j in range(16)]
            z = list(y)
            for p in range(4):
                i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + 4)
                # a complex number turned by the angle
                t = complex(y[i], y[j]) * complex(c[n, 0, p], s[n, 0, p])
                z[i], z[j] = t.real, t.imag
            assert np.allclose(out[n, h], z, rtol=1e-13, atol=1e-13)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradients_against_differences(interleaved, per_head, norm):
    x, do, w, c, s = _case(2, per_head=per_head)
    w = w if norm else None
    dx, mag, dw, _ = orc.norm_rope_bwd(x, do, w, c, s, interleaved, norm, 1e-3)
    assert (np.abs(dx) <= mag * (1 + 1e-12)).all()
    f = lambda x, w: (orc.norm_rope(x, w, c, s, interleaved, norm, 1e-3)[0] * do).sum()  # noqa: E731
    h = 1e-6
    for at in [(0, 0, 0), (1, 2, 5), (3, 1, 9), (2, 0, 15)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    if norm:
        dw = dw if per_head else dw.sum(0)
        for at in ([(0, 3), (2, 15)] if per_head else [(3,), (15,)]):
            e = np.zeros_like(w)
            e[at] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[at]) < 1e-7


@pytest.mark.parametrize("two_sided,far,n", [(False, 128, 32), (True, 128, 32), (False, 40, 8), (True, 1000, 64)])
def test_usual_buckets_are_those_of_the_logarithm(two_sided, far, n):
    from block_sparse_masked_02_gb300 import inputs

    starts = inputs.rel_starts(n, far, bidirectional=two_sided)
    side = n // 2 if two_sided else n
    e = side // 2
    at = orc.buckets(700, 900, starts, two_sided, 100)
    for i in range(0, 700, 37):
        for j in range(0, 900, 23):
            delta = j - (i + 100)
            a = abs(delta) if two_sided else max(-delta, 0)
            want = a if a < e else min(side - 1, e + int(math.floor(math.log(a / e) / math.log(far / e) * (side - e) + 1e-9)))
            assert at[i, j] == want + (side if two_sided and delta > 0 else 0)


def test_bias_and_its_gradient_are_adjoint():
    g = np.random.default_rng(3)
    starts, db = (0, 1, 2, 5, 5, 9), g.standard_normal((2, 3, 11, 16))
    for two_sided in (False, True):
        t = g.standard_normal((12 if two_sided else 6, 3))
        bias = orc.rel_bias(t, 11, 16, starts, two_sided, 4)
        dt, mag = orc.rel_bias_bwd(db, starts, two_sided, 4, False)
        assert np.isclose((bias[None] * db).sum(), (t * dt).sum(), rtol=1e-12)
        assert not dt[3].any() and (np.abs(dt) <= mag + 1e-12).all()
        dc, _ = orc.rel_bias_bwd(db, starts, two_sided, 4, True)
        assert np.isclose(dc.sum(), sum(db[:, :, i, :i + 5].sum() for i in range(11)), rtol=1e-12)


def test_rope_table_is_the_cosine_and_sine_of_64_bit_angles():
    from block_sparse_masked_02_gb300 import inputs

    t = inputs.rope_table(70001, 8, base=500.0, device="cpu")
    assert t.shape == (70001, 2, 4) and t.dtype == torch.float32
    for p in (0, 1, 69999):
        for i in range(4):
            a = p * 500.0 ** (-2 * i / 8)
            assert abs(t[p, 0, i] - math.cos(a)) < 1e-7 and abs(t[p, 1, i] - math.sin(a)) < 1e-7
