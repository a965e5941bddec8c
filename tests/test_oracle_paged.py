"""Pins of the paged-cache oracle (oracle/paged.py) against independent computations, on the CPU."""
import numpy as np
import pytest
import torch

from oracle import paged as orc


def test_e4m3_values_match_torch():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = orc.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_rounding_matches_torch_for_every_bf16_in_range():
    x = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(orc._round_e4m3(x.double().numpy()), want)


def test_quantise_takes_the_least_exponent_and_round_trips():
    g = np.random.default_rng(3)
    x = torch.tensor(g.standard_normal((40, 16)) * np.exp(g.uniform(-60, 60, (40, 1)))).bfloat16().double().numpy()
    x[0] = 0
    x[1, 0] = np.inf
    x[2, 0] = np.nan
    code, e = orc.quantise(x)
    y = orc.dequantise(code, e)
    assert e[0] == 1 and not y[0].any()
    assert np.isnan(y[2, 0]) and np.isfinite(y[2, 1:]).all()
    assert y[1, 0] == 448 * 2.0 ** (int(e[1]) - 127)
    for i in range(3, 40):
        top = np.abs(x[i]).max()
        assert top <= 448 * 2.0 ** (int(e[i]) - 127) and top > 448 * 2.0 ** (int(e[i]) - 128)
        # half a step of three mantissa bits, or of the least value
        assert (np.abs(y[i] - x[i]) <= np.maximum(np.abs(x[i]) * 2.0 ** -4, 2.0 ** (int(e[i]) - 127 - 10))).all()
    # the values are bf16 numbers
    z = y[3:]
    assert np.array_equal(torch.tensor(z).bfloat16().double().numpy(), z)


@pytest.mark.parametrize("n,nk,window,sinks,causal", [(1, 9, 0, 0, True), (5, 5, 0, 0, True), (4, 30, 7, 3, True),
                                                      (3, 20, 0, 0, False), (6, 4, 0, 0, True), (2, 12, 50, 1, True)])
def test_attend_matches_a_loop_over_scores(n, nk, window, sinks, causal):
    g = np.random.default_rng(n * 100 + nk)
    Hq, Hkv, d = 4, 2, 8
    q, K, V = g.standard_normal((n, Hq, d)), g.standard_normal((nk, Hkv, d)), g.standard_normal((nk, Hkv, d))
    out, lse, _, _ = orc.attend(q, K, V, 0.3, causal, window, sinks)
    for i in range(n):
        for h in range(Hq):
            num, den = np.zeros(d), 0.0
            p = nk - n + i
            for j in range(nk):
                if causal and j > p:
                    continue
                if window and not (j > p - window or j < sinks):
                    continue
                w = np.exp(0.3 * sum(q[i, h, c] * K[j, h // 2, c] for c in range(d)))
                num += w * V[j, h // 2]
                den += w
            if den == 0:
                assert not out[i, h].any() and lse[i, h] == -np.inf
            else:
                assert np.allclose(out[i, h], num / den, rtol=1e-12, atol=0) and np.isclose(lse[i, h], np.log(den), rtol=1e-12)


def test_gather_follows_the_table():
    cache = np.arange(5 * 16 * 2 * 3, dtype=np.float64).reshape(5, 16, 2, 3)
    rows = orc.gather(cache, [4, 1, 99], 20)
    assert np.array_equal(rows[:16], cache[4]) and np.array_equal(rows[16:], cache[1, :4])
