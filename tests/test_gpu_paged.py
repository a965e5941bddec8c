"""The paged key/value cache operators on the GPU against the float64 oracle (oracle/paged.py).

Bounds.  Let u be half a step of the type that the softmax weights are held in for the product with V,
relative to the value: 2^-8 for bf16 (bf16 caches, and every cache in the chunk kernel, whose values
are bf16 in shared memory), 2^-11 for f16 (e4m3 caches in the token kernel: up to 16 rows (new tokens
times heads of a group) a sequence).  A weight P_j carries its own rounding (u) and the error of its score: a sum of d products in
fp32 is off by at most d * 2^-24 * sum |q_c k_c| (times scale: d 2^-24 D), the exponent's argument
S * log2(e) - max and the exponential itself by a few 2^-22 relative to the score's size.  With
w = 2^-22 * (8 + d * D) for both numerator and denominator, every output element is off by at most
    2^-8 |out|  +  (u + 2 w) * A,      A = sum_j P_j |v_j|,
and lse by at most w + 2^-22 |lse|.  Quantised rows and rows read back are exact.
"""
import os

import numpy as np
import pytest
import torch

from oracle import paged as orc

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_masked_02_gb300 import fdma, paged

    paged.load()
    assert fdma.device_error() == 0
    return paged


@pytest.fixture(autouse=True)
def no_device_error(P):
    yield
    from block_sparse_masked_02_gb300 import fdma

    assert fdma.device_error() == 0


def _np(t):
    return t.double().cpu().numpy()


class Setup:
    """A cache filled with `lens` keys a sequence through scattered pages; what no sequence owns holds NaN."""

    def __init__(self, P, lens, Hkv, d, page=16, fp8=False, layout="head", seed=0, extra_pages=3, spare=2, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.fp8, self.Hkv, self.d = list(lens), page, fp8, Hkv, d
        pages = [-(-n // page) for n in lens]
        self.num = sum(pages) + extra_pages
        ids = torch.randperm(self.num, generator=g)
        self.table = torch.full((len(lens), max(pages + [0]) + spare), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = ids[at:at + n].int()
            at += n
        dt = E4M3 if fp8 else torch.bfloat16
        self.ke = self.ve = None
        if layout == "head":
            self.kc, self.vc, self.ke, self.ve = P.empty_cache(self.num, page, Hkv, d, dtype=dt)
        else:  # token-major, with a gap between tokens
            pad = 16
            self.kc = torch.empty(self.num, page, Hkv, d + pad, dtype=dt, device="cuda")[..., :d]
            self.vc = torch.empty(self.num, page, Hkv + 1, d, dtype=dt, device="cuda")[:, :, 1:]
            if fp8:
                self.ke = torch.empty(self.num, page, Hkv, dtype=torch.uint8, device="cuda")
                self.ve = torch.empty(self.num, page, Hkv, 2, dtype=torch.uint8, device="cuda")[..., 1]
        for c in (self.kc, self.vc):
            c.view(torch.uint8).fill_(0x7F) if fp8 else c.fill_(float("nan"))
        if fp8:
            self.ke.fill_(255)
            self.ve.fill_(255)
        self.K, self.V = [], []  # float64 rows of each sequence
        for b, n in enumerate(lens):
            rows = []
            for c, e in ((self.kc, self.ke), (self.vc, self.ve)):
                x = (torch.randn(n, Hkv, d, generator=g) * scale * torch.exp(torch.randn(n, Hkv, 1, generator=g))).bfloat16()
                pos = torch.arange(n)
                pg, sl = self.table[b, pos // page].long().cuda(), (pos % page).cuda()
                if fp8:
                    code, byte = orc.quantise(_np(x))
                    c.view(torch.uint8)[pg, sl] = torch.from_numpy(code).cuda()
                    e[pg, sl] = torch.from_numpy(byte).cuda()
                    rows.append(orc.dequantise(code, byte))
                else:
                    c[pg, sl] = x.cuda()
                    rows.append(_np(x))
            self.K.append(rows[0])
            self.V.append(rows[1])
        self.table = self.table.cuda()
        self.k_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.at = (self.kc, self.vc, self.table, self.k_lens)
        self.ex = dict(k_exp=self.ke, v_exp=self.ve)


def _cu(ns):
    return torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device="cuda")


def _queries(T, Hq, d, seed=1, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, Hq, d, generator=g) * gain).bfloat16().cuda()


def _check_attention(s, q, news, out, lse, causal=True, window=0, sinks=0, scale=None):
    d = s.d
    scale = d ** -0.5 if scale is None else scale
    f16 = s.fp8 and max(news) * (q.shape[1] // s.Hkv) <= 16
    at, worst = 0, 0.0
    out, lse, q = _np(out), _np(lse), _np(q)
    for b, n in enumerate(news):
        ref, rl, A, D = orc.attend(q[at:at + n], s.K[b], s.V[b], scale, causal, window, sinks)
        w = 2.0 ** -22 * (8 + d * D)[..., None]
        tol = 2.0 ** -8 * np.abs(ref) + ((2.0 ** -11 if f16 else 2.0 ** -8) + 2 * w) * A + 1e-30
        err = np.abs(out[at:at + n] - ref)
        assert np.isfinite(out[at:at + n]).all()
        assert (err <= tol).all(), (b, (err / tol).max())
        got = lse[:, at:at + n].T
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(got), empty)
        assert (np.abs(got[~empty] - rl[~empty]) <= (w[..., 0] + 2.0 ** -22 * np.abs(rl))[~empty]).all()
        if n:
            worst = max(worst, float((err / tol).max()))
        at += n
    return worst


# ------------------------------------------------------------------------------------------------ append, gather
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,Hkv,d,layout", [(16, 8, 128, "head"), (64, 1, 64, "token"), (32, 5, 96, "token"),
                                               (16, 3, 16, "head"), (4096, 2, 128, "head")])
def test_append_writes_its_slots_and_nothing_else(P, fp8, page, Hkv, d, layout):
    news, olds = [1, 0, 37, 16, 3], [0, 5, 20, 15, 130]
    s = Setup(P, [n + o for n, o in zip(news, olds)], Hkv, d, page, fp8, layout, seed=page + d)
    T = sum(news)
    g = torch.Generator().manual_seed(5)
    # rows of very different sizes, a zero row, strided inputs, two rows behind the last sequence
    k = (torch.randn(T + 2, Hkv, 2, d, generator=g) * torch.exp(12 * torch.randn(T + 2, Hkv, 2, 1, generator=g))).bfloat16()
    k[3] = 0
    k = k.cuda()
    k, v = k[:, :, 0], k[:, :, 1]
    before = [x.clone() for x in (s.kc.view(torch.uint8) if fp8 else s.kc, s.vc.view(torch.uint8) if fp8 else s.vc)]
    eb = [x.clone() for x in (s.ke, s.ve)] if fp8 else []
    P.kv_append(k, v, *s.at, _cu(news), **s.ex)
    at = 0
    for b, n in enumerate(news):
        pos = torch.arange(olds[b], olds[b] + n)
        pg, sl = s.table[b, pos // page].long(), pos.cuda() % page
        for i, x in enumerate((k, v)):
            rows = x[at:at + n]
            if fp8:
                code, byte = orc.quantise(_np(rows))
                before[i][pg, sl] = torch.from_numpy(code).cuda()
                eb[i][pg, sl] = torch.from_numpy(byte).cuda()
            else:
                before[i][pg, sl] = rows
        at += n
    for i, (c, e) in enumerate(((s.kc, s.ke), (s.vc, s.ve))):
        if fp8:
            assert torch.equal(c.view(torch.uint8), before[i]) and torch.equal(e, eb[i])
        else:
            assert torch.equal(c.view(torch.int16), before[i].view(torch.int16))


def test_append_e4m3_extremes(P):
    """Infinities saturate, NaN stays, rows at both ends of the range, and every rounding tie."""
    d = 128
    x = torch.zeros(8, 1, d)
    x[0, 0, :3] = torch.tensor([float("inf"), -float("inf"), 3.0])
    x[1, 0, :2] = torch.tensor([float("nan"), 1.0])
    x[2] = 3.3895313892515355e38
    x[3] = 2.0 ** -130
    x[4, 0] = torch.arange(128) + 128.0  # 128 .. 255: ties of three mantissa bits
    x[5, 0] = 448 * torch.ones(d)
    x[6, 0] = 450 * torch.ones(d)
    x[7, 0, 5] = -2.0 ** -140
    x = x.bfloat16().cuda()
    s = Setup(P, [8], 1, d, 16, True)
    P.kv_append(x, x, *s.at, _cu([8]), **s.ex)
    code, byte = orc.quantise(_np(x))
    pg = int(s.table[0, 0])
    assert np.array_equal(s.kc.view(torch.uint8)[pg, :8].cpu().numpy(), code)
    assert np.array_equal(s.ve[pg, :8].cpu().numpy(), byte)
    kk, vv = P.kv_gather(*s.at, _cu([8]), 8, **s.ex)
    want = torch.tensor(orc.dequantise(code, byte)).bfloat16()
    assert torch.equal(torch.nan_to_num(kk.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))
    assert torch.isnan(vv[1, 0, 0]) and torch.isfinite(vv[2]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,Hkv,d,layout", [(16, 8, 128, "token"), (64, 2, 64, "head"), (128, 3, 112, "token")])
def test_gather_reads_ragged_and_padded(P, fp8, page, Hkv, d, layout):
    lens = [1, 300, 0, 64, 65]
    s = Setup(P, lens, Hkv, d, page, fp8, layout, seed=3)
    k, v = P.kv_gather(*s.at, _cu(lens), sum(lens), **s.ex)
    assert np.array_equal(_np(k), np.concatenate(s.K)) and np.array_equal(_np(v), np.concatenate(s.V))
    # padded to 128 rows from an offset, with rows behind the last sequence
    N, first = 128, torch.tensor([0, 250, 3, -2, 60], dtype=torch.int32, device="cuda")
    cu = torch.arange(6, dtype=torch.int32, device="cuda") * N
    ko = torch.full((5 * N + 3, Hkv, d), 9.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    P.kv_gather(*s.at, cu, 5 * N + 3, first=first, k_out=ko, v_out=vo, **s.ex)
    for out, rows in ((ko, s.K), (vo, s.V)):
        want = np.zeros((5, N, Hkv, d))
        for b, f in enumerate(first.tolist()):
            for i in range(N):
                if 0 <= f + i < lens[b]:
                    want[b, i] = rows[b][f + i]
        assert np.array_equal(_np(out[:5 * N]).reshape(want.shape), want)
        assert (out[5 * N:] == 9).all()


@pytest.mark.parametrize("B", [1, 31, 32, 33, 1024, 2500])
def test_tokens_find_their_sequence_in_any_batch(P, B):
    g = np.random.default_rng(B)
    lens = g.integers(0, 4, B).tolist()
    lens[-1] = 2
    s = Setup(P, lens, 1, 16, 16, False, seed=B)
    k, v = P.kv_gather(*s.at, _cu(lens), sum(lens), **s.ex)
    assert np.array_equal(_np(k), np.concatenate(s.K)) and np.array_equal(_np(v), np.concatenate(s.V))


# ------------------------------------------------------------------------------------------------ attention
CASES = [
    # news, lens, Hq, Hkv, d, page, layout, window, sinks, causal
    ([1], [1], 1, 1, 64, 16, "head", 0, 0, True),
    ([1], [257], 2, 1, 64, 16, "head", 0, 0, True),
    ([1, 1, 1, 1], [15, 16, 17, 1000], 8, 2, 128, 16, "token", 0, 0, True),
    ([1, 1], [5000, 3], 16, 1, 128, 64, "head", 0, 0, True),
    ([1, 0, 1], [128, 77, 129], 6, 2, 96, 32, "token", 0, 0, True),
    ([1, 1], [700, 131], 5, 1, 112, 128, "head", 100, 0, True),
    ([1, 1, 1], [700, 90, 2100], 4, 4, 128, 16, "head", 64, 5, True),
    ([1, 1], [900, 400], 8, 8, 64, 256, "token", 300, 131, True),
    ([2, 5, 1], [40, 900, 300], 32, 8, 128, 16, "head", 0, 0, True),
    ([4, 4], [4, 260], 8, 1, 128, 64, "token", 0, 0, True),
    ([3, 8], [500, 333], 4, 1, 80, 16, "head", 33, 2, True),
    ([2, 3], [200, 129], 12, 4, 64, 16, "head", 0, 0, False),
    ([17, 1, 0, 40], [17, 2000, 5, 300], 4, 2, 128, 16, "head", 0, 0, True),
    ([130], [130], 3, 1, 128, 64, "token", 0, 0, True),
    ([200, 33], [1500, 33], 4, 1, 64, 32, "head", 0, 0, True),
    ([150], [1100], 6, 2, 96, 16, "token", 70, 3, True),
    ([300], [900], 2, 2, 128, 128, "head", 129, 130, True),
    ([100, 60], [350, 60], 4, 2, 128, 16, "head", 0, 0, False),
    ([5, 70], [3, 20], 4, 1, 128, 16, "head", 0, 0, True),  # more new tokens than keys: the first rows see none
    ([70, 1], [0, 0], 2, 1, 64, 16, "head", 0, 0, True),  # no keys at all
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention_matches_the_oracle(P, case, fp8):
    news, lens, Hq, Hkv, d, page, layout, window, sinks, causal = case
    s = Setup(P, lens, Hkv, d, page, fp8, layout, seed=sum(lens) + d)
    q = _queries(sum(news), Hq, d)
    out, lse = P.fwd(q, *s.at, _cu(news), max(news), window=window, sinks=sinks, causal=causal, **s.ex)
    _check_attention(s, q, news, out, lse, causal, window, sinks)


@pytest.mark.parametrize("seed", range(int(os.environ.get("FDMA_PAGED_FUZZ", "30"))))
def test_random_batches_match_the_oracle(P, seed):
    """Seeded draws over batch, lengths, heads, head dims, page sizes, layouts, types, windows and sinks:
    the rows are read back, then attended to (FDMA_PAGED_FUZZ=n draws n batches)."""
    g = np.random.default_rng(1000 + seed)
    fp8 = bool(g.integers(2))
    B, Hkv = int(g.integers(1, 6)), int(g.choice([1, 2, 3, 5]))
    G = int(g.choice([1, 2, 3, 4, 7, 8, 13]))
    d = int(g.choice([16, 32, 48, 64, 80, 96, 112, 128, 128])) if fp8 else int(g.choice([8, 24, 64, 72, 104, 120, 128, 128]))
    page, layout = int(g.choice([16, 32, 64, 128, 512])), str(g.choice(["head", "token"]))
    if layout == "token" and d % 16:
        d += 8
    most = int(g.choice([1, 1, 4, 20, 90, 300]))
    news = [int(n) for n in g.integers(0, most + 1, B)]
    news[int(g.integers(B))] = most
    lens = [int(n + k) for n, k in zip(news, g.integers(0, int(g.choice([1, 40, 300, 1500])), B))]
    causal = bool(g.random() < 0.85)
    window = int(g.integers(1, 400)) if causal and g.random() < 0.5 else 0
    sinks = int(g.choice([0, 1, 5, 130, 200]))
    s = Setup(P, lens, Hkv, d, page, fp8, layout, seed=seed)
    k, v = P.kv_gather(*s.at, _cu(lens), sum(lens), **s.ex)
    assert np.array_equal(_np(k), np.concatenate(s.K)) and np.array_equal(_np(v), np.concatenate(s.V))
    q = _queries(sum(news), Hkv * G, d, seed)
    out, lse = P.fwd(q, *s.at, _cu(news), most, window=window, sinks=sinks, causal=causal, **s.ex)
    _check_attention(s, q, news, out, lse, causal, window, sinks)


# ------------------------------------------------------------------------------------------------ masked values
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("news,lens,Hq,Hkv,window,sinks", [
    ([5], [300], 4, 1, 0, 0), ([3, 6], [40, 257], 8, 4, 20, 4), ([200, 70], [700, 70], 4, 2, 0, 0),
    ([260], [900], 2, 1, 100, 7), ([40], [129], 4, 1, 0, 0)])
def test_values_of_unseen_keys_reach_no_row(P, fp8, news, lens, Hq, Hkv, window, sinks):
    """NaN and infinities in K and V of keys that only some rows of a chunk see: the rows that do not see
    them are as if they were not there, the rows that do get what they make of the sum."""
    d, page = 128, 16
    s = Setup(P, lens, Hkv, d, page, fp8, seed=11)
    q = _queries(sum(news), Hq, d)
    kw = dict(window=window, sinks=sinks, **s.ex)
    cu = _cu(news)
    clean, clean_lse = P.fwd(q, *s.at, cu, max(news), **kw)
    at = 0
    for b, n in enumerate(news):
        # the last new token's V (seen by one row only), one in the middle, and one at the window's lower edge
        nk = lens[b]
        spots = {nk - 1, nk - 1 - n // 2}
        if window and nk - n - window // 2 >= sinks:
            spots.add(max(nk - n - window + 1 + n // 2, sinks))
        for x, j in enumerate(sorted(spots)):
            pg, sl = int(s.table[b, j // page]), j % page
            if fp8:
                s.vc.view(torch.uint8)[pg, sl, :, 5 + x] = 0x7F
            else:
                s.vc[pg, sl, :, 5 + x] = float("nan") if x % 2 else float("inf")
        out, lse = P.fwd(q, *s.at, cu, max(news), **kw)
        assert torch.equal(lse[:, at:at + n], clean_lse[:, at:at + n])
        for i in range(n):
            keep = orc.visible(nk - n + i, nk, True, window, sinks)
            row, ref = out[at + i].float(), clean[at + i].float()
            for x, j in enumerate(sorted(spots)):
                c = 5 + x
                if keep[j]:
                    bad = ~torch.isfinite(row[:, c])
                    assert bad.all()
                    if not fp8 and x % 2 == 0:
                        # (a weight below 2^-126 is 0 in fp32, and 0 * inf is NaN: looked at down to 2^-100)
                        for h in range(Hq):
                            sc = d ** -0.5 * float(s.K[b][j, h // (Hq // Hkv)] @ _np(q[at + i, h]))
                            if sc - float(clean_lse[h, at + i]) > -100 * np.log(2):
                                assert row[h, c] == float("inf")
                else:
                    assert torch.isfinite(row[:, c]).all()
            cols = [c for c in range(d) if c - 5 not in range(len(spots))]
            # (a run may be cut elsewhere for nothing else: the sums are the same ones)
            assert torch.equal(row[:, cols], ref[:, cols])
        at += n
        # K: a NaN in the last key reaches the last row alone
        pg, sl = int(s.table[b, (nk - 1) // page]), (nk - 1) % page
        if fp8:
            s.kc.view(torch.uint8)[pg, sl, :, 3] = 0x7F
        else:
            s.kc[pg, sl, :, 3] = float("nan")
        out, lse = P.fwd(q, *s.at, cu, max(news), **kw)
        if n > 1:
            assert torch.isfinite(lse[:, at - n:at - 1]).all()
            cols = [c for c in range(d) if c > 9]
            assert torch.equal(out[at - n:at - 1, :, cols], clean[at - n:at - 1, :, cols])
        assert torch.isnan(lse[:, at - 1]).all() and torch.isnan(out[at - 1]).all()
        clean, clean_lse = out, lse  # the next sequence's rows have not changed


def test_rows_of_lowest_and_largest_scores(P):
    """Scores of +-1e4 and a chunk whose first tiles are far below its last: the running maximum holds."""
    s = Setup(P, [600, 600], 1, 64, 16, False, seed=4, scale=6.0)
    q = _queries(2 * 40, 4, 64, gain=20.0)
    for news in ([40, 40], [1, 2]):
        T = sum(news)
        out, lse = P.fwd(q[:T], *s.at, _cu(news), max(news), scale=1.0)
        _check_attention(s, q[:T], news, out, lse, scale=1.0)
    out, lse = P.fwd(q[:3], *s.at, _cu([1, 2]), 2, scale=1e-30)
    _check_attention(s, q[:3], [1, 2], out, lse, scale=1e-30)
    out, lse = P.fwd(q, *s.at, _cu([40, 40]), 40, scale=1e-30)
    _check_attention(s, q, [40, 40], out, lse, scale=1e-30)


def test_e4m3_scales_from_end_to_end(P):
    """Rows whose scale bytes span the range: tiny, huge and zero rows in one sequence."""
    d, n = 128, 200
    g = torch.Generator().manual_seed(8)
    s = Setup(P, [n], 2, d, 16, True, seed=2)
    x = torch.randn(n, 2, d, generator=g)
    k = (x * torch.exp2(torch.randint(-8, 2, (n, 2, 1), generator=g).float())).bfloat16()
    v = (torch.randn(n, 2, d, generator=g) * torch.exp2(torch.randint(-10, 3, (n, 2, 1), generator=g).float())).bfloat16()
    v[7] = 0
    k[9] = 0
    P.kv_append(k.cuda(), v.cuda(), *s.at, _cu([n]), **s.ex)
    s.K = [orc.dequantise(*orc.quantise(_np(k)))]
    s.V = [orc.dequantise(*orc.quantise(_np(v)))]
    for new in (1, 5, 60):
        q = _queries(new, 8, d, seed=new)
        out, lse = P.fwd(q, *s.at, _cu([new]), new, **s.ex)
        _check_attention(s, q, [new], out, lse)
    # all values a factor 2^100 larger: the same sums, scaled
    big = Setup(P, [n], 2, d, 16, True, seed=2)
    big.kc.view(torch.uint8).copy_(s.kc.view(torch.uint8)), big.vc.view(torch.uint8).copy_(s.vc.view(torch.uint8))
    big.ke.copy_(s.ke)
    big.ve.copy_(torch.where(s.ve == 255, s.ve, s.ve + 90))
    big.table.copy_(s.table)
    for new in (1, 60):
        q = _queries(new, 8, d, seed=new)
        a, b = P.fwd(q, *s.at, _cu([new]), new, **s.ex), P.fwd(q, *big.at, _cu([new]), new, **big.ex)
        assert torch.equal(a[1], b[1]) and torch.equal(torch.ldexp(a[0].float(), torch.tensor(90)), b[0].float())


# ------------------------------------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_then_decode_like_one_long_call(P, fp8):
    """A prompt in two chunks and then single tokens, every step written to the cache first: the rows are those
    of attention over the whole sequence at once (the float64 oracle on what the cache holds)."""
    Hq, Hkv, d, page, total = 8, 2, 128, 16, 150
    steps = [90, 57] + [1] * 3
    g = torch.Generator().manual_seed(1)
    k, v = ((torch.randn(2, total + 11 * b, Hkv, d, generator=g)).bfloat16() for b in (0, 0))
    kc, vc, ke, ve = P.empty_cache(32, page, Hkv, d, dtype=E4M3 if fp8 else torch.bfloat16)
    ex = dict(k_exp=ke, v_exp=ve)
    table = torch.randperm(32, generator=g)[:24].view(2, 12).int().cuda()
    q = torch.randn(2, total, Hq, d, generator=g).bfloat16()
    outs, done = [], 0
    for n in steps:
        # the second sequence is a token behind until the last step
        lens = torch.tensor([done + n, done + n], dtype=torch.int32, device="cuda")
        cu = _cu([n, n])
        pack = lambda t: torch.cat([t[0, done:done + n], t[1, done:done + n]]).cuda()  # noqa: E731
        P.kv_append(pack(k), pack(v), kc, vc, table, lens, cu, **ex)
        outs.append(P.fwd(pack(q), kc, vc, table, lens, cu, n, window=64, sinks=3, **ex))
        done += n
    for b in range(2):
        K, V = (_np(t[b]) for t in (k, v))
        if fp8:
            K, V = (orc.dequantise(*orc.quantise(t)) for t in (K, V))
        ref, rl, A, D = orc.attend(_np(q[b]), K, V, d ** -0.5, True, 64, 3)
        got = torch.cat([o[0][n * b:n * (b + 1)] for (o, n) in zip(outs, steps)])
        w = 2.0 ** -22 * (8 + d * D)[..., None]
        assert (np.abs(_np(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * w) * A + 1e-30).all()
        gl = torch.cat([o[1][:, n * b:n * (b + 1)] for (o, n) in zip(outs, steps)], 1)
        assert (np.abs(_np(gl).T - rl) <= w[..., 0] + 2.0 ** -22 * np.abs(rl)).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_gathered_keys_feed_the_masked_forward(P, fp8):
    """kv_gather's padded rows through fdma.fwd (the masked, biased path) give the paged forward's rows."""
    from block_sparse_masked_02_gb300 import fdma

    lens, new, Hq, Hkv, d, N = [300, 384], 128, 4, 2, 128, 384
    s = Setup(P, lens, Hkv, d, 64, fp8, seed=9)
    q = _queries(2 * new, Hq, d)
    out, lse = P.fwd(q, *s.at, _cu([new, new]), new, **s.ex)
    cu = torch.tensor([0, N, 2 * N], dtype=torch.int32, device="cuda")
    k, v = P.kv_gather(*s.at, cu, 2 * N, **s.ex)
    k, v = k.view(2, N, Hkv, d), v.view(2, N, Hkv, d)
    for b in range(2):
        o, z = fdma.fwd(q.view(2, new, Hq, d)[b:b + 1], k[b:b + 1], v[b:b + 1], causal_offset=lens[b] - new)
        # both round the weights to bf16 and the result to bf16; fdma's lse carries the rounded weights (1.95e-3)
        assert float((o[0].float() - out[b * new:(b + 1) * new].float()).norm() / o[0].float().norm()) < 2.0 ** -7
        assert float((z[0] - lse[:, b * new:(b + 1) * new]).abs().max()) < 4e-3


def test_rows_behind_the_last_sequence_and_given_outputs(P):
    s = Setup(P, [40, 500], 2, 64, 16, False, seed=6)
    for news in ([1, 1], [3, 70]):
        T = sum(news)
        q = _queries(T + 5, 4, 64)
        q[T:] = float("nan")
        out = torch.full((T + 5, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, T + 5), 3.0, device="cuda")
        a = P.make_args(q, *s.at, _cu(news), max(news) + 9)
        ws = P.alloc_workspace(a, "cuda")
        ws.fill_(255)
        o, z = P.fwd(q, *s.at, _cu(news), max(news) + 9, out=out, lse=lse, workspace=ws)
        assert o is out and z is lse
        assert (out[T:] == 3).all() and (lse[:, T:] == 3).all()
        _check_attention(s, q[:T], news, out[:T], lse[:, :T])


def test_strided_queries_and_wide_batches(P):
    """Queries as a slice of a fused projection; 200 sequences of 0 to 40 keys (more than SMs and than a warp)."""
    g = np.random.default_rng(3)
    lens = g.integers(0, 41, 200).tolist()
    s = Setup(P, lens, 2, 64, 16, False, seed=5)
    for news in ([min(1, n) for n in lens], [min(n, 17) for n in lens]):
        T = sum(news)
        big = torch.randn(T, 3, 6, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
        q = big[:, 1, 1:5]
        out, lse = P.fwd(q, *s.at, _cu(news), max(news))
        _check_attention(s, q, news, out, lse)


def test_repeats_bit_for_bit(P):
    s = Setup(P, [3000, 70, 900], 2, 128, 16, True, seed=7)
    for news in ([1, 1, 1], [300, 70, 5]):
        q = _queries(sum(news), 8, 128)
        a = P.fwd(q, *s.at, _cu(news), max(news), **s.ex)
        for _ in range(5):
            b = P.fwd(q, *s.at, _cu(news), max(news), **s.ex)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_step_replays_from_a_cuda_graph(P, fp8):
    """A decoding step (append, attention) captured once: replays follow the lengths, pages, offsets and
    tokens that change in place."""
    Hq, Hkv, d, page = 8, 2, 128, 16
    s = Setup(P, [200, 31], Hkv, d, page, fp8, seed=3, extra_pages=10)
    s.table[:, -2:] = torch.tensor([[s.num - 1, s.num - 2]], dtype=torch.int32).cuda()  # (not used by any sequence)
    used = set(s.table[0, :13].tolist() + s.table[1, :2].tolist())
    free = [i for i in range(s.num) if i not in used]
    s.table[0, 13], s.table[1, 2] = free[0], free[1]
    k, v, q = (torch.randn(2, h, d, device="cuda").bfloat16() for h in (Hkv, Hkv, Hq))
    cu = _cu([1, 1])
    out, lse = torch.empty_like(q), torch.empty(Hq, 2, device="cuda")

    def step():
        P.kv_append(k, v, *s.at, cu, **s.ex)
        P.fwd(q, *s.at, cu, 1, out=out, lse=lse, **s.ex)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(12):  # crosses into a new page
        s.k_lens += 1
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).bfloat16())
        graph.replay()
        got = out.clone(), lse.clone()
        step()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    K, V = P.kv_gather(*s.at, _cu(s.k_lens.tolist()), int(s.k_lens.sum()), **s.ex)
    n = int(s.k_lens[0])
    s.K, s.V = ([_np(t[:n]), _np(t[n:])] for t in (K, V))
    _check_attention(s, q, [1, 1], out, lse)


def test_two_streams_at_once(P):
    """Calls on two side streams, outputs and workspaces allocated by the calls, inputs ready."""
    s = Setup(P, [2000, 900], 2, 128, 16, False, seed=8)
    cases = [([1, 1], _queries(2, 8, 128, 1)), ([200, 33], _queries(233, 8, 128, 2))]
    want = [P.fwd(q, *s.at, _cu(n), max(n)) for n, q in cases]
    cus = [_cu(n) for n, _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, (n, q) in enumerate(cases):
            got[i].append(P.fwd(q, *s.at, cus[i], max(n), stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, z in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(z, want[i][1])


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(P, fp8):
    """A cache of more than 2^32 bytes a tensor whose used pages lie at its end."""
    Hkv, d, page = 8, 128, 64
    per = page * Hkv * d * (1 if fp8 else 2)
    num = (1 << 32) // per + 70
    kc, vc, ke, ve = P.empty_cache(num, page, Hkv, d, dtype=E4M3 if fp8 else torch.bfloat16)
    ex = dict(k_exp=ke, v_exp=ve)
    n = 300
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(n, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.tensor([[num - 1, 0, num - 3, num - 2, num - 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    at = (kc, vc, table, lens)
    P.kv_append(k, v, *at, _cu([n]), **ex)
    kk, vv = P.kv_gather(*at, _cu([n]), n, **ex)
    if fp8:
        K, V = (orc.dequantise(*orc.quantise(_np(t))) for t in (k, v))
        assert np.array_equal(_np(kk), K) and np.array_equal(_np(vv), V)
    else:
        assert torch.equal(kk, k) and torch.equal(vv, v)
    s = Setup.__new__(Setup)
    s.d, s.Hkv, s.fp8, s.K, s.V = d, Hkv, fp8, [_np(kk)], [_np(vv)]
    for new in (1, 64):
        q = _queries(new, Hkv * 2, d)
        out, lse = P.fwd(q, *at, _cu([new]), new, **ex)
        _check_attention(s, q, [new], out, lse)


def test_broadcast_heads_of_a_cache(P):
    """kv heads that share one row (stride 0): read like any other cache, refused as a target."""
    s = Setup(P, [500], 1, 64, 16, False, seed=3)
    kc, vc = s.kc.expand(-1, -1, 4, -1), s.vc.expand(-1, -1, 4, -1)
    at = (kc, vc, s.table, s.k_lens)
    t = Setup.__new__(Setup)
    t.d, t.Hkv, t.fp8 = 64, 4, False
    t.K, t.V = [np.repeat(s.K[0], 4, 1)], [np.repeat(s.V[0], 4, 1)]
    for new in (1, 100):
        q = _queries(new, 8, 64)
        out, lse = P.fwd(q, *at, _cu([new]), new)
        _check_attention(t, q, [new], out, lse)
    k = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    from block_sparse_masked_02_gb300 import fdma

    with pytest.raises(fdma.FdmaError):
        P.kv_append(k, k, *at, _cu([1]))


@pytest.mark.parametrize("d", [64, 80, 128])
def test_broadcast_heads_of_an_e4m3_cache(P, d):
    """Rows and scale bytes that kv heads share (stride 0), for single tokens and chunks of one and two slots of rows."""
    s = Setup(P, [500, 77], 1, d, 16, True, seed=4)
    heads = lambda x: x.expand(*x.shape[:2], 4, *x.shape[3:])
    t = Setup.__new__(Setup)
    t.d, t.Hkv, t.fp8 = d, 4, True
    t.K, t.V = [np.repeat(x, 4, 1) for x in s.K], [np.repeat(x, 4, 1) for x in s.V]
    for news in ([1, 1], [30, 7], [150, 77]):
        q = _queries(sum(news), 8, d)
        out, lse = P.fwd(q, heads(s.kc), heads(s.vc), s.table, s.k_lens, _cu(news), max(news), k_exp=heads(s.ke),
                         v_exp=heads(s.ve))
        _check_attention(t, q, news, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 100])
def test_keys_of_a_page_that_is_not_there_read_as_zeros(P, fp8, window):
    from block_sparse_masked_02_gb300 import fdma

    s = Setup(P, [600, 333], 2, 128, 16, fp8, seed=6)
    table = s.table.clone()
    table[0, 3], table[0, 36], table[1, 20] = -1, s.num, 1 << 30
    for b, pages in ((0, (3, 36)), (1, (20,))):
        for x in pages:
            s.K[b][16 * x:16 * x + 16] = 0
            s.V[b][16 * x:16 * x + 16] = 0
    for news in ([1, 1], [5, 20], [40, 333]):
        q = _queries(sum(news), 8, 128)
        out, lse = P.fwd(q, s.kc, s.vc, table, s.k_lens, _cu(news), max(news), window=window, sinks=9 if window else 0, **s.ex)
        assert fdma.device_error() == fdma.FDMA_ERR_INVALID
        _check_attention(s, q, news, out, lse, window=window, sinks=9 if window else 0)


# ------------------------------------------------------------------------------------------------ refusals
def test_bad_device_arrays_are_reported_and_not_followed(P):
    """Page numbers, lengths and offsets out of range: nothing is read or written there, the rest is right,
    and the device error says so."""
    from block_sparse_masked_02_gb300 import fdma

    s = Setup(P, [40, 200], 2, 64, 16, False, seed=1)
    bad = s.table.clone()
    bad[0, 1] = s.num  # one past the last page
    at = (s.kc, s.vc, bad, s.k_lens)
    kk, _ = P.kv_gather(*at, _cu([40, 200]), 240)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    want = np.concatenate([s.K[0], s.K[1]])
    want[16:32] = 0
    assert np.array_equal(_np(kk), want)
    for news in ([1, 1], [30, 100]):
        q = _queries(sum(news), 4, 64)
        out, lse = P.fwd(q, *at, _cu(news), max(news))
        assert fdma.device_error() == fdma.FDMA_ERR_INVALID
        assert torch.isfinite(out).all()
        ref, rl = P.fwd(q, *s.at, _cu(news), max(news))
        assert torch.equal(out[news[0]:], ref[news[0]:])  # the other sequence
        # more new tokens than max_q: the rest is left out
        part = torch.full_like(out, 5.0)
        P.fwd(q, *s.at, _cu(news), max(news) - 1 if max(news) > 1 else 1, out=part)
        if max(news) > 1:
            assert fdma.device_error() == fdma.FDMA_ERR_INVALID
            assert (part[-1] == 5).all()
    # a length past the table: keys of the whole table, reported
    far = s.k_lens.clone()
    far[1] = 1 << 30
    full = s.table.clamp(min=0)
    P.fwd(_queries(2, 4, 64), s.kc, s.vc, full, far, _cu([1, 1]), 1)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    P.kv_gather(s.kc, s.vc, full, far, _cu([40, 10]), 50)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    # an append to a position before the first key, past the table, or to a page that is not there
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = s.kc.clone()
    P.kv_append(k, k, s.kc, s.vc, bad, torch.tensor([18, 1], dtype=torch.int32, device="cuda"), _cu([1, 2]))
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    pg = int(s.table[1, 0])
    before[pg, 0] = 1
    assert torch.equal(torch.nan_to_num(s.kc, nan=9.0), torch.nan_to_num(before, nan=9.0))
    # offsets that run backwards or past the tokens
    q = _queries(4, 4, 64)
    cu = torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda")
    P.fwd(q, *s.at, cu, 3)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    cu = torch.tensor([3, 1, 2], dtype=torch.int32, device="cuda")
    P.fwd(q, *s.at, cu, 3)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID


def test_empty_calls_do_nothing(P):
    s = Setup(P, [20], 2, 64, 16, False)
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    P.kv_append(none, none, *s.at, _cu([0]))
    out, lse = P.fwd(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), *s.at, _cu([0]), 0)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    k, v = P.kv_gather(*s.at, _cu([0]), 0)
    assert k.shape == (0, 2, 64)


def test_tensors_of_a_call_are_checked(P):
    from block_sparse_masked_02_gb300 import fdma

    s = Setup(P, [40], 2, 64, 16, False)
    q = _queries(1, 4, 64)
    cu = _cu([1])
    with pytest.raises(ValueError):
        P.fwd(q.float(), *s.at, cu, 1)
    with pytest.raises(ValueError):
        P.fwd(q, s.kc, s.vc, s.table.cpu(), s.k_lens, cu, 1)
    with pytest.raises(ValueError):
        P.fwd(q, s.kc, s.vc, s.table.long(), s.k_lens, cu, 1)
    with pytest.raises(ValueError):
        P.fwd(q, *s.at, _cu([1, 1]), 1)
    with pytest.raises(ValueError):
        P.fwd(q, *s.at, cu, 1, k_exp=torch.zeros(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        P.fwd(q, s.kc.to(E4M3), s.vc.to(E4M3), s.table, s.k_lens, cu, 1)
    with pytest.raises(ValueError):
        P.fwd(q, *s.at, cu, 1, lse=torch.zeros(1, 4, device="cuda"))
    with pytest.raises(fdma.FdmaError):
        P.fwd(q, *s.at, cu, 1, window=8, causal=False)
    with pytest.raises(fdma.FdmaError):
        P.fwd(q, *s.at, cu, 1, scale=float("nan"))
    with pytest.raises(fdma.FdmaError):
        P.fwd(q, *s.at, cu, 1, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------------------------------------ scales far apart
# e4m3 caches, at most 16 rows: a weight is an f16 number in units of the row's largest value scale, so its own error
# is 2^-11 of it or, where it gets subnormal (step 2^-24, scales at most 2^16 apart, the largest unit 2^15), at most
# 2^-25 * 2^-15 * 2^16 = 2^-24.  Rows whose scales lie further apart take weights in fp32.  So the bound above
# grows by 2^-24 sum_j |v_j| / (sum of the weights, which is at least 1).
def _plant_scale(s, b, j, delta, kind):
    """Key j of sequence b with a value scale `delta` powers of two above the sequence's largest."""
    pg, sl = int(s.table[b, j // s.page]), j % s.page
    top = int(np.log2(np.abs(s.V[b]).max() / 448).max()) + 128
    code = s.vc.view(torch.uint8)[pg, sl].clone()
    if kind == "column":  # one value, and seven eighths of the others' columns are its zeros
        code[:, s.d // 8:] = 0
        s.vc.view(torch.uint8)[pg, sl] = code
    if kind == "light":  # far below the others' scores: queries have 8 in column 0
        kcode, kbyte = orc.quantise(np.where(np.arange(s.d) == 0, -8.0 * s.d ** 0.5, s.K[b][j]))
        s.kc.view(torch.uint8)[pg, sl], s.ke[pg, sl] = torch.from_numpy(kcode).cuda(), torch.from_numpy(kbyte).cuda()
        s.K[b][j] = orc.dequantise(kcode, kbyte)
    s.ve[pg, sl] = top + delta
    s.V[b][j] = orc.dequantise(code.cpu().numpy(), np.full(s.Hkv, top + delta))


@pytest.mark.parametrize("delta", [12, 30, 40, 100])
@pytest.mark.parametrize("kind", ["unseen", "light", "column"])
@pytest.mark.parametrize("new,G,d", [(1, 1, 128), (2, 1, 64), (3, 2, 128), (4, 4, 128), (16, 1, 64), (5, 4, 128)])
def test_a_large_value_leaves_the_other_keys_their_weights(P, new, G, d, kind, delta):
    if kind == "unseen" and new == 1:
        pytest.skip("a single token sees every key")
    for n in (20, 300, 3000):
        s = Setup(P, [n], 2, d, 16, True, seed=n + d)
        q = _queries(new, 2 * G, d, seed=delta)
        q[..., 0] = 8
        cu = _cu([new])
        if kind == "light":  # (its score is -64 nats, the others within some of 0)
            s.kc.view(torch.uint8)[..., 0] = 0
            s.K[0][..., 0] = 0
        clean, clean_lse = P.fwd(q, *s.at, cu, new, **s.ex)
        j = n - 1 if kind == "unseen" else n - new - 3
        _plant_scale(s, 0, j, delta, kind)
        out, lse = P.fwd(q, *s.at, cu, new, **s.ex)
        ref, rl, A, D = orc.attend(_np(q), s.K[0], s.V[0], d ** -0.5)
        w = 2.0 ** -22 * (8 + d * D)[..., None]
        others = np.repeat(np.abs(np.delete(s.V[0], j, 0)).sum(0), G, 0)[None]
        u = 2.0 ** -11 if new * G <= 16 else 2.0 ** -8
        tol = 2.0 ** -8 * np.abs(ref) + (u + 2 * w) * A + 2.0 ** -24 * others
        if delta <= 16:
            tol = tol + 2.0 ** -40 * np.repeat(np.abs(s.V[0][j]), G, 0)[None]
        err = np.abs(_np(out) - ref)
        assert (err <= tol).all(), (n, (err / tol).max())
        assert (np.abs(_np(lse).T - rl) <= w[..., 0] + 2.0 ** -22 * np.abs(rl)).all()
        if kind == "unseen":  # the rows that do not see it have not changed
            assert torch.equal(out[:-1], clean[:-1]) and torch.equal(lse[:, :-1], clean_lse[:, :-1])


@pytest.mark.parametrize("order", ["shuffled", "rising", "falling"])
@pytest.mark.parametrize("news,G", [([1], 1), ([2], 4), ([4], 4), ([1, 3], 8), ([6], 4)])
def test_value_scales_over_the_whole_range(P, news, G, order):
    """Scale bytes 20 to 240 in one sequence, each octave of bytes with columns of its own: every column has to
    be right by itself, however small beside the others."""
    d, lens = 128, [700 + 31 * b for b in range(len(news))]
    s = Setup(P, lens, 1, d, 16, True, seed=len(lens))
    g = np.random.default_rng(G)
    for b, n in enumerate(lens):
        byte = np.sort(g.integers(20, 241, n))
        byte = byte[::-1].copy() if order == "falling" else g.permutation(byte) if order == "shuffled" else byte
        code = g.integers(8, 120, (n, 1, d)).astype(np.uint8) | (g.integers(0, 2, (n, 1, d)) << 7).astype(np.uint8)
        band = np.arange(d)[None, None] // 8 == (byte // 16)[:, None, None]
        code = np.where(band, code, 0).astype(np.uint8)
        pos = torch.arange(n)
        pg, sl = s.table[b, (pos // 16).cuda()].long(), (pos % 16).cuda()
        s.vc.view(torch.uint8)[pg, sl] = torch.from_numpy(code).cuda()
        s.ve[pg, sl] = torch.from_numpy(byte[:, None].astype(np.uint8)).cuda()
        s.V[b] = orc.dequantise(code, byte[:, None])
    q = _queries(sum(news), G, d, seed=4)
    out, lse = P.fwd(q, *s.at, _cu(news), max(news), **s.ex)
    out, lse, at = _np(out), _np(lse), 0
    u = 2.0 ** -11 if max(news) * G <= 16 else 2.0 ** -8
    for b, n in enumerate(news):
        ref, rl, A, D = orc.attend(_np(q[at:at + n]), s.K[b], s.V[b], d ** -0.5)
        w = 2.0 ** -22 * (8 + d * D)[..., None]
        # 2^-130: bf16's least step is 2^-133, fp32's 2^-149.  The f16 term of above: a warp whose keys' scales are at most
        # 2^16 apart has f16 weights; beside a largest unit of 2^15 key j's is 2^(15 - x), x <= 16, half a step of a
        # subnormal f16 2^-25, so w_j is off by at most 2^-25 / 2^(15 - x) = 2^(x - 40) <= 2^-24.  Some heads' weights
        # of a whole band are below that (2^-36 of the row's largest), and only keys of the band have the column.
        tol = 2.0 ** -8 * np.abs(ref) + (u + 2 * w) * A + 2.0 ** -130
        if max(news) * G <= 16:
            tol = tol + 2.0 ** -24 * np.abs(s.V[b][:, 0]).sum(0)
        err = np.abs(out[at:at + n] - ref)
        assert (err <= tol).all(), (err / tol).max()
        assert (np.abs(lse[:, at:at + n].T - rl) <= w[..., 0] + 2.0 ** -22 * np.abs(rl)).all()
        at += n


def test_zero_value_rows_do_not_disturb_the_others(P):
    """Rows of zeros (scale byte 1) beside ordinary ones: the same rows as with any other scale byte."""
    s = Setup(P, [500], 2, 128, 16, True, seed=3)
    for j in (0, 33, 250, 499):
        pg, sl = int(s.table[0, j // 16]), j % 16
        s.vc.view(torch.uint8)[pg, sl] = torch.tensor([0, 0x80], dtype=torch.uint8, device="cuda").repeat(64)
        s.ve[pg, sl] = 1
        s.V[0][j] = 0
    for new in (1, 4, 30):
        q = _queries(new, 8, 128, new)
        a = P.fwd(q, *s.at, _cu([new]), new, **s.ex)
        _check_attention(s, q, [new], *a)
        for byte in (110, 20, 240):
            ve = s.ve.clone()
            ve[ve == 1] = byte
            b = P.fwd(q, *s.at, _cu([new]), new, k_exp=s.ke, v_exp=ve)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------------------------------------ parts left out
def _check_kept_rows(s, q, news, keep, out, lse, window=0, sinks=0, f16=False):
    """Rows `keep` (a number for each sequence) of the sequences' first, as with nothing left out; the others as they were (5)."""
    at = 0
    for b, n in enumerate(news):
        ref, rl, A, D = orc.attend(_np(q[at:at + n]), s.K[b], s.V[b], s.d ** -0.5, True, window, sinks)
        m = keep[b]
        w = 2.0 ** -22 * (8 + s.d * D)[..., None]
        tol = (2.0 ** -8 * np.abs(ref) + ((2.0 ** -11 if f16 else 2.0 ** -8) + 2 * w) * A + 1e-30)[:m]
        o, z = _np(out[at:at + n]), _np(lse[:, at:at + n]).T
        assert (np.abs(o[:m] - ref[:m]) <= tol).all(), (b, (np.abs(o[:m] - ref[:m]) / tol).max())
        assert (np.abs(z[:m] - rl[:m]) <= w[:m, :, 0] + 2.0 ** -22 * np.abs(rl[:m])).all()
        assert (o[m:] == 5).all() and (z[m:] == 5).all()
        at += n


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 4)])
@pytest.mark.parametrize("max_q", [1, 4, 20, 150])
def test_rows_past_max_q_are_left_out_and_the_others_keep_their_positions(P, fp8, window, sinks, max_q):
    from block_sparse_masked_02_gb300 import fdma

    news, lens = [6, 1, 200], [50, 77, 500]
    s = Setup(P, lens, 2, 64, 16, fp8, seed=5)
    T = sum(news)
    q = _queries(T, 4, 64)
    out, lse = torch.full((T, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, T), 5.0, device="cuda")
    P.fwd(q, *s.at, _cu(news), max_q, window=window, sinks=sinks, out=out, lse=lse, **s.ex)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    _check_kept_rows(s, q, news, [min(n, max_q) for n in news], out, lse, window, sinks, fp8 and 2 * max_q <= 16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("news", [[3, 4], [30, 100]])
def test_tokens_behind_the_packed_axis_are_left_out(P, fp8, news):
    """cu_q[B] past T by two: the last two tokens are not there, the others keep their positions."""
    from block_sparse_masked_02_gb300 import fdma

    s = Setup(P, [40, 300], 2, 128, 16, fp8, seed=6)
    T = sum(news)
    q = _queries(T, 4, 128)
    out, lse = torch.full((T, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, T), 5.0, device="cuda")
    short, z = out[:T - 2], torch.full((4, T - 2), 5.0, device="cuda")
    P.fwd(q[:T - 2], *s.at, _cu(news), max(news), out=short, lse=z, **s.ex)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    lse[:, :T - 2] = z
    _check_kept_rows(s, q, news, [news[0], news[1] - 2], out, lse, f16=fp8 and max(news) * 2 <= 16)
    # ranges that begin before the first token: those tokens are left out
    cu = _cu(news) - 2
    P.fwd(q[:T - 2], *s.at, cu, max(news), out=short, lse=z, **s.ex)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    full = torch.cat([q[:2], q[:T - 2]])
    o = torch.cat([torch.zeros_like(out[:2]), short])
    for b, (a, n) in enumerate(((2, news[0] - 2), (news[0], news[1]))):
        ref, _, A, D = orc.attend(_np(full[a + n - news[b]:a + n]), s.K[b], s.V[b], 128 ** -0.5)
        w = 2.0 ** -22 * (8 + 128 * D)[..., None]
        err = np.abs(_np(o[a:a + n]) - ref[-n:])
        assert (err <= (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * w) * A + 1e-30)[-n:]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("news", [[3, 4, 2], [30, 100, 1]])
@pytest.mark.parametrize("bad", [-1, -(1 << 31), "past", 1 << 30, (1 << 31) - 1])
def test_sequences_with_a_length_out_of_range_are_left_out(P, fp8, news, bad):
    """fwd leaves their rows, append their slots as they were; the others are right."""
    from block_sparse_masked_02_gb300 import fdma

    s = Setup(P, [40, 300, 25], 2, 128, 16, fp8, seed=6, spare=0)
    lens = s.k_lens.clone()
    lens[0] = s.table.shape[1] * 16 + 1 if bad == "past" else bad
    at = (s.kc, s.vc, s.table, lens)
    T = sum(news)
    q = _queries(T, 4, 128)
    out, lse = torch.full((T, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, T), 5.0, device="cuda")
    P.fwd(q, *at, _cu(news), max(news), out=out, lse=lse, **s.ex)
    assert fdma.device_error() == fdma.FDMA_ERR_INVALID
    _check_kept_rows(s, q, news, [0] + news[1:], out, lse, f16=fp8 and max(news) * 2 <= 16)


# ------------------------------------------------------------------------------------------------ division of the work
PLAN_PROBE = r"""
#include "fdma_paged.cuh"
template <int ROWS, int NT>
__global__ void __launch_bounds__(NT) probe(const __grid_constant__ fdma::PagedParams p, int* out) {
  __shared__ fdma::PlanSmem sm;
  fdma::Cursor<ROWS, 128> c;
  int quota = 0;
  const bool any = fdma::plan_run<ROWS, 128, NT>(p, &sm, c, quota);
  if (threadIdx.x == 0) {
    int* o = out + blockIdx.x * 8;
    o[0] = any;
    if (any) o[1] = c.b, o[2] = c.g, o[3] = c.rt, o[4] = c.t, o[5] = c.left, o[6] = quota;
  }
}
extern "C" __attribute__((visibility("default"))) int plan_probe(
    const int* cu, const int* k_len, int B, int Hkv, int G, int T, int max_q, int page_shift, int max_pages, int causal,
    int window, int sinks, int rows, int lanes, int min_run, int* out, int* err) {
  fdma::PagedParams p{};
  p.cu = cu, p.c.k_len = k_len, p.c.B = B, p.c.Hkv = Hkv, p.G = G, p.T = T, p.max_q = max_q, p.c.page_shift = page_shift;
  p.c.max_pages = max_pages, p.causal = causal, p.window = window, p.sinks = sinks, p.plan_lanes = lanes, p.min_run = min_run;
  p.err = err;
  if (rows == 256) probe<256, 512><<<fdma::kPagedCtas, 512>>>(p, out);
  else if (rows == 8) probe<8, 256><<<fdma::kPagedCtas, 256>>>(p, out);
  else return -1;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? static_cast<int>(cudaDeviceSynchronize()) : static_cast<int>(e);
}
"""


@pytest.fixture(scope="module")
def plan_probe(P, tmp_path_factory):
    """The division of the work by itself: what every CTA begins with, without the attention."""
    import ctypes
    import subprocess

    from block_sparse_masked_02_gb300 import build

    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan_probe.cu", d / "plan_probe.so"
    src.write_text(PLAN_PROBE)
    subprocess.run([build._nvcc(), *build.ARCH, *build.CFLAGS, "-I", build.CSRC, "-shared", str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib)).plan_probe


def _line(news, lens, G, Hkv, causal, window, sinks, rows):
    """Key tiles of every item, (sequence, kv head, row block) in order, as (sequence, tiles of each block)."""
    for b, (n, kl) in enumerate(zip(news, lens)):
        r0 = np.arange(0, n * G, rows, dtype=np.int64)
        i0, i1 = r0 // G, np.minimum((r0 + rows - 1) // G + 1, n)
        pos0 = kl - n
        hi = np.maximum(pos0 + i1, 0) if causal else np.full(len(r0), kl)
        lo = np.maximum(np.maximum(pos0 + i0, 0) - window + 1, 0) if window else np.zeros(len(r0), np.int64)
        sink = np.minimum(sinks, lo) if window else lo
        st = -(-sink // 128)
        yield b, np.where(hi > 0, st - (-hi // 128) - np.maximum(lo // 128, st), 0)


@pytest.mark.parametrize("case", [
    # news, lens, Hkv, G, causal, window, sinks, rows of an item
    ([1] * 200, list(range(200)), 2, 4, True, 0, 0, 8),
    ([2, 0, 1], [5000, 7, 70000], 8, 4, True, 0, 0, 8),
    ([200, 33, 0, 1000], [1500, 33, 9, 4000], 4, 4, True, 0, 0, 256),
    ([300, 300], [900, 5000], 2, 2, True, 129, 130, 256),
    ([100, 600], [350, 600], 3, 5, False, 0, 0, 256),
    ([700, 1], [90, 0], 1, 4, True, 0, 0, 256),  # blocks without a key
    ([1 << 16, 5], [1 << 20, 999], 2, 8, True, 0, 0, 256),
    ([5, 1 << 21, 77], [40, 1 << 21, 3000], 1, 64, True, 0, 0, 256),  # 4.3e9 places in one kv head
    ([1 << 20, 1 << 20], [1 << 20, 1 << 22], 2, 64, True, 0, 0, 256),
    ([1 << 20], [1 << 24], 1, 64, False, 0, 0, 256),
], ids=[str(i) for i in range(10)])
def test_the_work_is_divided_into_equal_runs(plan_probe, case):
    """Every CTA's first tile and the length of its run, against whole-number arithmetic."""
    import ctypes

    news, lens, Hkv, G, causal, window, sinks, rows = case
    blocks, lanes = -(-max(news) * G // rows), 1
    while lanes < min(32, blocks):
        lanes *= 2
    min_run = 1 if rows == 8 else 2
    cu, kl = _cu(news), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, err = torch.zeros(152, 8, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    args = (ptr(cu), ptr(kl), len(news), Hkv, G, sum(news), max(news), 12, 1 << 18, int(causal), window, sinks, rows, lanes,
            min_run, ptr(out), ptr(err))
    assert plan_probe(*args) == 0 and int(err) == 0
    items = list(_line(news, lens, G, Hkv, causal, window, sinks, rows))
    places = [np.where(t > 0, t + 2, 0) for _, t in items]  # an item costs two places more than its tiles
    ends = [np.cumsum(x) for x in places]
    heads = [int(e[-1]) if len(e) else 0 for e in ends]
    total = sum(heads) * Hkv
    quota = max(-(-total // 152), min_run)
    for i, got in enumerate(out.tolist()):
        start, left = i * quota, min(quota, total - i * quota)
        want = None
        while left > 0:
            at, x = start, 0
            while at >= heads[x] * Hkv:
                at -= heads[x] * Hkv
                x += 1
            g, at = divmod(at, heads[x])
            rt = int(np.searchsorted(ends[x], at, side="right"))
            t = at - int(ends[x][rt] - places[x][rt])
            if t < items[x][1][rt]:
                want = [1, items[x][0], g, rt, t, left, quota]
                break
            step = int(places[x][rt]) - t  # the two places behind an item's tiles
            start, left = start + step, left - step
        assert got[:7] == want if want else got[0] == 0, (i, got, want)


def test_more_work_than_runs_can_hold_is_refused(plan_probe):
    import ctypes

    from block_sparse_masked_02_gb300 import fdma

    n, kl = 1 << 24, 1 << 30
    cu, lens = _cu([n]), torch.tensor([kl], dtype=torch.int32, device="cuda")
    out, err = torch.zeros(152, 8, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert plan_probe(ptr(cu), ptr(lens), 1, 1, 64, n, n, 12, 1 << 18, 0, 0, 0, 256, 32, 2, ptr(out), ptr(err)) == 0
    assert int(err) == fdma.FDMA_ERR_UNSUPPORTED and not out[:, 0].any()


def _appended(P, s, k, cu, lens):
    """Slots (page, slot) whose K bytes an append changes (k holds no row that the cache had)."""
    raw = lambda: s.kc.view(torch.uint8 if s.fp8 else torch.int16).clone()  # noqa: E731
    before = raw()
    P.kv_append(k, k, s.kc, s.vc, s.table, lens, cu, **s.ex)
    return {tuple(x) for x in (raw() != before).flatten(2).any(-1).nonzero().tolist()}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv", [2, 4, 8])
def test_appends_and_gathers_report_bad_offsets_and_lengths(P, fp8, Hkv):
    """Token ranges past T, that begin before 0 or run backwards, and lengths past the table: reported, and
    only slots of tokens that are there are written."""
    from block_sparse_masked_02_gb300 import fdma

    lens = [40, 300, 25]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(3)

    def slots(s, b, positions):
        return {(int(s.table[b, p // 16]), p % 16) for p in positions}

    def run(cu, T, k_lens=lens):
        s = Setup(P, lens, Hkv, 64, 16, fp8, seed=6, spare=0)
        assert fdma.device_error() == 0
        k = (3 + torch.rand(T, Hkv, 64, generator=g)).bfloat16().cuda()
        got = _appended(P, s, k, i32(*cu), i32(*k_lens))
        return s, got, fdma.device_error()

    bad = fdma.FDMA_ERR_INVALID
    s, got, err = run((0, 3, 7, 9), 9)
    assert err == 0 and got == slots(s, 0, range(37, 40)) | slots(s, 1, range(296, 300)) | slots(s, 2, range(23, 25))
    # past T: inside a sequence, and a sequence that no token belongs to
    s, got, err = run((0, 3, 7, 9), 5)
    assert err == bad and got == slots(s, 0, range(37, 40)) | slots(s, 1, range(296, 298))
    s, got, err = run((0, 3, 5, 9), 5)
    assert err == bad and got == slots(s, 0, range(37, 40)) | slots(s, 1, range(298, 300))
    # before the first token
    s, got, err = run((-2, 1, 2, 3), 3)
    assert err == bad and got == slots(s, 0, [39]) | slots(s, 1, [299]) | slots(s, 2, [24])
    # backwards: only slots of tokens in a range that has them
    s, got, err = run((0, 3, 1, 3), 3)
    assert err == bad and got <= slots(s, 0, range(37, 40)) | slots(s, 2, range(23, 25))
    s, got, err = run((3, 1, 2, 2), 4)
    assert err == bad and got <= slots(s, 1, [299])
    # lengths: none of that sequence's tokens
    cap = s.table.shape[1] * 16
    for n in (cap + 1, cap + 2, 1 << 30, (1 << 31) - 1, -1, -(1 << 31)):
        s, got, err = run((0, 3, 7, 9), 9, (n, 300, 25))
        assert err == bad and got == slots(s, 1, range(296, 300)) | slots(s, 2, range(23, 25))

    s = Setup(P, lens, Hkv, 64, 16, fp8, seed=6, spare=0)
    for cu, T in (((0, 40, 340, 365), 364), ((0, 40, 340, 365), 340), ((-2, 38, 338, 363), 363), ((0, 40, 30, 55), 55)):
        k, v = P.kv_gather(*s.at, i32(*cu), T, **s.ex)
        assert fdma.device_error() == bad
        if cu[2] > cu[1]:
            want = np.concatenate(s.K)[-cu[0]:][:T]
            assert np.array_equal(_np(k), want)
    k, v = P.kv_gather(*s.at, i32(0, 40, 340, 365), 365, **s.ex)
    assert fdma.device_error() == 0 and np.array_equal(_np(v), np.concatenate(s.V))


@pytest.mark.parametrize("d", [64, 112, 128])
def test_scale_bytes_out_of_range_read_as_the_nearest_one(P, d):
    """Bytes that no append writes (0, and 247 to 255): the nearest of 1 .. 246."""
    n = 300
    s = Setup(P, [n], 2, d, 16, True, seed=d)
    pos = torch.arange(n)
    pg, sl = s.table[0, (pos // 16).cuda()].long(), (pos % 16).cuda()
    for x, rows in ((s.ke, s.K), (s.ve, s.V)):
        byte = torch.tensor([0, 1, 246, 247, 250, 255] * (n // 6), dtype=torch.uint8, device="cuda")
        x[pg, sl] = byte[:, None].expand(-1, 2)
        code = (s.kc if x is s.ke else s.vc).view(torch.uint8)[pg, sl].cpu().numpy()
        rows[0] = orc.dequantise(code, np.clip(byte.cpu().numpy(), 1, 246)[:, None].repeat(2, 1))
    k, v = P.kv_gather(*s.at, _cu([n]), n, **s.ex)
    for got, rows in ((k, s.K), (v, s.V)):
        assert torch.equal(got.cpu(), torch.tensor(rows[0]).bfloat16())


@pytest.mark.parametrize("d", [64, 112, 128])
def test_scale_bytes_of_unseen_keys_reach_no_row(P, d):
    """Any scale bytes in a key that only the last row sees: the others get the same bits."""
    n = 300
    s = Setup(P, [n], 2, d, 16, True, seed=d)
    clean = s.ke.clone(), s.ve.clone()
    at = int(s.table[0, (n - 1) // 16]), (n - 1) % 16
    for new in (2, 4, 40, 150):
        q = _queries(new, 8, d, new)
        want = P.fwd(q, *s.at, _cu([new]), new, **s.ex)
        for byte in (246, 247, 255, 0):
            s.ke[at], s.ve[at] = byte, byte
            got = P.fwd(q, *s.at, _cu([new]), new, **s.ex)
            s.ke.copy_(clean[0]), s.ve.copy_(clean[1])
            assert torch.equal(got[0][:-1], want[0][:-1]) and torch.equal(got[1][:, :-1], want[1][:, :-1])

def test_least_codes_at_the_least_scales_read_back_rounded_once(P):
    """Scale bytes 1 and 2 with subnormal codes lie below bf16's least step, 2^-133: rounded once, to nearest even.
    From byte 3 on every value is exact."""
    s = Setup(P, [3], 1, 128, 16, True, seed=1)
    pg = int(s.table[0, 0])
    code = torch.arange(128, dtype=torch.uint8)
    code[127] = 126
    byte = torch.tensor([1, 2, 3], dtype=torch.uint8)
    s.vc.view(torch.uint8)[pg, :3, 0] = code.cuda()
    s.ve[pg, :3, 0] = byte.cuda()
    want = torch.tensor(orc.dequantise(code.numpy()[None].repeat(3, 0), byte.numpy()))
    _, v = P.kv_gather(*s.at, _cu([3]), 3, **s.ex)
    assert torch.equal(v[:, 0].cpu(), want.bfloat16())
    assert torch.equal(v[2, 0].cpu().double(), want[2]) and not torch.equal(v[0, 0].cpu().double(), want[0])


@pytest.mark.parametrize("news,G", [([1], 1), ([2, 1], 4), ([4], 4), ([5], 4)])
@pytest.mark.parametrize("size", [124, 116, 60, -60, -112, -116, -127])
def test_queries_of_any_size_meet_keys_that_undo_it(P, news, G, size):
    """q of 2^size and K of 2^-size: scores of ordinary size, wherever in fp32's range q itself lies (below 2^-126 it is
    subnormal, and rounded to that when it is made)."""
    d, lens = 128, [300 + 70 * b for b in range(len(news))]
    s = Setup(P, lens, 2, d, 16, True, seed=size % 7)
    for b, n in enumerate(lens):
        x = torch.randn(n, 2, d, generator=torch.Generator().manual_seed(b)).bfloat16().double().numpy() * 2.0 ** min(-size, 124)
        code, byte = orc.quantise(x)
        pos = torch.arange(n)
        pg, sl = s.table[b, (pos // 16).cuda()].long(), (pos % 16).cuda()
        s.kc.view(torch.uint8)[pg, sl], s.ke[pg, sl] = torch.from_numpy(code).cuda(), torch.from_numpy(byte).cuda()
        s.K[b] = orc.dequantise(code, byte)
    g = torch.Generator().manual_seed(9)
    q = (torch.randn(sum(news), 2 * G, d, generator=g).bfloat16().double() * 2.0 ** size).bfloat16().cuda()
    assert torch.isfinite(q).all() and bool((q != 0).any())
    out, lse = P.fwd(q, *s.at, _cu(news), max(news), **s.ex)
    _check_attention(s, q, news, out, lse)


def test_a_large_key_at_right_angles_scores_zero(P):
    """Keys of 2^118 in a column where q is zero, beside keys that undo a q of 2^100."""
    d, n = 128, 200
    s = Setup(P, [n], 1, d, 16, True, seed=3)
    x = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(5)).bfloat16().double().numpy() * 2.0 ** -100
    x[:, :, 0] = 0
    x[::9] = 0
    x[::9, :, 0] = 2.0 ** 118
    code, byte = orc.quantise(x)
    pos = torch.arange(n)
    pg, sl = s.table[0, (pos // 16).cuda()].long(), (pos % 16).cuda()
    s.kc.view(torch.uint8)[pg, sl], s.ke[pg, sl] = torch.from_numpy(code).cuda(), torch.from_numpy(byte).cuda()
    s.K[0] = orc.dequantise(code, byte)
    for new in (1, 4, 20):
        q = (torch.randn(new, 4, d, generator=torch.Generator().manual_seed(new)).double() * 2.0 ** 100).bfloat16().cuda()
        q[..., 0] = 0
        out, lse = P.fwd(q, *s.at, _cu([new]), new, **s.ex)
        _check_attention(s, q, [new], out, lse)
