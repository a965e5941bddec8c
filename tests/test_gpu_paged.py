"""The paged key/value cache operators on the GPU against the float64 oracle (oracle/paged.py).

Bounds.  Let u be half a step of the type that the softmax weights are held in for the product with V,
relative to the value: 2^-8 for bf16 (bf16 caches, and every cache in the chunk kernel, whose values
are bf16 in shared memory), 2^-11 for f16 (e4m3 caches in the token kernel: up to 24 rows (new tokens
times heads of a group) a sequence).  A weight P_j carries its own rounding (u) and the error of its score: a sum of d products in
fp32 is off by at most d * 2^-24 * sum |q_c k_c| (times scale: d 2^-24 D), the exponent's argument
S * log2(e) - max and the exponential itself by a few 2^-22 relative to the score's size.  With
w = 2^-22 * (8 + d * D) for both numerator and denominator, every output element is off by at most
    2^-8 |out|  +  (u + 2 w) * A,      A = sum_j P_j |v_j|,
and lse by at most w + 2^-22 |lse|.  Quantised rows and rows read back are exact.
"""
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
    f16 = s.fp8 and max(news) * (q.shape[1] // s.Hkv) <= 24
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
