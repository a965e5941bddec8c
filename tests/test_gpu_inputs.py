"""The operators on attention's inputs on the GPU against the float64 oracle (oracle/inputs.py).

Bounds.  u = 2^-24 is half a step of fp32.  The sum of d squares is off by at most d u relative to itself, its mean,
square root and reciprocal (rsqrtf: 2 steps, 4 u) included the factor 1 / sqrt(mean + eps) by (d / 2 + 6) u, a product with
value and weight by 2 u more; turning a pair adds 3 u of the magnitudes of its two terms.  So an output of the forward is
off by (d / 2 + 12) u M, M the sum of its terms' magnitudes, and by its rounding to bf16, 2^-8 of what is rounded.

Backward: the turned gradient is off by 3 u of its terms, g w x r by (d / 2 + 14) u, the mean of d of them by d u more, and
dx by twice all that and its few products: (2 d + 64) u M, then 2^-8 for bf16.  A weight's gradient sums products that are
off by (d / 2 + 14) u through the steps of a slot, the slots of a CTA and the CTAs' parts: at these sizes fewer than 256
additions in a row, so (d + 300) u of the sum of magnitudes.

The bias is table values rounded once, so it is compared by bits.  Its table's gradient adds, in fp32 and one after the
other, at most 8 values of each of at most 33 blocks of a diagonal, 2 neighbouring lanes', 8 warps', 2 diagonals of a thread
and 5 + 8 in a CTA, and then at most 100 CTAs' and 5 + 8 again at these sizes: 600 u of the sum of magnitudes.  Half of bf16's least step, 2^-134, is added to every bound of a bf16 value.
"""
import numpy as np
import pytest
import torch

from oracle import inputs as orc
from oracle import paged as porc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def I():  # noqa: E743
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_masked_02_gb300 import fdma, inputs

    inputs.load()
    assert fdma.device_error() == 0
    return inputs


@pytest.fixture(autouse=True)
def no_device_error(I):
    yield
    from block_sparse_masked_02_gb300 import fdma

    assert fdma.device_error() == 0


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _rows(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale * torch.exp(torch.randn(*shape[:-1], 1, generator=g))).bfloat16().cuda()


class Case:
    """Queries and keys as slices of one projection, with weights and a table."""

    def __init__(self, I, B, N, Hq, Hk, d, rot=None, weight="shared", wdtype=torch.float32, length=None, seed=0, packed=False):
        g = torch.Generator().manual_seed(seed)
        rot = d if rot is None else rot
        lead = (N,) if packed else (B, N)
        x = _rows(g, *lead, Hq + Hk + 1, d)
        self.q, self.k = x[..., 1:Hq + 1, :], (x[..., Hq + 1:, :] if Hk else None)
        self.rope = I.rope_table(length or N, rot) if rot else None
        self.w = []
        for H in (Hq, Hk):
            w = 1 + 0.3 * torch.randn(*((H, d) if weight == "head" else (d,)), generator=g)
            self.w.append(w.to(wdtype).cuda() if weight and H else None)
        self.dq = _rows(g, *lead, Hq, d)
        self.dk = _rows(g, *lead, Hk, d) if Hk else None
        self.kw = dict(q_weight=self.w[0], k_weight=self.w[1], rope=self.rope)
        self.N, self.lead = N, lead

    def turns(self, pos=None, first=0):
        if self.rope is None:
            return None, None
        pos = np.arange(first, first + self.N) if pos is None else np.clip(pos, 0, self.rope.shape[0] - 1)
        t = _np(self.rope)[pos]
        return t[..., 0, :][..., None, :], t[..., 1, :][..., None, :]


def _check_rows(got, ref, mag, d, back=False, keep=None):
    got = _np(got)
    tol = (2 * d + 64 if back else d / 2 + 12) * U * mag
    tol = 2.0 ** -8 * (np.abs(ref) + tol) + tol + 2.0 ** -134
    err = np.abs(got - ref)
    if keep is not None:
        err, tol = err[keep], tol[keep]
    assert (err <= tol).all(), (err / tol).max()


def _check_forward(c, out, interleaved=False, norm=True, eps=1e-6, pos=None, first=0):
    cos, sin = c.turns(pos, first)
    keep = None if pos is None else np.broadcast_to(pos >= 0, c.lead)
    for x, w, got in zip((c.q, c.k), c.w, out):
        if x is None:
            assert got is None
            continue
        ref, mag = orc.norm_rope(_np(x), _np(w), cos, sin, interleaved, norm, eps)
        assert got.shape == x.shape and got.dtype == torch.bfloat16
        _check_rows(got, ref, mag, x.shape[-1], keep=keep)


def _check_backward(c, grads, interleaved=False, norm=True, eps=1e-6, pos=None, dweight=True):
    cos, sin = c.turns(pos)
    keep = None if pos is None else np.broadcast_to(pos >= 0, c.lead)[..., None, None]
    for x, do, w, got, gw in zip((c.q, c.k), (c.dq, c.dk), c.w, grads[:2], grads[2:]):
        if x is None:
            assert got is None and gw is None
            continue
        d, xd, dd = x.shape[-1], _np(x), _np(do)
        if keep is not None:
            xd, dd = np.where(keep, xd, 0), np.where(keep, dd, 0)
        ref, mag, dw, dwm = orc.norm_rope_bwd(xd, dd, _np(w), cos, sin, interleaved, norm, eps)
        _check_rows(got, ref, mag, d, back=True)
        if keep is not None:
            assert not _np(got)[np.broadcast_to(~keep, got.shape)].any()
        if w is None or not dweight:
            assert gw is None
            continue
        if w.dim() == 1:
            dw, dwm = dw.sum(0), dwm.sum(0)
        assert gw.dtype == torch.float32 and gw.shape == w.shape
        err, tol = np.abs(_np(gw) - dw), (d + 300) * U * dwm + 1e-300
        assert (err <= tol).all(), (err / tol).max()


SHAPES = [  # B, N, Hq, Hk, d, rot, weight, wdtype
    (1, 1, 1, 1, 8, 8, "shared", torch.float32),
    (1, 1, 16, 4, 128, 128, "shared", torch.bfloat16),
    (2, 37, 6, 2, 96, 32, "head", torch.float32),
    (3, 65, 5, 5, 80, 0, "shared", torch.float32),
    (1, 130, 4, 0, 64, 64, "head", torch.bfloat16),
    (1, 33, 3, 1, 72, 72, None, None),
    (2, 19, 2, 1, 256, 128, "head", torch.float32),
    (1, 300, 70, 3, 40, 24, "head", torch.bfloat16),
    (1, 9, 1, 1, 192, 192, "shared", torch.float32),
    (4, 257, 1, 1, 16, 16, "head", torch.float32),
    (1, 3000, 12, 4, 128, 64, "shared", torch.bfloat16),
]


# ------------------------------------------------------------------------------------------------ rows
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,weight,wdtype", SHAPES)
def test_forward(I, B, N, Hq, Hk, d, rot, weight, wdtype, interleaved):
    c = Case(I, B, N, Hq, Hk, d, rot, weight, wdtype, seed=N + d)
    _check_forward(c, I.norm_rope(c.q, c.k, interleaved=interleaved, **c.kw), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,weight,wdtype", SHAPES)
def test_backward(I, B, N, Hq, Hk, d, rot, weight, wdtype, interleaved):
    c = Case(I, B, N, Hq, Hk, d, rot, weight, wdtype, seed=N + d + 1)
    grads = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, interleaved=interleaved, **c.kw)
    _check_backward(c, grads, interleaved)
    again = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, interleaved=interleaved, **c.kw)
    for x, y in zip(grads, again):
        assert (x is None and y is None) or torch.equal(x, y)


@pytest.mark.parametrize("packed", [False, True])
def test_positions_padding_and_places_behind_the_table(I, packed):
    from block_sparse_masked_02_gb300 import fdma

    B, N = (1, 50) if packed else (2, 50)
    c = Case(I, B, N, 3, 2, 64, length=40, packed=packed)
    g = np.random.default_rng(5)
    pos = g.integers(0, 40, c.lead)
    pos.flat[::7] = -1
    pos.flat[3] = -(2 ** 31)
    pt = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for x in (c.q, c.dq, c.k, c.dk):  # padding may hold anything
        x[torch.tensor(pos < 0, device="cuda")] = float("nan")
    qo, ko = torch.full_like(c.q, 7.0), torch.full_like(c.k, 7.0)
    out = I.norm_rope(c.q, c.k, positions=pt, q_out=qo, k_out=ko, **c.kw)
    assert out[0] is qo and out[1] is ko
    for x, y in zip((c.q, c.k), (qo, ko)):
        assert (y[torch.tensor(pos < 0, device="cuda")] == 7).all()
    _check_forward(c, out, pos=pos)
    _check_backward(c, I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, positions=pt, **c.kw), pos=pos)
    assert fdma.device_error() == 0
    pt.view(-1)[5] = 40  # behind the table: left out like padding, and reported
    pos.flat[5] = -1
    qo.fill_(7)
    I.norm_rope(c.q, c.k, positions=pt, q_out=qo, **c.kw)
    assert fdma.device_error() == 1 and (qo.view(-1, 3, 64)[5] == 7).all()
    grads = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, positions=pt, **c.kw)
    assert fdma.device_error() == 1
    _check_backward(c, grads, pos=pos)


def test_positions_in_other_layouts(I):
    c = Case(I, 2, 20, 3, 1, 64, length=100)
    pos = np.random.default_rng(1).integers(0, 100, (2, 20))
    for t in (torch.tensor(pos.T, dtype=torch.int32, device="cuda").T.contiguous(),
              torch.tensor(pos.T.copy(), dtype=torch.int32, device="cuda").T,
              torch.tensor(np.repeat(pos, 3, 1), dtype=torch.int32, device="cuda")[:, ::3]):
        _check_forward(c, I.norm_rope(c.q, c.k, positions=t, **c.kw), pos=pos)
    one = torch.tensor(pos[0], dtype=torch.int32, device="cuda")
    _check_forward(c, I.norm_rope(c.q, c.k, positions=one, **c.kw), pos=np.stack([pos[0]] * 2))
    _check_forward(c, I.norm_rope(c.q, c.k, first=80, **c.kw), first=80)


def test_rotation_alone_and_norm_alone(I):
    c = Case(I, 2, 21, 3, 2, 96, weight=None)
    _check_forward(c, I.norm_rope(c.q, c.k, norm=False, **c.kw), norm=False)
    _check_backward(c, I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, norm=False, **c.kw), norm=False)
    c.rope, c.kw["rope"] = None, None
    _check_forward(c, I.norm_rope(c.q, c.k, eps=0.1), eps=0.1)
    _check_backward(c, I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, eps=0.1), eps=0.1)
    with pytest.raises(RuntimeError):
        I.norm_rope(c.q, c.k, norm=False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_strided_outputs(I, interleaved):
    c = Case(I, 2, 33, 4, 2, 128, 64, "head")
    kw = dict(interleaved=interleaved, **c.kw)
    want, grads = I.norm_rope(c.q, c.k, **kw), I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **kw)
    wide = torch.full((2, 33, 9, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    I.norm_rope(c.q, c.k, q_out=wide[:, :, 1:5, :128], k_out=wide[:, :, 6:8, :128], **kw)
    assert torch.equal(wide[:, :, 1:5, :128], want[0]) and torch.equal(wide[:, :, 6:8, :128], want[1])
    wide[:, :, 1:5, :128] = 3
    wide[:, :, 6:8, :128] = 3
    assert (wide == 3).all()
    dq, dk = c.dq.clone(), c.dk.clone()
    ws = I.norm_rope_bwd_workspace(c.q, c.k, interleaved=interleaved, **c.kw)
    dw = torch.full_like(c.w[0], 9.0)
    got = I.norm_rope_bwd(c.q, c.k, dq, dk, grads=(dq, dk, dw, None), workspace=ws, **kw)
    assert got[0] is dq and got[2] is dw
    for x, y in zip(got, grads):
        assert torch.equal(x, y)
    x = torch.cat((c.q, c.k), 2)
    I.norm_rope(x[:, :, :4], x[:, :, 4:], q_out=x[:, :, :4], k_out=x[:, :, 4:], **kw)
    assert torch.equal(x[:, :, :4], want[0]) and torch.equal(x[:, :, 4:], want[1])
    got = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, want_dweight=False, **kw)
    assert torch.equal(got[0], grads[0]) and torch.equal(got[1], grads[1]) and got[2] is None and got[3] is None
    # one weight of the two
    got = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, interleaved=interleaved, rope=c.rope, q_weight=c.w[0])
    assert torch.equal(got[0], grads[0]) and torch.equal(got[2], grads[2]) and got[3] is None
    got = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, interleaved=interleaved, rope=c.rope, k_weight=c.w[1])
    assert torch.equal(got[1], grads[1]) and torch.equal(got[3], grads[3]) and got[2] is None


def test_rows_of_any_size(I):
    """Squares that fp32 does not hold, rows of zeros, and values that are not finite, which stay in their own row (and, where
    nothing is turned, a value that is not finite does not reach its neighbours but through the norm)."""
    c = Case(I, 1, 40, 2, 1, 128, 64)
    q = c.q
    q[0, 0] *= 1e30
    q[0, 1] = 0
    q[0, 2] = torch.finfo(torch.bfloat16).max
    q[0, 3] *= 1e-30
    q[0, 4, :, 5] = 2e38
    q[0, 5] *= 2.0 ** 64
    _check_forward(c, I.norm_rope(c.q, c.k, **c.kw))
    assert (I.norm_rope(c.q, c.k, **c.kw)[0][0, 1] == 0).all()
    _check_backward(c, I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **c.kw))
    want = I.norm_rope(c.q, c.k, **c.kw)[0]
    q[0, 7, 0, 3] = float("nan")
    q[0, 8, 1, 100] = float("inf")
    got = I.norm_rope(c.q, c.k, **c.kw)[0]
    odd = torch.zeros(40, 2, dtype=torch.bool, device="cuda")
    odd[7, 0] = odd[8, 1] = True
    assert torch.equal(got[0][~odd], want[0][~odd])
    assert torch.isnan(got[0, 7, 0]).all() and torch.isnan(got[0, 8, 1, 100]) and (got[0, 8, 1, :100] == 0).all()
    plain = Case(I, 1, 8, 1, 0, 64, 16, None)
    plain.q[0, 3, 0, 20] = float("inf")
    plain.q[0, 4, 0, 63] = float("nan")
    for inter in (False, True):
        got, _ = I.norm_rope(plain.q, norm=False, rope=plain.rope, interleaved=inter)
        assert torch.isfinite(got).sum() == got.numel() - 2 and torch.isinf(got[0, 3, 0, 20]) and torch.isnan(got[0, 4, 0, 63])


def test_rows_near_both_ends_of_fp32(I):
    """Rows so large or small that the squares of their norms, or the norms' inverses, leave fp32, with small gradients.  The
    bounds are those of all rows: they count relative roundings alone, so no step may leave fp32's normal range."""
    c = Case(I, 1, 48, 2, 1, 128, 64)
    at = 0
    for power in (30, 45, 56, 60, 63, 66, 90):  # (their gradients are of 2^-power times those of the output)
        for small in (0, 20, 30, 40):
            c.q[0, at] *= 2.0 ** power
            c.dq[0, at] *= 2.0 ** -small
            at += 1
    _check_forward(c, I.norm_rope(c.q, c.k, **c.kw))
    _check_backward(c, I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **c.kw))
    for eps in (1e-30, 1e-38, 1e-40, 2.0 ** -149):
        eps = float(np.float32(eps))
        c = Case(I, 1, 48, 2, 1, 128, 64, seed=1)
        for i, power in enumerate((-30, -50, -60, -64, -70, -75, -80, -100, -120)):
            c.q[0, 2 * i] *= 2.0 ** power
            c.q[0, 2 * i + 1] *= 2.0 ** power
            c.dq[0, 2 * i + 1] *= 2.0 ** 10
        c.q[0, 20:30] = 0
        _check_forward(c, I.norm_rope(c.q, c.k, eps=eps, **c.kw), eps=eps)
        _check_backward(c, I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, eps=eps, **c.kw), eps=eps)


def test_a_gradient_that_is_not_finite_stays_in_its_row(I):
    c = Case(I, 1, 40, 2, 1, 128, 64)
    want = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **c.kw)
    c.dq[0, 9, 1, 100] = float("inf")
    got = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **c.kw)
    odd = torch.zeros(40, 2, dtype=torch.bool, device="cuda")
    odd[9, 1] = True
    assert torch.equal(got[0][0][~odd], want[0][0][~odd]) and torch.equal(got[1], want[1]) and torch.equal(got[3], want[3])
    assert not torch.isfinite(got[2][100]) and torch.equal(got[2][:100], want[2][:100])


def _loose(x):
    """The same values with strides of 1 in the dimensions of one."""
    return x.as_strided(x.shape, [1 if n == 1 else s for n, s in zip(x.shape, x.stride())])


@pytest.mark.parametrize("d,rot", [(128, 128), (72, 72), (32, 16), (256, 0)])
@pytest.mark.parametrize("B,N", [(1, 70), (1, 1), (5, 1), (3, 40)])
def test_strides_of_dimensions_of_one_do_not_matter(I, B, N, d, rot):
    """One head, token or batch: a pass has fewer rows than lanes for them, and the stride may be anything."""
    for Hq, Hk, weight in ((1, 1, "shared"), (1, 1, "head"), (1, 3, "shared"), (3, 1, None)):
        c = Case(I, B, N, Hq, Hk, d, rot, weight, seed=N)
        q, k, dq, dk = (x.contiguous() for x in (c.q, c.k, c.dq, c.dk))
        want, grads = I.norm_rope(q, k, **c.kw), I.norm_rope_bwd(q, k, dq, dk, **c.kw)
        q, k, dq, dk = (_loose(x) for x in (q, k, dq, dk))
        assert Hq > 1 or q.stride(2) == 1
        out = [_loose(torch.empty_like(x)) for x in (q, k, dq, dk)]
        got = I.norm_rope(q, k, q_out=out[0], k_out=out[1], **c.kw)
        got += I.norm_rope_bwd(q, k, dq, dk, grads=(out[2], out[3], None, None), **c.kw)
        for x, y in zip(got, want + grads):
            assert (x is None and y is None) or torch.equal(x, y)


def test_no_tokens(I):
    c = Case(I, 1, 3, 2, 1, 64)
    q, k = c.q[:, :0], c.k[:, :0]
    out = I.norm_rope(q, k, **c.kw)
    assert out[0].shape == (1, 0, 2, 64)
    g = I.norm_rope_bwd(q, k, c.dq[:, :0], c.dk[:, :0], **c.kw)
    assert not g[2].any() and not g[3].any() and g[2].shape == (64,)


def test_offsets_past_32_bits(I):
    N, step = 3, (1 << 30) + 64  # elements between tokens: the third is behind 2^31
    big = torch.empty(2 * step + 2 * 64, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(3)
    q = big.as_strided((N, 2, 64), (step, 64, 1))
    q.copy_(_rows(g, N, 2, 64))
    rope = I.rope_table(N, 64)
    want, _ = I.norm_rope(q.clone().contiguous(), rope=rope)
    assert torch.equal(I.norm_rope(q, rope=rope)[0], want)
    do = _rows(g, N, 2, 64)
    grads = I.norm_rope_bwd(q.clone().contiguous(), None, do, None, rope=rope)
    assert torch.equal(I.norm_rope_bwd(q, None, do, None, rope=rope)[0], grads[0])
    I.norm_rope(q, rope=rope, q_out=q)
    assert torch.equal(q, want)


def test_norm_rope_refusals(I):
    c = Case(I, 1, 4, 2, 1, 64)
    ok = dict(c.kw)
    with pytest.raises(ValueError, match="one device"):
        I.norm_rope(c.q, c.k, **{**ok, "q_weight": c.w[0].cpu()})
    with pytest.raises(ValueError):
        I.norm_rope(c.q, c.k, q_out=torch.empty(1, 4, 2, 32, dtype=torch.bfloat16, device="cuda"), **ok)
    with pytest.raises(ValueError):
        I.norm_rope_bwd(c.q, c.k, c.dq, None, **ok)
    with pytest.raises(ValueError):
        I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, grads=(None, None, torch.empty(32, device="cuda"), None), **ok)
    with pytest.raises(ValueError):
        I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, grads=(None, None), **ok)
    with pytest.raises(RuntimeError, match="workspace"):
        I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), **ok)
    for kw in (dict(eps=0.0), dict(first=1), dict(first=-1)):
        with pytest.raises(RuntimeError, match="invalid"):
            I.norm_rope(c.q, c.k, **ok, **kw)
    with pytest.raises(RuntimeError, match="unsupported"):
        I.norm_rope(torch.empty(4, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64], rope=c.rope)


# ------------------------------------------------------------------------------------------------ append
class Serving:
    """A cache in scattered pages and new tokens behind some that it holds."""

    def __init__(self, I, news, olds, Hq, Hkv, d, page=16, fp8=False, rot=None, weight="shared", extra=3, seed=0, wdtype=torch.float32):
        from block_sparse_masked_02_gb300 import paged

        self.P, self.news, self.page, self.fp8 = paged, news, page, fp8
        g = torch.Generator().manual_seed(seed)
        lens = [n + o for n, o in zip(news, olds)]
        pages = [-(-n // page) for n in lens]
        num = sum(pages) + 2
        ids, at = torch.randperm(num, generator=g), 0
        table = torch.full((len(news), max(pages + [0]) + 1), -5, dtype=torch.int32)
        for b, n in enumerate(pages):
            table[b, :n] = ids[at:at + n].int()
            at += n
        self.kc, self.vc, self.ke, self.ve = paged.empty_cache(num, page, Hkv, d, dtype=E4M3 if fp8 else torch.bfloat16)
        for x in (self.kc, self.vc):
            x.view(torch.uint8).fill_(0x55)
        self.ex = dict(k_exp=self.ke, v_exp=self.ve)
        if fp8:
            self.ke.fill_(9)
            self.ve.fill_(9)
        self.T = sum(news) + extra
        self.table, self.k_lens = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
        x = _rows(g, self.T, Hq + 2 * Hkv, d)
        self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        rot = d if rot is None else rot
        self.rope = I.rope_table(max(lens + [1]), rot) if rot else None
        self.w = []
        for H in (Hq, Hkv):
            w = 1 + 0.3 * torch.randn(*((H, d) if weight == "head" else (d,)), generator=g)
            self.w.append(w.to(wdtype).cuda() if weight else None)
        self.kw = dict(q_weight=self.w[0], k_weight=self.w[1], rope=self.rope)
        self.pos = np.concatenate([np.arange(o, o + n) for n, o in zip(news, olds)] + [np.full(extra, -1)]).astype(np.int64)
        self.at = (self.kc, self.vc, self.table, self.k_lens)

    def slots(self):
        b = np.repeat(np.arange(len(self.news)), self.news)
        p = self.pos[:len(b)]
        return self.table.cpu().numpy()[b, p // self.page], p % self.page

    def exact(self, pos=None, interleaved=False):
        pos = np.clip(self.pos if pos is None else pos, 0, None)
        cos = sin = None
        if self.rope is not None:
            t = _np(self.rope)[np.minimum(pos, self.rope.shape[0] - 1)]
            cos, sin = t[:, None, 0], t[:, None, 1]
        return [orc.norm_rope(_np(x), _np(w), cos, sin, interleaved, True, 1e-6) for x, w in zip((self.q, self.k), self.w)]


APPENDS = [  # news, olds, Hq, Hkv, d, page, rot, weight
    ([1], [0], 1, 1, 64, 16, None, "shared"),
    ([1, 1, 1, 1, 1], [3, 0, 15, 16, 200], 8, 2, 128, 16, None, "shared"),
    ([5, 0, 33, 1, 18], [11, 4, 0, 31, 14], 6, 3, 96, 32, 32, "head"),
    ([0, 7], [0, 9], 5, 5, 48, 64, 0, "shared"),
    ([130, 70], [1, 64], 16, 4, 128, 64, 64, None),
    ([2] * 40, list(range(40)), 4, 1, 16, 16, None, "head"),
    ([20, 1], [7, 300], 13, 7, 80, 16, 48, "head"),
    ([3, 9], [2, 30], 7, 2, 32, 32, 32, "shared"),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("news,olds,Hq,Hkv,d,page,rot,weight", APPENDS)
def test_append(I, news, olds, Hq, Hkv, d, page, rot, weight, interleaved, fp8):
    s = Serving(I, news, olds, Hq, Hkv, d, page, fp8, rot, weight, seed=d + page, wdtype=torch.bfloat16 if d > 64 else torch.float32)
    q_out = torch.full_like(s.q, 7.0)
    before = [x.clone() for x in (s.kc, s.vc)]
    got = s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, interleaved=interleaved, q_out=q_out, **s.kw, **s.ex)
    n = sum(news)
    (qr, qm), (kr, km) = s.exact(interleaved=interleaved)
    assert got is q_out and (got[n:] == 7).all()
    _check_rows(got[:n], qr[:n], qm[:n], d)
    pg, sl = (torch.tensor(x, device="cuda") for x in s.slots())
    if not fp8:
        _check_rows(s.kc[pg, sl], kr[:n], km[:n], d)
        assert torch.equal(s.vc[pg, sl], s.v[:n])
        # bit for bit what the two calls give
        q2, k2 = I.norm_rope(s.q[:n], s.k[:n], interleaved=interleaved,
                             positions=torch.tensor(s.pos[:n], dtype=torch.int32, device="cuda"), **s.kw)
        assert torch.equal(got[:n], q2) and torch.equal(s.kc[pg, sl], k2)
    else:
        vcode, vexp = porc.quantise(_np(s.v[:n]))
        assert np.array_equal(s.vc.view(torch.uint8)[pg, sl].cpu().numpy(), vcode)
        assert np.array_equal(s.ve[pg, sl].cpu().numpy(), vexp)
        delta = (d / 2 + 12) * U * km[:n]
        top, off = np.abs(kr[:n]).max(-1), delta.max(-1)
        least = lambda m: np.clip(np.ceil(np.log2(np.maximum(m, 1e-300) / 448)), -126, 119) + 127  # noqa: E731
        e = s.ke[pg, sl].cpu().numpy().astype(np.float64)
        assert (least(top - off) <= e).all() and (e <= least(top + off)).all()
        step = 2.0 ** (e - 127)[..., None]
        val = porc.dequantise(s.kc.view(torch.uint8)[pg, sl].cpu().numpy(), e.astype(np.uint8))
        tol = delta + np.maximum(2.0 ** -4 * (np.abs(kr[:n]) + delta), 2.0 ** -10 * step)
        assert (np.abs(val - kr[:n]) <= tol).all()
    keep = torch.ones(s.kc.shape[:2], dtype=torch.bool, device="cuda")
    keep[pg, sl] = False
    for x, y in zip((s.kc, s.vc), before):
        assert torch.equal(x.view(torch.uint8)[keep], y.view(torch.uint8)[keep])
    if fp8:
        assert (s.ke[keep] == 9).all() and (s.ve[keep] == 9).all()


def test_append_at_other_positions_and_with_padding(I):
    from block_sparse_masked_02_gb300 import fdma

    s = Serving(I, [6, 9], [10, 3], 4, 2, 64, rot=32)
    n = 15
    pos = np.concatenate([np.random.default_rng(2).integers(0, s.rope.shape[0], n), [-1, -1, -1]])
    pos[[2, 8]] = -1
    pt = torch.tensor(pos, dtype=torch.int32, device="cuda")
    q_out = torch.full_like(s.q, 7.0)
    kept = s.kc.clone()
    s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, positions=pt, q_out=q_out, **s.kw)
    assert fdma.device_error() == 0
    (qr, qm), (kr, km) = s.exact(pos)
    real = pos[:n] >= 0
    pg, sl = s.slots()
    _check_rows(q_out[:n], qr[:n], qm[:n], 64, keep=real)
    _check_rows(s.kc[torch.tensor(pg).cuda(), torch.tensor(sl).cuda()], kr[:n], km[:n], 64, keep=real)
    for i in np.flatnonzero(~real):
        assert (q_out[i] == 7).all() and torch.equal(s.kc[pg[i], sl[i]].view(torch.uint8), kept[pg[i], sl[i]].view(torch.uint8))
    pt[4] = s.rope.shape[0]
    q_out.fill_(7)
    s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, positions=pt, q_out=q_out, **s.kw)
    assert fdma.device_error() == 1 and (q_out[4] == 7).all() and not (q_out[5] == 7).all()


def test_append_leaves_out_what_the_plan_does_not_reach(I):
    from block_sparse_masked_02_gb300 import fdma

    s = Serving(I, [6, 9, 4], [30, 3, 0], 4, 2, 64)
    want = torch.full_like(s.q, 7.0)
    s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, q_out=want, **s.kw)
    kc = s.kc.clone()
    for x in (s.kc, s.vc):
        x.view(torch.uint8).fill_(0x55)
    s.table[0, 2] = s.kc.shape[0] + 5  # the page of positions 32 to 35 of sequence 0
    s.k_lens[1] = 1 << 20  # behind the table
    q_out = torch.full_like(s.q, 7.0)
    s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, q_out=q_out, **s.kw)
    assert fdma.device_error() == 1
    assert torch.equal(q_out[:2], want[:2]) and (q_out[2:15] == 7).all() and torch.equal(q_out[15:], want[15:])
    for i, (pg, sl) in enumerate(zip(*s.slots())):
        if i < 2 or i >= 15:
            assert torch.equal(s.kc[pg, sl], kc[pg, sl])
    s.k_lens[1] = 12
    s.cu[2] = 100  # runs back after it
    s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, q_out=q_out, **s.kw)
    assert fdma.device_error() == 1


def test_append_to_nothing(I):
    s = Serving(I, [2], [0], 2, 1, 64, extra=0)
    out = s.P.norm_rope_append(s.q[:0], s.k[:0], s.v[:0], *s.at, torch.zeros(2, dtype=torch.int32, device="cuda"), **s.kw)
    assert out.shape == (0, 2, 64)
    none = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    s.P.norm_rope_append(s.q, s.k, s.v, s.kc, s.vc, none, none[:, 0], s.cu[:1], **s.kw)
    assert (s.kc.view(torch.uint8) == 0x55).all()
    with pytest.raises(ValueError):
        s.P.norm_rope_append(s.q, s.k, s.v[:, :, :32], *s.at, s.cu, **s.kw)
    with pytest.raises(ValueError):
        s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, positions=torch.zeros(2, 2, dtype=torch.int32, device="cuda"), **s.kw)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_in_other_layouts_and_on_another_stream(I, fp8):
    """Token-major pages with gaps, a page stride past 32 bits, q_out among other rows: as in the usual layout."""
    s = Serving(I, [9, 3], [12, 30], 4, 2, 64, fp8=fp8)
    want = s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, **s.kw, **s.ex)
    num, dt = s.kc.shape[0], s.kc.dtype
    kc = torch.empty(num, 16, 2, 96, dtype=dt, device="cuda")[..., :64]
    step = ((1 << 31) + 4096) // (num - 1) // 128 * 128 + 128  # the last page begins behind 2^31 elements
    vc = torch.empty(step * (num - 1) + 16 * 2 * 64, dtype=dt, device="cuda").as_strided((num, 16, 2, 64), (step, 128, 64, 1))
    ke = torch.empty(num, 16, 3, dtype=torch.uint8, device="cuda")[..., 1:] if fp8 else None
    ve = torch.empty(num, 2, 2, 16, dtype=torch.uint8, device="cuda")[:, :, 1].transpose(1, 2) if fp8 else None
    rows = torch.empty(s.T, 9, 64, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s.P.norm_rope_append(s.q, s.k, s.v, kc, vc, s.table, s.k_lens, s.cu, q_out=rows[:, 2:6], k_exp=ke, v_exp=ve,
                               stream=side, **s.kw)
    side.synchronize()
    pg, sl = (torch.tensor(x, device="cuda") for x in s.slots())
    n = 12
    assert torch.equal(got[:n], want[:n])
    for x, y in ((kc, s.kc), (vc, s.vc)) + (((ke, s.ke), (ve, s.ve)) if fp8 else ()):
        assert torch.equal(x[pg, sl].view(torch.uint8), y[pg, sl].view(torch.uint8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("news", [[1], [9, 3], [700, 900]])
def test_append_with_any_stride_of_one_head(I, fp8, news):
    s = Serving(I, news, [12] * len(news), 1, 1, 64, fp8=fp8, extra=0)
    q, k, v = (x.contiguous() for x in (s.q, s.k, s.v))
    want = s.P.norm_rope_append(q, k, v, *s.at, s.cu, **s.kw, **s.ex)
    kept = [x.clone() for x in (s.kc, s.vc, s.ke, s.ve) if x is not None]
    for x in (s.kc, s.vc):
        x.view(torch.uint8).fill_(0x55)
    q, k, v = (_loose(x) for x in (q, k, v))
    assert k.stride(1) == 1
    got = s.P.norm_rope_append(q, k, v, *s.at, s.cu, q_out=_loose(torch.empty_like(q)), **s.kw, **s.ex)
    assert torch.equal(got, want)
    for x, y in zip([x for x in (s.kc, s.vc, s.ke, s.ve) if x is not None], kept):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_of_values_that_are_not_finite(I):
    for fp8 in (False, True):
        s = Serving(I, [8], [5], 2, 2, 64, fp8=fp8, extra=0)
        s.v[3, 0, 7] = float("inf")
        s.v[4, 1, 2] = float("nan")
        s.k[5, 0, 1] = float("nan")
        s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, **s.kw, **s.ex)
        pg, sl = (torch.tensor(x, device="cuda") for x in s.slots())
        if not fp8:
            assert torch.equal(s.vc[pg, sl].view(torch.int16), s.v.view(torch.int16))
            assert torch.isnan(s.kc[pg, sl][5, 0]).all() and torch.isfinite(s.kc[pg, sl][5, 1]).all()
            continue
        code, byte = porc.quantise(_np(s.v))
        assert np.array_equal(s.vc.view(torch.uint8)[pg, sl].cpu().numpy() & 0x7F, code & 0x7F)
        assert np.array_equal(s.ve[pg, sl].cpu().numpy(), byte)


# ------------------------------------------------------------------------------------------------ bias
BIASES = [  # H, Nq, Nk, starts, two_sided, offset
    (1, 1, 8, (0,), False, None),
    (3, 1, 4096, (0, 1, 2, 4, 8, 64, 1000), False, None),
    (2, 5, 264, (0, 1, 2, 4, 8, 64), True, None),
    (4, 129, 136, "usual", True, None),
    (1, 1000, 64, "usual", True, None),
    (2, 300, 520, "usual", False, 17),
    (2, 77, 2056, (0, 0, 3, 3, 3, 900), True, 700),
    (5, 64, 128, tuple(range(256)), True, -500),
    (1, 2050, 2048, (0, 300, 600), False, 1 << 30),
    (1, 16, 16, (0, 5), True, -(1 << 30)),
]


def _starts(I, s, two_sided):
    return I.rel_starts(32, 128, bidirectional=two_sided) if s == "usual" else s


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,Nq,Nk,starts,two,offset", BIASES)
def test_bias(I, H, Nq, Nk, starts, two, offset, dtype):
    starts = _starts(I, starts, two)
    n = len(starts) * (2 if two else 1)
    table = torch.randn(n, H, generator=torch.Generator().manual_seed(Nq)).to(dtype).cuda()
    off = Nk - Nq if offset is None else offset
    at = torch.tensor(orc.buckets(Nq, Nk, starts, two, off), device="cuda")
    want = table.bfloat16()[at].permute(2, 0, 1)[None]
    got = I.rel_bias(table, Nq, Nk, starts, bidirectional=two, offset=offset)
    assert got.shape == (1, H, Nq, Nk) and torch.equal(got, want)
    # another order of the table, and rows with something between them
    wide = torch.full((1, H, Nq + 1, Nk + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    I.rel_bias(table.T.contiguous().T, Nq, Nk, starts, bidirectional=two, offset=offset, out=wide[:, :, :Nq, 8:8 + Nk])
    assert torch.equal(wide[:, :, :Nq, 8:8 + Nk], want)
    wide[:, :, :Nq, 8:8 + Nk] = 3
    assert (wide == 3).all()
    rows = torch.full((Nq, H, Nk), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[None]
    I.rel_bias(table, Nq, Nk, starts, bidirectional=two, offset=offset, out=rows)
    assert torch.equal(rows, want)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("H,Nq,Nk,starts,two,offset", BIASES)
def test_bias_gradient(I, H, Nq, Nk, starts, two, offset, B, causal):
    starts = _starts(I, starts, two)
    off = Nk - Nq if offset is None else offset
    g = torch.Generator().manual_seed(Nq + B)
    db = (torch.randn(B, H, Nq, Nk, generator=g) * torch.exp(torch.randn(B, H, Nq, 1, generator=g))).bfloat16().cuda()
    ref, mag = orc.rel_bias_bwd(_np(db), starts, two, off, causal)
    if causal:  # what is behind the diagonal may hold anything
        i, j = torch.arange(Nq, device="cuda")[:, None], torch.arange(Nk, device="cuda")[None]
        db.masked_fill_(j > i + off, float("nan"))
    kw = dict(bidirectional=two, offset=offset, causal=causal)
    got = I.rel_bias_bwd(db, starts, **kw)
    assert got.dtype == torch.float32 and got.shape == ref.shape
    err, tol = np.abs(_np(got) - ref), 600 * U * mag
    assert (err <= tol).all(), np.nanmax(err / np.maximum(tol, 1e-300))
    assert torch.equal(got, I.rel_bias_bwd(db, starts, **kw))
    wide = torch.zeros(B, H, Nq, Nk + 8, dtype=torch.bfloat16, device="cuda")[..., 8:]
    wide.copy_(db)
    ws = I.rel_bias_bwd_workspace(B, H, Nq, Nk, starts, bidirectional=two)
    ws.fill_(255)
    out = torch.full_like(got, 5.0)
    assert I.rel_bias_bwd(wide, starts, dtable=out, workspace=ws, **kw) is out and torch.equal(out, got)


def test_bias_gradient_of_a_repeated_batch_and_of_nothing(I):
    starts = (0, 1, 4)
    db = torch.randn(1, 1, 20, 32, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    one, many = (I.rel_bias_bwd(x, starts, bidirectional=False) for x in (db, db.expand(4, 3, 20, 32)))
    assert np.allclose(_np(many), 4 * _np(one).repeat(3, 1), rtol=1e-6, atol=1e-5)
    for shape in ((0, 2, 8, 8), (2, 2, 0, 8), (2, 2, 8, 0)):
        g = I.rel_bias_bwd(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), starts)
        assert g.shape == (6, 2) and not g.any()
    assert I.rel_bias(torch.zeros(3, 2, device="cuda"), 0, 8, starts, bidirectional=False).shape == (1, 2, 0, 8)


def test_bias_values_that_are_not_finite(I):
    table = torch.tensor([[float("inf")], [float("nan")], [-float("inf")], [torch.finfo(torch.bfloat16).min]], device="cuda")
    got = I.rel_bias(table, 16, 16, (0, 2, 4, 6), bidirectional=False)[0, 0]
    assert torch.isinf(got[0, 0]) and torch.isnan(got[3, 0]) and got[5, 0] == -float("inf") and got[15, 0] == table[3, 0]
    db = torch.zeros(1, 1, 16, 16, dtype=torch.bfloat16, device="cuda")
    db[0, 0, 9, 6] = float("nan")
    g = I.rel_bias_bwd(db, (0, 2, 4, 6), bidirectional=False)
    assert torch.isnan(g[1, 0]) and not g[[0, 2, 3]].any()


def test_bias_offsets_past_32_bits(I):
    H, Nq, Nk, step = 3, 9, 16, (1 << 30) + 8
    big = torch.empty(2 * step + Nq * Nk, dtype=torch.bfloat16, device="cuda")
    out = big.as_strided((1, H, Nq, Nk), (0, step, Nk, 1))
    table = torch.randn(8, H, generator=torch.Generator().manual_seed(2)).cuda()
    starts = (0, 1, 2, 5)
    want = I.rel_bias(table, Nq, Nk, starts)
    assert torch.equal(I.rel_bias(table, Nq, Nk, starts, out=out), want)
    assert torch.equal(I.rel_bias_bwd(out, starts), I.rel_bias_bwd(want, starts))


def test_bias_refusals(I):
    t = torch.zeros(8, 2, device="cuda")
    for bad in (dict(starts=(0, 1, 2)), dict(table=t.half()), dict(table=t[0])):
        with pytest.raises(ValueError):
            I.rel_bias(bad.get("table", t), 8, 8, bad.get("starts", (0, 1, 2, 3)))
    for out in (torch.empty(1, 2, 8, 16, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 2, 8, 8, device="cuda")):
        with pytest.raises(ValueError):
            I.rel_bias(t, 8, 8, (0, 1, 2, 3), out=out)
    for kw in (dict(Nk=12), dict(starts=(0, 2, 1, 3)), dict(starts=(1, 2, 3, 4)), dict(offset=(1 << 30) + 1)):
        with pytest.raises(RuntimeError):
            I.rel_bias(t, 8, kw.get("Nk", 8), kw.get("starts", (0, 1, 2, 3)), offset=kw.get("offset"))
    db = torch.zeros(1, 2, 8, 8, dtype=torch.bfloat16, device="cuda")
    for x in (db.float(), db[0], db.transpose(2, 3)):
        with pytest.raises(ValueError):
            I.rel_bias_bwd(x, (0, 1))
    with pytest.raises(ValueError):
        I.rel_bias_bwd(db, (0, 1), dtable=torch.empty(2, 2, device="cuda"))
    with pytest.raises(RuntimeError, match="workspace"):
        I.rel_bias_bwd(db, (0, 1), workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------------------------------------ many shapes
@pytest.mark.parametrize("seed", range(24))
def test_random_rows(I, seed):
    """Random sizes, layouts and options; rows that a warp's walk, a chunk of heads or a pass does not divide."""
    r = np.random.default_rng(1000 + seed)
    d = int(r.integers(1, 33)) * 8
    rot = int(r.integers(0, d // 8 + 1)) * 8
    B, N = int(r.integers(1, 5)), int(2 ** r.uniform(0, 9))
    Hq, Hk = int(r.integers(1, 12)), int(r.integers(0, 6))
    weight = [None, "shared", "head"][seed % 3]
    inter = bool(r.integers(0, 2))
    c = Case(I, B, N, Hq, Hk, d, rot, weight, [torch.float32, torch.bfloat16][seed % 2], length=N + 7, seed=seed)
    pos = None
    kw = dict(interleaved=inter, **c.kw)
    if r.integers(0, 2):
        pos = r.integers(-2, N + 7, (B, N))
        kw["positions"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    _check_forward(c, I.norm_rope(c.q, c.k, **kw), inter, pos=pos)
    grads = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **kw)
    _check_backward(c, grads, inter, pos=pos)


def test_walks_of_many_tokens(I):
    """More than 32 tokens for every warp, some of them padding, of one and of many batches."""
    for B, N, Hq, Hk in ((1, 150000, 1, 1), (50000, 3, 1, 0)):
        c = Case(I, B, N, Hq, Hk, 16, 8, "shared", length=500, seed=N)
        pos = np.random.default_rng(N).integers(-100, 500, (B, N))
        pt = torch.tensor(pos, dtype=torch.int32, device="cuda")
        _check_forward(c, I.norm_rope(c.q, c.k, positions=pt, **c.kw), pos=pos)
        cos, sin = c.turns(pos)
        keep = (pos >= 0)[..., None, None]
        grads = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, positions=pt, **c.kw)
        for x, do, w, got, gw in zip((c.q, c.k), (c.dq, c.dk), c.w, grads[:2], grads[2:]):
            if x is None:
                continue
            ref, mag, dw, dwm = orc.norm_rope_bwd(np.where(keep, _np(x), 0), np.where(keep, _np(do), 0), _np(w), cos, sin, False, True, 1e-6)
            _check_rows(got, ref, mag, 16, back=True)
            # (every one of a slot's up to 100 tokens and of up to 152 CTAs one after the other)
            assert (np.abs(_np(gw) - dw.sum(0)) <= (16 + 700) * U * dwm.sum(0)).all()


# Tokens that leave a warp one to three of them, whole or in chunks of heads.  (A weight's sum: a lane adds fewer than
# 64 passes, a CTA 32 lanes, and fewer than 2 * 456 parts are added 32 side by side: under the 256 of the tolerance.)
@pytest.mark.parametrize("B,N,Hq,Hk,d", [(1, 700, 64, 8, 128), (2, 401, 28, 4, 128), (3, 333, 36, 0, 128), (1, 1300, 48, 16, 64),
                                         (1, 900, 5, 40, 256)])
def test_tokens_in_chunks_of_heads(I, B, N, Hq, Hk, d):
    c = Case(I, B, N, Hq, Hk, d, seed=N)
    _check_forward(c, I.norm_rope(c.q, c.k, **c.kw))
    _check_backward(c, I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **c.kw))


@pytest.mark.parametrize("B,N,Hq,Hk,d,rot", [(3, 1100, 40, 4, 64, 64), (700, 3, 5, 1, 128, 32), (2, 900, 21, 3, 72, 72)])
def test_walks_with_a_weight_a_head(I, B, N, Hq, Hk, d, rot):
    """Several tokens a warp, over the ends of batches, with padding; a warp has one pass of each."""
    c = Case(I, B, N, Hq, Hk, d, rot, "head", length=N, seed=B)
    pos = np.random.default_rng(B).integers(0, N, (B, N))
    pos.flat[::5] = -1
    pt = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for kw, p in ((dict(), None), (dict(positions=pt), pos)):
        qo, ko = torch.full_like(c.q, 7.0), torch.full_like(c.k, 7.0)
        _check_forward(c, I.norm_rope(c.q, c.k, q_out=qo, k_out=ko, **kw, **c.kw), pos=p)
        assert p is None or all((x[pt < 0] == 7).all() for x in (qo, ko))
        _check_backward(c, I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **kw, **c.kw), pos=p)


@pytest.mark.parametrize("B,N,Hq,Hk,d", [(1, 40000, 16, 4, 128), (5, 6007, 21, 3, 96)])
def test_rows_of_more_than_l2_holds(I, B, N, Hq, Hk, d):
    """Row for row what calls of a few tokens give; the weights' gradients are those calls' sums.  (Each sum, and
    that of the calls, is off by at most (d + 300) u of the magnitudes, as everywhere here; a turned value is at most the sum of
    its pair.)"""
    c = Case(I, B, N, Hq, Hk, d, length=N)
    pos = torch.randint(-N // 8, N, (B, N), dtype=torch.int32, device="cuda")
    qo, ko = torch.full_like(c.q, 7.0), torch.full_like(c.k, 7.0)
    I.norm_rope(c.q, c.k, positions=pos, q_out=qo, k_out=ko, **c.kw)
    dq, dk, *dw = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, positions=pos, **c.kw)
    total, mag = [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2)], [0.0, 0.0]
    for n in range(0, N, N // 5):
        s = slice(n, n + N // 5)
        p, a, b = pos[:, s].contiguous(), torch.full_like(qo[:, s], 7.0), torch.full_like(ko[:, s], 7.0)
        I.norm_rope(c.q[:, s], c.k[:, s], positions=p, q_out=a, k_out=b, **c.kw)
        assert torch.equal(a, qo[:, s]) and torch.equal(b, ko[:, s])
        a, b, *w = I.norm_rope_bwd(c.q[:, s], c.k[:, s], c.dq[:, s], c.dk[:, s], positions=p, **c.kw)
        assert torch.equal(a, dq[:, s]) and torch.equal(b, dk[:, s])
        for i, (x, g) in enumerate(((c.q, c.dq), (c.k, c.dk))):
            total[i] += w[i].double()
            x, g = x[:, s].double(), g[:, s].double().abs() * (p >= 0)[..., None, None]
            g = g + torch.cat((g[..., d // 2:], g[..., :d // 2]), -1)
            mag[i] = mag[i] + (g * x.abs() * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()).sum((0, 1, 2))
    for i in range(2):
        assert ((dw[i].double() - total[i]).abs() <= 2 * (d + 300) * U * mag[i]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_append_of_many_tokens(I, fp8):
    """So many that a warp takes whole tokens, with an empty sequence, a sequence of one and rows behind the last."""
    s = Serving(I, [3000, 0, 1, 2100], [5, 9, 63, 640], 3, 2, 32, 64, fp8, rot=16, extra=9, seed=3)
    got = s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, **s.kw, **s.ex)
    (qr, qm), (kr, km) = s.exact()
    n = 5101
    _check_rows(got[:n], qr[:n], qm[:n], 32)
    pg, sl = (torch.tensor(x, device="cuda") for x in s.slots())
    if fp8:
        vcode, vexp = porc.quantise(_np(s.v[:n]))
        assert np.array_equal(s.vc.view(torch.uint8)[pg, sl].cpu().numpy(), vcode)
        assert np.array_equal(s.ve[pg, sl].cpu().numpy(), vexp)
    else:
        _check_rows(s.kc[pg, sl], kr[:n], km[:n], 32)
        assert torch.equal(s.vc[pg, sl], s.v[:n])


@pytest.mark.parametrize("seed", range(24))
def test_random_biases(I, seed):
    r = np.random.default_rng(2000 + seed)
    H, B = int(r.integers(1, 5)), int(r.integers(1, 4))
    Nq, Nk = int(2 ** r.uniform(0, 10)), 8 * int(2 ** r.uniform(0, 7))
    two = bool(seed % 2)
    n = int(r.integers(1, 257 if seed % 5 == 0 else 40))
    starts = (0,) + tuple(int(x) for x in np.sort(r.integers(0, int(2 ** r.uniform(1, 11)), n - 1)))
    offset = None if r.integers(0, 2) else int(r.integers(-700, 700))
    off = Nk - Nq if offset is None else offset
    table = torch.tensor(r.standard_normal((n * (2 if two else 1), H)), dtype=torch.float32, device="cuda")
    at = torch.tensor(orc.buckets(Nq, Nk, starts, two, off), device="cuda")
    got = I.rel_bias(table, Nq, Nk, starts, bidirectional=two, offset=offset)
    assert torch.equal(got, table.bfloat16()[at].permute(2, 0, 1)[None])
    db = torch.tensor(r.standard_normal((B, H, Nq, Nk)), dtype=torch.bfloat16, device="cuda")
    for causal in (False, True):
        ref, mag = orc.rel_bias_bwd(_np(db), starts, two, off, causal)
        g = I.rel_bias_bwd(db, starts, bidirectional=two, offset=offset, causal=causal)
        assert (np.abs(_np(g) - ref) <= 600 * U * mag).all()


# ------------------------------------------------------------------------------------------------ together
def test_a_training_step(I):
    """norm_rope, rel_bias, attention and their gradients against torch's in 64 bits: relative to the norm of each result, each
    attention gradient is held to 1e-2 by its own tests, q and k are rounded to bf16 before it (2^-8 each, at most
    doubled through the scores), and each gradient once after it."""
    from block_sparse_masked_02_gb300 import fdma

    B, N, Hq, Hk, d = 2, 200, 4, 2, 64
    c = Case(I, B, N, Hq, Hk, d, 32, "head", torch.float32, seed=11)
    g = torch.Generator().manual_seed(12)
    v, do = _rows(g, B, N, Hk, d), _rows(g, B, N, Hq, d)
    starts = I.rel_starts(16, 64, bidirectional=False)
    table = torch.randn(16, Hk, generator=g).cuda()
    bias = I.rel_bias(table, N, N, starts, bidirectional=False).expand(B, -1, -1, -1)
    q, k = I.norm_rope(c.q, c.k, **c.kw)
    out, lse = fdma.fwd(q, k, v, bias=bias, causal=True)
    dq, dk, dv, db = fdma.bwd(q, k, v, out, do, lse, bias=bias, causal=True)
    dt = I.rel_bias_bwd(db, starts, bidirectional=False, causal=True)
    dx, dy, dqw, dkw = I.norm_rope_bwd(c.q, c.k, dq, dk, **c.kw)

    x, y, wq, wk, t = (z.double().cpu().requires_grad_() for z in (c.q, c.k, c.w[0], c.w[1], table))
    cos, sin = (z.double().cpu()[:, None] for z in c.rope.unbind(1))

    def rows(x, w):
        z = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = z[..., :16], z[..., 16:32]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, z[..., 32:]), -1)

    Q, K = rows(x, wq), rows(y, wk).repeat_interleave(2, 2)
    at = torch.tensor(orc.buckets(N, N, starts, False, 0))
    S = torch.einsum("bihd,bjhd->bhij", Q, K) * d ** -0.5 + t[at].permute(2, 0, 1).repeat_interleave(2, 0)
    S = S.masked_fill(torch.triu(torch.ones(N, N, dtype=torch.bool), 1), float("-inf"))
    O = torch.einsum("bhij,bjhd->bihd", S.softmax(-1), v.double().cpu().repeat_interleave(2, 2))
    O.backward(do.double().cpu())
    for got, want in ((out, O.detach()), (dx, x.grad), (dy, y.grad), (dqw, wq.grad), (dkw, wk.grad), (dt, t.grad)):
        rel = (got.double().cpu() - want).norm() / want.norm()
        assert rel <= 1e-2 + 3 * 2.0 ** -8, rel


def test_a_bias_of_one_head_for_all(I):
    """A table of one head, its bias expanded over batch and kv heads: as a table with that column for each kv head."""
    from block_sparse_masked_02_gb300 import fdma

    B, N, Hq, Hk, d = 2, 160, 4, 2, 64
    g = torch.Generator().manual_seed(6)
    q, k, v, do = (_rows(g, B, N, H, d) for H in (Hq, Hk, Hk, Hq))
    starts = I.rel_starts(16, 64, bidirectional=False)
    table = torch.randn(16, 1, generator=g).cuda()
    res = []
    for t in (table, table.expand(16, Hk)):
        bias = I.rel_bias(t, N, N, starts, bidirectional=False).expand(B, Hk, -1, -1)
        out, lse = fdma.fwd(q, k, v, bias=bias, causal=True)
        db = fdma.bwd(q, k, v, out, do, lse, bias=bias, causal=True)[3]
        res.append((out, lse, I.rel_bias_bwd(db, starts, bidirectional=False, causal=True)))
    for x, y in zip(*res):
        assert torch.equal(x, y)
    assert res[0][2].shape == (16, Hk)


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_steps_from_a_captured_graph(I, fp8):
    """norm_rope_append and the attention over the cache, captured once and replayed for several steps: bit for bit what
    calls of their own give."""
    B, Hq, Hkv, d, steps = 3, 8, 2, 128, 4
    s = Serving(I, [1] * B, [14, 0, 40], Hq, Hkv, d, fp8=fp8, extra=1)
    s.rope = s.kw["rope"] = I.rope_table(64, d)
    s.table[:] = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)[:, :s.table.shape[1]]
    P = s.P
    num = B * 4
    fresh = lambda: P.empty_cache(num, 16, Hkv, d, dtype=E4M3 if fp8 else torch.bfloat16)  # noqa: E731
    g = torch.Generator().manual_seed(4)
    table = torch.arange(num, dtype=torch.int32, device="cuda").view(B, 4)
    prompt = [14, 1, 40]
    tokens = [_rows(g, B + 1, Hq + 2 * Hkv, d) for _ in range(steps)]
    first = _rows(g, sum(prompt), Hq + 2 * Hkv, d)
    cut = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])  # noqa: E731

    def begin():
        kc, vc, ke, ve = fresh()
        lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(prompt)]), dtype=torch.int32, device="cuda")
        P.norm_rope_append(*cut(first), kc, vc, table, lens, cu, k_exp=ke, v_exp=ve, **s.kw)
        return kc, vc, ke, ve, lens

    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")

    def step(x, c):
        kc, vc, ke, ve, lens = c
        lens += 1
        q = P.norm_rope_append(*cut(x), kc, vc, table, lens, cu, k_exp=ke, v_exp=ve, **s.kw)
        return P.fwd(q, kc, vc, table, lens, cu, 1, k_exp=ke, v_exp=ve)

    c = begin()
    want = [[y.clone() for y in step(x, c)] for x in tokens]
    c = begin()
    x = tokens[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, c)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, c)
    for a, b in zip(c, begin()):  # as it was before the warm-up
        if a is not None:
            a.copy_(b)
    for y, w in zip(tokens, want):
        x.copy_(y)
        graph.replay()
        assert torch.equal(out[0][:B], w[0][:B]) and torch.equal(out[1][:, :B], w[1][:, :B])


def test_two_captured_backward_passes_with_workspaces_of_their_own(I):
    starts = I.rel_starts(32, 128)
    g = torch.Generator().manual_seed(9)
    jobs = []
    for i in range(2):
        c = Case(I, 1, 700, 4, 2, 128, seed=20 + i)
        db = torch.randn(1, 2, 512, 1024, generator=g).bfloat16().cuda()
        ws = (I.norm_rope_bwd_workspace(c.q, c.k, q_weight=c.w[0], k_weight=c.w[1]), I.rel_bias_bwd_workspace(1, 2, 512, 1024, starts))
        jobs.append((c, db, ws))

    def run(job):
        c, db, ws = job
        return I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, workspace=ws[0], **c.kw) + (I.rel_bias_bwd(db, starts, workspace=ws[1]),)

    want = [[x.clone() for x in run(j)] for j in jobs]
    graphs, outs = [], []
    for j in jobs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(j))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x, y in zip(o, w):
            assert torch.equal(x, y)


def test_calls_on_another_stream(I):
    c = Case(I, 1, 2000, 8, 2, 128)
    starts = I.rel_starts(32, 128)
    db = torch.randn(1, 2, 1024, 1024, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    table = torch.randn(32, 2, generator=torch.Generator().manual_seed(2)).cuda()
    calls = [lambda **k: I.norm_rope(c.q, c.k, **c.kw, **k), lambda **k: I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **c.kw, **k),
             lambda **k: (I.rel_bias(table, 1024, 1024, starts, **k),), lambda **k: (I.rel_bias_bwd(db, starts, **k),)]
    want = [f() for f in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [f(stream=side) for f in calls]
    with torch.cuda.stream(side):
        got += [f() for f in calls]
    side.synchronize()
    for o, w in zip(got, want + want):
        for x, y in zip(o, w):
            assert torch.equal(x, y)


@pytest.mark.parametrize("raw", [True, False])
def test_backward_passes_without_workspaces_in_a_captured_graph(I, raw, monkeypatch):
    """What a call allocates for itself inside a capture lives as long as the graph: replays follow the inputs, and what is
    allocated between them changes nothing.  Also with a torch that lends no memory without a tensor around it."""
    if not raw:
        monkeypatch.setattr(I, "_raw_alloc", None)
    starts = I.rel_starts(32, 128)
    cases = [Case(I, 1, 700, 4, 2, 128, seed=30 + i) for i in range(3)]
    dbs = [torch.randn(1, 2, 512, 1024, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(3)]

    def run(c, db):
        return I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **c.kw) + (I.rel_bias_bwd(db, starts),)

    want = [[x.clone() for x in run(c, db)] for c, db in zip(cases, dbs)]
    now, db = Case(I, 1, 700, 4, 2, 128, seed=40), torch.zeros_like(dbs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(now, db)
    for c, d, w in list(zip(cases, dbs, want)) * 2:
        for x, y in ((now.q, c.q), (now.k, c.k), (now.dq, c.dq), (now.dk, c.dk), (now.w[0], c.w[0]), (now.w[1], c.w[1]), (db, d)):
            x.copy_(y)
        graph.replay()
        other = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 10, 1 << 16, 1 << 20)]
        for x, y in zip(out, w):
            assert torch.equal(x, y)
        del other
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = cases[0]
    got = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, stream=side, **c.kw) + (I.rel_bias_bwd(dbs[0], starts, stream=side),)
    side.synchronize()
    for x, y in zip(got, want[0]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (96, 32, False), (80, 80, True), (128, 24, False)])
def test_append_without_a_norm(I, fp8, d, rot, interleaved):
    s = Serving(I, [7, 1, 40], [9, 60, 0], 5, 3, d, fp8=fp8, rot=rot, weight=None, seed=d)
    kw = dict(rope=s.rope, interleaved=interleaved, norm=False)
    q_out = torch.full_like(s.q, 7.0)
    s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, q_out=q_out, **kw, **s.ex)
    n = 48
    positions = torch.tensor(s.pos[:n], dtype=torch.int32, device="cuda")
    q, k = I.norm_rope(s.q[:n], s.k[:n], positions=positions, **kw)
    assert torch.equal(q_out[:n], q) and (q_out[n:] == 7).all()
    t = _np(s.rope)[s.pos[:n]]
    (qr, qm), (kr, km) = [orc.norm_rope(_np(x[:n]), None, t[:, None, 0], t[:, None, 1], interleaved, False, 1e-6) for x in (s.q, s.k)]
    _check_rows(q, qr, qm, d)
    pg, sl = (torch.tensor(x, device="cuda") for x in s.slots())
    if not fp8:
        assert torch.equal(s.kc[pg, sl], k) and torch.equal(s.vc[pg, sl], s.v[:n])
        return
    code, byte = porc.quantise(_np(s.v[:n]))
    assert np.array_equal(s.vc.view(torch.uint8)[pg, sl].cpu().numpy(), code)
    assert np.array_equal(s.ve[pg, sl].cpu().numpy(), byte)
    # each code is the fp32 value rounded once: half a step of e4m3, of its least step where it has no normal code
    delta = (d / 2 + 12) * U * km
    e = s.ke[pg, sl].cpu().numpy().astype(np.float64)
    val = porc.dequantise(s.kc.view(torch.uint8)[pg, sl].cpu().numpy(), e.astype(np.uint8))
    tol = delta + np.maximum(2.0 ** -4 * (np.abs(kr) + delta), 2.0 ** -10 * 2.0 ** (e - 127)[..., None])
    assert (np.abs(val - kr) <= tol).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("news", [[5, 1, 33], [3000, 2500]])
def test_append_in_place(I, fp8, news):
    """q_out being q: short runs of a token's rows a warp, and whole tokens."""
    s = Serving(I, news, [9] * len(news), 6, 2, 64, fp8=fp8, rot=32)
    n = sum(news)
    q = s.q.clone()
    want = s.P.norm_rope_append(q, s.k, s.v, *s.at, s.cu, **s.kw, **s.ex)
    kc, vc = s.kc.clone(), s.vc.clone()
    behind = s.q[n:].clone()
    assert s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, q_out=s.q, **s.kw, **s.ex) is s.q
    assert torch.equal(s.q[:n], want[:n]) and torch.equal(s.q[n:], behind)
    pg, sl = (torch.tensor(x, device="cuda") for x in s.slots())
    for x, y in ((s.kc, kc), (s.vc, vc)):
        assert torch.equal(x[pg, sl].view(torch.uint8), y[pg, sl].view(torch.uint8))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,Hq,Hk,d,rot", [(40000, 16, 4, 128, 128), (30000, 21, 3, 104, 40)])
def test_rows_of_more_than_l2_holds_in_place(I, N, Hq, Hk, d, rot, interleaved):
    c = Case(I, 1, N, Hq, Hk, d, rot)
    pos = torch.randint(-N // 8, N, (N,), dtype=torch.int32, device="cuda")
    kw = dict(interleaved=interleaved, positions=pos, **c.kw)
    qo, ko = c.q.clone(), c.k.clone()
    I.norm_rope(c.q, c.k, q_out=qo, k_out=ko, **kw)
    grads = I.norm_rope_bwd(c.q, c.k, c.dq, c.dk, **kw)
    dq, dk = c.dq.clone(), c.dk.clone()
    got = I.norm_rope_bwd(c.q, c.k, dq, dk, grads=(dq, dk, None, None), **kw)
    assert got[0] is dq and got[1] is dk
    for x, y in zip(got, grads):
        assert torch.equal(x, y)
    I.norm_rope(c.q, c.k, q_out=c.q, k_out=c.k, **kw)
    assert torch.equal(c.q, qo) and torch.equal(c.k, ko)


@pytest.mark.parametrize("seed", range(32))
def test_random_appends(I, seed):
    """Every width of a cache's rows, any part of it turned, random batches and layouts: bit for bit what norm_rope and
    kv_append give (an e4m3 cache's keys, which take their codes from values that are rounded once less: within that of
    the codes' own bound)."""
    r = np.random.default_rng(3000 + seed)
    fp8 = seed % 4 == 3
    d = 16 * int(r.integers(1, 9)) if fp8 else 8 * (seed % 16 + 1)
    rot = 8 * int(r.integers(0, d // 8 + 1))
    Hq, Hkv = int(r.integers(1, 14)), int(r.integers(1, 7))
    inter, norm = bool(r.integers(0, 2)), bool(rot == 0 or r.integers(0, 4))
    weight = [None, "shared", "head"][seed % 3] if norm else None
    news = [int(2 ** r.uniform(0, 8)) - 1 for _ in range(int(r.integers(1, 8)))]
    olds = [int(r.integers(0, 100)) for _ in news]
    s = Serving(I, news, olds, Hq, Hkv, d, [16, 64][seed % 2], fp8, rot, weight, seed=seed, wdtype=[torch.float32, torch.bfloat16][seed % 2])
    kw, n = dict(interleaved=inter, norm=norm, **s.kw), sum(news)
    q_out = torch.full_like(s.q, 7.0)
    s.P.norm_rope_append(s.q, s.k, s.v, *s.at, s.cu, q_out=q_out, **kw, **s.ex)
    pos = torch.tensor(s.pos, dtype=torch.int32, device="cuda")
    q2, k2 = torch.full_like(s.q, 7.0), torch.zeros_like(s.k)
    I.norm_rope(s.q, s.k, positions=pos, q_out=q2, k_out=k2, **kw)
    assert torch.equal(q_out, q2)
    got = [x.clone() for x in (s.kc, s.vc, s.ke, s.ve) if x is not None]
    for x in (s.kc, s.vc):
        x.view(torch.uint8).fill_(0x55)
    if fp8:
        s.ke.fill_(9)
        s.ve.fill_(9)
    s.P.kv_append(k2, s.v, *s.at, s.cu, **s.ex)
    assert torch.equal(got[1].view(torch.uint8), s.vc.view(torch.uint8))
    if not fp8:
        assert torch.equal(got[0].view(torch.uint8), s.kc.view(torch.uint8))
        return
    assert torch.equal(got[3], s.ve)
    pg, sl = s.slots()
    keep = np.ones(s.kc.shape[:2], dtype=bool)
    keep[pg, sl] = False
    assert np.array_equal(got[0].view(torch.uint8).cpu().numpy()[keep], s.kc.view(torch.uint8).cpu().numpy()[keep])
    assert np.array_equal(got[2].cpu().numpy()[keep], s.ke.cpu().numpy()[keep])
    code, e = got[0].view(torch.uint8).cpu().numpy()[pg, sl], got[2].cpu().numpy()[pg, sl]
    # k2 is the fp32 value y to half a step of bf16: |y| <= |k2| (1 + 2^-7); the code is y to half a step of e4m3
    k = np.abs(_np(k2[:n])) * (1 + 2.0 ** -7) + 2.0 ** -133
    step = 2.0 ** (e.astype(np.float64) - 127)[..., None]
    tol = 2.0 ** -7 * k + 2.0 ** -133 + np.maximum(2.0 ** -4 * k, 2.0 ** -10 * step)
    assert (np.abs(porc.dequantise(code, e) - _np(k2[:n])) <= tol).all()
