"""What goes into attention, as cases to be measured.

Five operators, of `block_sparse_masked_02_gb300.inputs` and (append) of `.paged`:

  norm_rope       queries and keys, each head's row divided by its root mean square, times a learned weight, and turned
                  by the angle of its position, in one pass;
  norm_rope_bwd   its gradients: of the rows and of the weights;
  append          the same for the new tokens of a serving step, with the keys (and the values as they are) written into
                  the pages of a cache, bf16 or e4m3 with one power-of-two scale for each row;
  rel_bias        a learned bias by buckets of the distance between query and key, as the bias that attention reads;
  rel_bias_bwd    the gradient of its table from the gradient of that bias.

With `own` false, `run` computes them with elementary torch operations; with `own` true it calls the framework.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # queries and keys of a long training sequence, slices of one projection
        dict(name="rope_train", op="norm_rope", B=1, N=16384, Hq=16, Hkv=4, d=128, rot=128, pairs="halves", weight="shared",
             wdtype="bf16", docs=0),
        # a few documents packed into two short rows, adjacent pairs, a third of the columns turned, a weight for each head
        dict(name="rope_docs_partial", op="norm_rope", B=2, N=333, Hq=6, Hkv=2, d=96, rot=32, pairs="adjacent", weight="head",
             wdtype="fp32", docs=3),
        # the backward pass of the long training sequence
        dict(name="rope_bwd_train", op="norm_rope_bwd", B=1, N=16384, Hq=16, Hkv=4, d=128, rot=128, pairs="halves",
             weight="shared", wdtype="bf16", docs=0),
        # two sequences, a weight for each head
        dict(name="rope_bwd_heads", op="norm_rope_bwd", B=2, N=4096, Hq=32, Hkv=8, d=128, rot=64, pairs="halves",
             weight="head", wdtype="fp32", docs=0),
        # a small odd batch: norms alone, as beside a learned bias
        dict(name="rope_bwd_small", op="norm_rope_bwd", B=3, N=257, Hq=5, Hkv=5, d=80, rot=0, pairs="halves", weight="shared",
             wdtype="fp32", docs=0),
        # one new token of one sequence (latency)
        dict(name="append_one", op="append", B=1, new_lo=1, new_hi=1, old_lo=4000, old_hi=4000, Hq=16, Hkv=4, d=128, rot=128,
             pairs="halves", weight="shared", wdtype="bf16", page=64, fp8=False),
        # one decoding step of a batch, quantised
        dict(name="append_step_e4m3", op="append", B=32, new_lo=1, new_hi=1, old_lo=257, old_hi=8191, Hq=32, Hkv=8, d=128,
             rot=128, pairs="halves", weight="shared", wdtype="bf16", page=16, fp8=True),
        # four ragged prompts
        dict(name="append_prompts", op="append", B=4, new_lo=1531, new_hi=8192, old_lo=0, old_hi=777, Hq=32, Hkv=8, d=128,
             rot=128, pairs="halves", weight="shared", wdtype="bf16", page=64, fp8=False),
        # the bias of a long training sequence
        dict(name="bias_train", op="rel_bias", H=4, Nq=16384, Nk=16384, buckets=32, far=128, two_sided=False, tdtype="bf16"),
        # a few new queries over the keys so far (latency)
        dict(name="bias_rows", op="rel_bias", H=8, Nq=5, Nk=4096, buckets=32, far=128, two_sided=False, tdtype="fp32"),
        # the gradient of the table of the long training sequence
        dict(name="bias_bwd_train", op="rel_bias_bwd", B=1, H=4, Nq=16384, Nk=16384, buckets=32, far=128, two_sided=False,
             causal=True),
        # an encoder's: both directions, a batch, odd sizes, distances told apart up to 800
        dict(name="bias_bwd_batch", op="rel_bias_bwd", B=3, H=6, Nq=1001, Nk=1528, buckets=64, far=800, two_sided=True,
             causal=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "norm_rope_bwd", "append", "rel_bias", "rel_bias_bwd"))
    if op in ("rel_bias", "rel_bias_bwd"):
        H = rng.choice((1, 2, 4, 5, 8))
        B = 1 if op == "rel_bias" else rng.choice((1, 1, 2, 3))
        Nq = _log(rng, 1, 16384)
        Nk = 8 * _log(rng, 1, max(1, min(16384, (1 << 30) // (B * H * Nq)) // 8))
        two = rng.random() < 0.5
        case = dict(op=op, H=H, Nq=Nq, Nk=Nk, buckets=rng.choice((16, 32, 32, 64, 128)), far=_log(rng, 96, 2048), two_sided=two)
        if op == "rel_bias":
            return dict(case, tdtype=rng.choice(("fp32", "bf16")))
        return dict(case, B=B, causal=not two and rng.random() < 0.7)
    d = rng.choice((64, 80, 96, 128, 128, 128) if op == "append" else (64, 80, 96, 128, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    Hq = Hkv * rng.choice((1, 2, 3, 4, 6, 8))
    case = dict(op=op, Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice((0, d // 16 * 8, d, d, d)), pairs=rng.choice(("halves", "adjacent")),
                weight=rng.choice(("shared", "shared", "head", "none")), wdtype=rng.choice(("fp32", "bf16")))
    # values of all rows, at most as many as the largest listed case has
    most = (20 << 20) // ((Hq + 2 * Hkv) * d) * 2
    if op == "append":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(16384, most) // B))
        old = _log(rng, 1, 4096)
        return dict(case, B=B, new_lo=rng.randint(1, hi), new_hi=hi, old_lo=rng.randint(0, old), old_hi=old,
                    page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5)
    B = rng.choice((1, 1, 2, 3))
    return dict(case, B=B, N=_log(rng, 1, max(1, min(32768, most) // B)), docs=rng.choice((0, 0, 1, 4)))


def _spread(B, lo, hi):
    """B lengths from hi down to lo, the longest first."""
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def _lengths(case):
    """(new tokens, keys) of each sequence when the new tokens' rows are in the cache."""
    new = _spread(case["B"], case["new_lo"], case["new_hi"])
    old = _spread(case["B"], case["old_lo"], case["old_hi"])
    return new, [o + n for o, n in zip(reversed(old), new)]


# ------------------------------------------------------------------------------------------------ inputs
def _starts(case):
    """The first distance of each bucket of one side: one each up to half of them, the others evenly in the logarithm up to
    `far`.  Borders are found in whole numbers: distance a is in bucket e + k or behind where
    (a / e)^m >= (far / e)^k."""
    n = case["buckets"] // 2 if case["two_sided"] else case["buckets"]
    e, far = n // 2, case["far"]
    m = n - e
    at = list(range(e))
    for k in range(m):
        a = at[-1] + 1 if k == 0 else at[-1]
        while a ** m * e ** k < far ** k * e ** m:
            a += 1
        at.append(a)
    return tuple(at)


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _angles(length, rot):
    """Cosines and sines of rot / 2 angles of each position, (length, 2, rot / 2)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)

    def randn(*shape, **kw):
        return torch.randn(*shape, generator=g, device="cuda", **kw)

    if case["op"] in ("rel_bias", "rel_bias_bwd"):
        s["starts"] = _starts(case)
        if case["op"] == "rel_bias":
            s["table"] = randn(case["buckets"], case["H"]).to(torch.bfloat16 if case["tdtype"] == "bf16" else torch.float32)
        else:
            x = randn(case["B"], case["H"], case["Nq"], case["Nk"], dtype=torch.bfloat16)
            # zeros behind the diagonal if causal, as attention's backward pass writes it
            s["dbias"] = x.tril_(case["Nk"] - case["Nq"]) if case["causal"] else x
        return s
    Hq, Hkv, d, rot = case["Hq"], case["Hkv"], case["d"], case["rot"]
    for name, H in (("q_weight", Hq), ("k_weight", Hkv)):
        w = 1 + 0.2 * randn(*((H, d) if case["weight"] == "head" else (d,)))
        s[name] = None if case["weight"] == "none" else w.to(torch.bfloat16 if case["wdtype"] == "bf16" else torch.float32)

    def rows(*shape):
        # rows of uneven size, as the projections give
        return (randn(*shape) * torch.exp(0.5 * randn(*shape[:-1], 1))).bfloat16()

    if case["op"] == "append":
        page = case["page"]
        new, keys = _lengths(case)
        pages = [-(-k // page) for k in keys]
        total = sum(pages)
        # every sequence's pages, scattered over the cache; entries behind its last page are not read
        ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        first = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1]
        col = torch.arange(max(pages), device="cuda")
        used = col[None] < torch.tensor(pages, device="cuda")[:, None]
        s["page_table"] = torch.where(used, ids[(first[:, None] + col[None]).clamp(max=total - 1)], -1).contiguous()
        s["k_lens"], s["cu_q"] = torch.tensor(keys, dtype=torch.int32, device="cuda"), _offsets(new)
        s["rope"] = _angles(max(keys), rot) if rot else None
        T = sum(new)
        x = rows(T, Hq + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        shape = (total, Hkv, page, d)  # a page holds each head's rows together
        for name in ("k", "v"):
            s[name + "_cache"] = torch.zeros(shape, dtype=E4M3 if case["fp8"] else torch.bfloat16, device="cuda").transpose(1, 2)
            s[name + "_exp"] = torch.zeros(shape[:3], dtype=torch.uint8, device="cuda").transpose(1, 2) if case["fp8"] else None
        s["first"], s["T"] = s["k_lens"] - (s["cu_q"][1:] - s["cu_q"][:-1]), T
        return s
    B, N = case["B"], case["N"]
    x = rows(B, N, Hq + 2 * Hkv, d)
    s["q"], s["k"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    s["positions"] = None
    if case["docs"]:  # documents packed into a row: each begins at position 0
        cut = torch.sort(torch.randint(0, N, (B, case["docs"]), generator=g, device="cuda")).values
        n = torch.arange(N, device="cuda").expand(B, N).contiguous()
        at = torch.searchsorted(cut, n, right=True) - 1
        s["positions"] = torch.where(at < 0, n, n - cut.gather(1, at.clamp(min=0))).to(torch.int32)
    s["rope"] = _angles(N, rot) if rot else None
    if case["op"] == "norm_rope_bwd":
        s["dq_out"], s["dk_out"] = (0.1 * randn(B, N, Hq, d)).bfloat16(), (0.1 * randn(B, N, Hkv, d)).bfloat16()
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        from block_sparse_masked_02_gb300 import inputs, paged

        if c["op"] == "rel_bias":
            return inputs.rel_bias(s["table"], c["Nq"], c["Nk"], s["starts"], bidirectional=c["two_sided"])
        if c["op"] == "rel_bias_bwd":
            return inputs.rel_bias_bwd(s["dbias"], s["starts"], bidirectional=c["two_sided"], causal=c["causal"])
        kw = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], rope=s["rope"], interleaved=c["pairs"] == "adjacent", eps=EPS)
        if c["op"] == "norm_rope":
            return inputs.norm_rope(s["q"], s["k"], positions=s["positions"], **kw)
        if c["op"] == "norm_rope_bwd":
            return inputs.norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], positions=s["positions"], **kw)
        at = (s["k_cache"], s["v_cache"], s["page_table"], s["k_lens"])
        ex = dict(k_exp=s["k_exp"], v_exp=s["v_exp"])
        q = paged.norm_rope_append(s["q"], s["k"], s["v"], *at, s["cu_q"], **kw, **ex)
        if not c["fp8"]:
            return q, s["k_cache"], s["v_cache"]
        # what is held in 8 bits, as the values it stands for
        return (q,) + tuple(paged.kv_gather(*at, s["cu_q"], s["T"], first=s["first"], **ex))
    if c["op"] == "rel_bias":
        return _rel_bias(s)
    if c["op"] == "rel_bias_bwd":
        return _rel_bias_bwd(s)
    if c["op"] == "append":
        return _append(s)
    cos, sin = _turns(s, s["positions"], c["N"])
    if c["op"] == "norm_rope":
        return tuple(_forward(s[x].float(), s[x + "_weight"], cos, sin, c).bfloat16() for x in ("q", "k"))
    dq, dqw = _backward(s["q"], s["dq_out"], s["q_weight"], cos, sin, c)
    dk, dkw = _backward(s["k"], s["dk_out"], s["k_weight"], cos, sin, c)
    return dq, dk, dqw, dkw


def _turns(s, positions, N):
    """Cosines and sines of every token, with an axis for the heads."""
    if s["rope"] is None:
        return None, None
    t = s["rope"][:N] if positions is None else s["rope"][positions.long()]
    return t[..., 0, :].unsqueeze(-2), t[..., 1, :].unsqueeze(-2)


def _split(y, c):
    r = c["rot"]
    if c["pairs"] == "halves":
        return y[..., :r // 2], y[..., r // 2:r]
    return y[..., 0:r:2], y[..., 1:r:2]


def _join(a, b, y, c):
    both = torch.cat((a, b), -1) if c["pairs"] == "halves" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((both, y[..., c["rot"]:]), -1)


def _forward(x, w, cos, sin, c):
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    if w is not None:
        y = y * w.float()
    if cos is None:
        return y
    a, b = _split(y, c)
    return _join(a * cos - b * sin, b * cos + a * sin, y, c)


def _backward(x, dout, w, cos, sin, c):
    x, g = x.float(), dout.float()
    if cos is not None:
        a, b = _split(g, c)
        g = _join(a * cos + b * sin, b * cos - a * sin, g, c)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat = x * r
    dw = None
    if w is not None:
        dw = (g * xhat).sum((0, 1) if c["weight"] == "head" else (0, 1, 2), dtype=torch.float64).float()
        g = g * w.float()
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    return dx.bfloat16(), dw


def _tokens(cu, T):
    """Sequence and index within it of each of T packed tokens."""
    t = torch.arange(T, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b]


def _codes(x):
    """Rows of x (fp32) as e4m3 codes and the biased exponent of their power-of-two scale."""
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m 2^e with m in [1/2, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)  # the least power of two whose 448-fold reaches amax
    e = torch.where(m == 0, -126, e).clamp(-126, 119)
    return torch.ldexp(x, -e[..., None]).to(E4M3), e


def _append(s):
    c = s["case"]
    b, i = _tokens(s["cu_q"], s["T"])
    pos = s["first"][b] + i
    p, o = s["page_table"][b, pos // c["page"]].long(), (pos % c["page"]).long()
    cos, sin = _turns(s, pos, 0)
    q = _forward(s["q"].float(), s["q_weight"], cos, sin, c).bfloat16()
    k = _forward(s["k"].float(), s["k_weight"], cos, sin, c)
    if not c["fp8"]:
        s["k_cache"][p, o], s["v_cache"][p, o] = k.bfloat16(), s["v"]
        return q, s["k_cache"], s["v_cache"]
    (kc, ke), (vc, ve) = _codes(k), _codes(s["v"].float())
    s["k_cache"].view(torch.uint8)[p, o], s["v_cache"].view(torch.uint8)[p, o] = kc.view(torch.uint8), vc.view(torch.uint8)
    s["k_exp"][p, o], s["v_exp"][p, o] = (ke + 127).to(torch.uint8), (ve + 127).to(torch.uint8)
    return q, torch.ldexp(kc.float(), ke[..., None]).bfloat16(), torch.ldexp(vc.float(), ve[..., None]).bfloat16()


def _bucket(s, delta):
    """Buckets of distances delta = key - query."""
    starts = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
    a = delta.abs() if s["case"]["two_sided"] else (-delta).clamp(min=0)
    at = torch.bucketize(a, starts, right=True, out_int32=True) - 1
    return at + len(s["starts"]) * (delta > 0).int() if s["case"]["two_sided"] else at


def _rel_bias(s):
    c = s["case"]
    i = torch.arange(c["Nq"], device="cuda", dtype=torch.int32)[:, None] + (c["Nk"] - c["Nq"])
    at = _bucket(s, torch.arange(c["Nk"], device="cuda", dtype=torch.int32) - i)
    return s["table"].float().T[:, at].bfloat16()[None]


def _rel_bias_bwd(s):
    c, x = s["case"], s["dbias"]
    B, H, Nq, Nk = x.shape
    # rows of width Nq + Nk read as rows of one less: column j - i + Nq - 1 of every row is one diagonal
    x = torch.nn.functional.pad(x.flip(2), (0, Nq)).view(B, H, -1)[..., :Nq * (Nq + Nk - 1)].view(B, H, Nq, Nq + Nk - 1)
    diagonal = x.sum((0, 2), dtype=torch.float64)
    delta = torch.arange(1 - Nq, Nk, device="cuda", dtype=torch.int32) - (Nk - Nq)
    if c["causal"]:
        diagonal = torch.where(delta > 0, 0, diagonal)
    of = torch.nn.functional.one_hot(_bucket(s, delta).long(), c["buckets"]).double()
    return (of.T @ diagonal.T).float()


# ------------------------------------------------------------------------------------------------ work
def work(case):
    if case["op"] == "rel_bias":
        n = case["H"] * case["Nq"] * case["Nk"]
        return dict(bytes=2 * n + case["H"] * case["buckets"] * 4, flops=n)
    if case["op"] == "rel_bias_bwd":
        Nq, Nk = case["Nq"], case["Nk"]
        n = sum(min(Nk, max(0, Nk - Nq + i + 1)) for i in range(Nq)) if case["causal"] else Nq * Nk
        n *= case["B"] * case["H"]
        return dict(bytes=2 * n + case["H"] * case["buckets"] * 4, flops=n)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    weights = {"none": 0, "shared": 2, "head": Hq + Hkv}[case["weight"]] * d * (2 if case["wdtype"] == "bf16" else 4)
    if case["op"] == "append":
        new, keys = _lengths(case)
        T = sum(new)
        stored = Hkv * 2 * (d + 1 if case["fp8"] else 2 * d)  # one token's K and V rows in the cache
        rows = T * (2 * Hq * d * 2 + 2 * Hkv * d * 2 + stored)
        if case["fp8"]:  # read back once more to return their values
            rows += T * (stored + 2 * Hkv * d * 2)
        return dict(bytes=rows + weights + 4 * min(T, max(keys)) * case["rot"], flops=T * (Hq + Hkv) * d * 8)
    T = case["B"] * case["N"]
    rows = T * (Hq + Hkv) * d * 2
    back = case["op"] == "norm_rope_bwd"
    grads = 0 if case["weight"] == "none" else weights // (2 if case["wdtype"] == "bf16" else 4) * 4
    return dict(bytes=rows * (3 if back else 2) + weights + (grads if back else 0) + 4 * case["N"] * case["rot"] +
                (4 * T if case["docs"] else 0), flops=T * (Hq + Hkv) * d * (20 if back else 8))


# ------------------------------------------------------------------------------------------------ 64 bits
def _exact_turn(y, t, c, sign):
    """Rows y (..., H, d) turned pair by pair with the angles t (..., 2, rot / 2); sign -1 turns back."""
    z = y.clone()
    r = c["rot"]
    p = torch.arange(r // 2, device="cuda")
    at, to = (p, p + r // 2) if c["pairs"] == "halves" else (2 * p, 2 * p + 1)
    cos, sin = t[..., None, 0, :].double(), sign * t[..., None, 1, :].double()
    z[..., at] = y[..., at] * cos - y[..., to] * sin
    z[..., to] = y[..., to] * cos + y[..., at] * sin
    return z


def _exact_rows(x, w, t, c):
    x = x.double()
    y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS)
    y = y if w is None else y * w.double()
    return y if t is None else _exact_turn(y, t, c, 1)


def _exact_grads(x, dout, w, t, c):
    x, g = x.double(), dout.double()
    g = g if t is None else _exact_turn(g, t, c, -1)
    rms = torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS)
    dw = None
    if w is not None:
        dw = (g * x / rms).flatten(0, 1).sum(0)
        dw = dw if c["weight"] == "head" else dw.sum(0)
        g = g * w.double()
    return g / rms - x * (g * x).sum(-1, keepdim=True) / (c["d"] * rms ** 3), dw


def _exact_side(a, n, far):
    """The bucket of distance a (64 bits, whole) among the n of one side."""
    e = n // 2
    up = torch.floor(torch.log(a.clamp(min=e) / e) / math.log(far / e) * (n - e) + 1e-9)
    return torch.where(a < e, a, (e + up).clamp(max=n - 1)).long()


def _exact_bucket(c, delta):
    if not c["two_sided"]:
        return _exact_side((-delta).clamp(min=0).double(), c["buckets"], c["far"])
    n = c["buckets"] // 2
    return _exact_side(delta.abs().double(), n, c["far"]) + torch.where(delta > 0, n, 0)


def _e4m3(x):
    """x (64 bits) rounded to the nearest number of e4m3, ties to even, at most 448 in size."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_stored(x):
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top / 448))  # raised by one where 448 of it do not reach
    e = torch.where(torch.exp2(e) * 448 < top, e + 1, e).clamp(-126, 119)
    return _e4m3(x / torch.exp2(e)) * torch.exp2(e)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] in ("rel_bias", "rel_bias_bwd"):
        i = torch.arange(c["Nq"], device="cuda")[:, None] + (c["Nk"] - c["Nq"])
        delta = torch.arange(c["Nk"], device="cuda") - i
        at = _exact_bucket(c, delta)
        if c["op"] == "rel_bias":
            return torch.stack([s["table"][:, h].double()[at] for h in range(c["H"])])[None]
        out = torch.zeros(c["buckets"], c["H"], dtype=torch.float64, device="cuda")
        for h in range(c["H"]):
            x = s["dbias"][:, h].sum(0, dtype=torch.float64)
            if c["causal"]:
                x = torch.where(delta > 0, 0, x)
            for k in range(c["buckets"]):
                out[k, h] = torch.where(at == k, x, 0).sum()
        return out
    if c["op"] != "append":
        pos = torch.arange(c["N"], device="cuda").expand(c["B"], -1) if s["positions"] is None else s["positions"]
        t = None if s["rope"] is None else s["rope"][pos.long()]
        if c["op"] == "norm_rope":
            return tuple(_exact_rows(s[x], s[x + "_weight"], t, c) for x in ("q", "k"))
        (dq, dqw), (dk, dkw) = (_exact_grads(s[x], s["d" + x + "_out"], s[x + "_weight"], t, c) for x in ("q", "k"))
        return dq, dk, dqw, dkw
    new, keys = _lengths(c)
    pos = torch.cat([torch.arange(n - m, n, device="cuda") for m, n in zip(new, keys)])
    t = None if s["rope"] is None else s["rope"][pos]
    q, k, v = _exact_rows(s["q"], s["q_weight"], t, c), _exact_rows(s["k"], s["k_weight"], t, c), s["v"].double()
    if c["fp8"]:
        return q, _exact_stored(k), _exact_stored(v)
    out, at = [q], s["cu_q"].tolist()
    for x, name in ((k, "k_cache"), (v, "v_cache")):
        to = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            p = pos[at[b]:at[b + 1]]
            to[s["page_table"][b, p // c["page"]].long(), p % c["page"]] = x[at[b]:at[b + 1]]
        out.append(to)
    return tuple(out)
