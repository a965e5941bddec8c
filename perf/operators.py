"""The paged key/value cache operators, as cases to be measured.

Three operators of `block_sparse_masked_02_gb300.paged`:

  append   new tokens' K and V rows written into the pages of a cache, as bf16 or quantised to e4m3 with one
           power-of-two scale per (token, kv head);
  gather   ragged sequences read back from their pages into packed bf16 rows;
  fwd      attention of each sequence's newest tokens (one, a few, or a long chunk) over its pages, causal,
           optionally with a sliding window and a few first tokens that stay visible (sinks).

With `own` false, `run` computes them with elementary torch operations; with `own` true it calls the framework.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of eight sequences: the cache write of every decoding step (latency)
        dict(name="append_token_bf16", op="append", B=8, new_lo=1, new_hi=1, old_lo=100, old_hi=3001, Hkv=8, d=128,
             page=16, fp8=False),
        # the cache write of a ragged prefill, quantised, and the rows as attention will see them
        dict(name="append_prefill_e4m3", op="append", B=4, new_lo=1531, new_hi=8192, old_lo=0, old_hi=777, Hkv=8, d=128,
             page=64, fp8=True),
        # a long context read back for a masked or biased attention call over contiguous keys
        dict(name="gather_long_bf16", op="gather", B=2, len_lo=16384, len_hi=65536, Hkv=4, d=128, page=64, fp8=False),
        # many short sequences of a quantised cache read back
        dict(name="gather_short_e4m3", op="gather", B=32, len_lo=129, len_hi=2047, Hkv=8, d=64, page=16, fp8=True),
        # one token, one short sequence (latency)
        dict(name="token_one_short", op="fwd", B=1, new_lo=1, new_hi=1, len_lo=256, len_hi=256, Hq=2, Hkv=1, d=64, page=16,
             fp8=False, window=0, sinks=0),
        # one decoding step of a ragged batch
        dict(name="token_ragged_bf16", op="fwd", B=32, new_lo=1, new_hi=1, len_lo=257, len_hi=8191, Hq=32, Hkv=8, d=128,
             page=16, fp8=False, window=0, sinks=0),
        # one decoding step of few long contexts: the keys of one sequence have to be split over the machine
        dict(name="token_long_e4m3", op="fwd", B=2, new_lo=1, new_hi=1, len_lo=65521, len_hi=65536, Hq=16, Hkv=2, d=128,
             page=64, fp8=True, window=0, sinks=0),
        # one decoding step of a large batch with a sliding window and sinks
        dict(name="token_window_sinks", op="fwd", B=64, new_lo=1, new_hi=1, len_lo=2049, len_hi=16384, Hq=16, Hkv=4, d=128,
             page=64, fp8=False, window=2048, sinks=64),
        # five tokens a sequence (drafted tokens being verified) over a quantised cache
        dict(name="few_tokens_e4m3", op="fwd", B=16, new_lo=2, new_hi=5, len_lo=1000, len_hi=4096, Hq=32, Hkv=8, d=128,
             page=16, fp8=True, window=0, sinks=0),
        # a chunk of a long prompt
        dict(name="chunk_bf16", op="fwd", B=1, new_lo=2048, new_hi=2048, len_lo=16384, len_hi=16384, Hq=16, Hkv=4, d=128,
             page=64, fp8=False, window=0, sinks=0),
        # chunks of two prompts over a quantised cache
        dict(name="chunk_ragged_e4m3", op="fwd", B=2, new_lo=333, new_hi=1024, len_lo=4097, len_hi=8192, Hq=32, Hkv=8,
             d=128, page=16, fp8=True, window=0, sinks=0),
        # a chunk of a long prompt with a sliding window and sinks
        dict(name="chunk_window_sinks", op="fwd", B=1, new_lo=2048, new_hi=2048, len_lo=32768, len_hi=32768, Hq=32, Hkv=8,
             d=128, page=64, fp8=False, window=4096, sinks=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    page = rng.choice((16, 32, 64, 128))
    d = rng.choice((64, 80, 96, 128, 128, 128))
    fp8 = rng.random() < 0.5
    kind = rng.choice(("append", "gather", "token", "token", "few", "chunk"))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    G = rng.choice((1, 2, 3, 4, 6, 8))
    if kind == "append":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 16384 // B))
        old = _log(rng, 1, 4096)
        return dict(op="append", B=B, new_lo=rng.randint(1, hi), new_hi=hi, old_lo=rng.randint(0, old), old_hi=old, Hkv=Hkv,
                    d=d, page=page, fp8=fp8)
    if kind == "gather":
        B = _log(rng, 1, 64)
        hi = _log(rng, 64, 65536 // B)
        return dict(op="gather", B=B, len_lo=rng.randint(1, hi), len_hi=hi, Hkv=Hkv, d=d, page=page, fp8=fp8)
    if kind == "chunk":
        B = rng.choice((1, 1, 2, 3))
        new = _log(rng, 33, 2048 // B)
        hi = new + _log(rng, 1, 14000)
        lo = rng.randint(new, hi)
        Hkv, G = rng.choice((1, 2, 4)), min(G, 4)
    else:
        B = _log(rng, 1, 64)
        new = 1 if kind == "token" else rng.randint(2, 8)
        hi = _log(rng, 64, min(65536, 262144 // B))
        lo = rng.randint(min(new, hi), hi)
    window, sinks = 0, 0
    if rng.random() < 0.4:
        window = _log(rng, 32, 4096)
        sinks = rng.choice((0, 4, 64, 130))
    return dict(op="fwd", B=B, new_lo=rng.randint(1, new), new_hi=new, len_lo=max(lo, new), len_hi=max(hi, new), Hq=Hkv * G,
                Hkv=Hkv, d=d, page=page, fp8=fp8, window=window, sinks=sinks)


def _spread(B, lo, hi):
    """B lengths from hi down to lo, the longest first."""
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def _lengths(case):
    """(new tokens, keys) of each sequence after the new tokens' rows are in the cache."""
    B = case["B"]
    if case["op"] == "gather":
        return [0] * B, _spread(B, case["len_lo"], case["len_hi"])
    new = _spread(B, case["new_lo"], case["new_hi"])
    if case["op"] == "append":
        old = _spread(B, case["old_lo"], case["old_hi"])
        return new, [o + n for o, n in zip(reversed(old), new)]
    return new, [max(n, k) for n, k in zip(new, reversed(_spread(B, case["len_lo"], case["len_hi"])))]


# ------------------------------------------------------------------------------------------------ inputs
def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _codes(x):
    """Rows of x as e4m3 codes and the biased exponent of their power-of-two scale."""
    m, e = torch.frexp(x.abs().amax(-1).float())  # amax = m 2^e with m in [1/2, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)  # the least power of two whose 448-fold reaches amax
    e = torch.where(m == 0, -126, e).clamp(-126, 119)
    return torch.ldexp(x.float(), -e[..., None]).to(E4M3), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    new, keys = _lengths(case)
    pages = [-(-k // page) for k in keys]
    per, total = max(pages), sum(pages)
    # every sequence's pages, scattered over the cache; entries behind its last page are not read
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1]
    col = torch.arange(per, device="cuda")
    used = col[None] < torch.tensor(pages, device="cuda")[:, None]
    table = torch.where(used, ids[(first[:, None] + col[None]).clamp(max=total - 1)], -1)

    def rows(*shape):
        # unit rows of uneven size, as the key and value projections give
        x = torch.randn(*shape, generator=g, device="cuda")
        return (x * torch.exp(0.25 * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))).bfloat16()

    s = dict(case=case, table=table.contiguous(), k_lens=torch.tensor(keys, dtype=torch.int32, device="cuda"),
             cu_q=_offsets(new), max_q=max(new), k_exp=None, v_exp=None, keys=keys)
    shape = (total, Hkv, page, d)  # a page holds each head's rows together
    if case["op"] == "append":
        T = sum(new)
        s["k"], s["v"] = rows(T, Hkv, d), rows(T, Hkv, d)
        dt = E4M3 if case["fp8"] else torch.bfloat16
        s["k_cache"] = torch.zeros(shape, dtype=dt, device="cuda").permute(0, 2, 1, 3)
        s["v_cache"] = torch.zeros(shape, dtype=dt, device="cuda").permute(0, 2, 1, 3)
        if case["fp8"]:
            s["k_exp"] = torch.zeros(shape[:3], dtype=torch.uint8, device="cuda").permute(0, 2, 1)
            s["v_exp"] = torch.zeros(shape[:3], dtype=torch.uint8, device="cuda").permute(0, 2, 1)
        s["first"] = s["k_lens"] - (s["cu_q"][1:] - s["cu_q"][:-1])
        s["T"] = T
        return s
    for name in ("k", "v"):
        x = rows(*shape)
        if case["fp8"]:
            x, e = _codes(x)
            s[name + "_exp"] = e.permute(0, 2, 1)
        s[name + "_cache"] = x.permute(0, 2, 1, 3)
    if case["op"] == "gather":
        s["cu_k"], s["T"] = _offsets(keys), sum(keys)
    else:
        s["q"] = torch.randn(sum(new), case["Hq"], d, generator=g, device="cuda").bfloat16()
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        from block_sparse_masked_02_gb300 import paged

        at = (s["k_cache"], s["v_cache"], s["table"], s["k_lens"])
        ex = dict(k_exp=s["k_exp"], v_exp=s["v_exp"])
        if c["op"] == "append":
            paged.kv_append(s["k"], s["v"], *at, s["cu_q"], **ex)
            if not c["fp8"]:
                return s["k_cache"], s["v_cache"]
            # what is held in 8 bits, as the values it stands for, and the scales' exponents
            return paged.kv_gather(*at, s["cu_q"], s["T"], first=s["first"], **ex) + (s["k_exp"], s["v_exp"])
        if c["op"] == "gather":
            return paged.kv_gather(*at, s["cu_k"], s["T"], **ex)
        return paged.fwd(s["q"], *at, s["cu_q"], s["max_q"], window=c["window"], sinks=c["sinks"], **ex)
    if c["op"] == "append":
        return _append(s)
    if c["op"] == "gather":
        return _gather(s, s["cu_k"], None)
    return _attend(s)


def _tokens(cu, T):
    """Sequence and index within it of each of T packed tokens."""
    t = torch.arange(T, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, t - cu[b]


def _slots(s, b, pos):
    page = s["case"]["page"]
    return s["table"][b, pos // page].long(), (pos % page).long()


def _append(s):
    n = s["cu_q"][1:] - s["cu_q"][:-1]
    b, i = _tokens(s["cu_q"], s["T"])
    p, o = _slots(s, b, (s["k_lens"] - n)[b] + i)
    if not s["case"]["fp8"]:
        s["k_cache"][p, o], s["v_cache"][p, o] = s["k"], s["v"]
        return s["k_cache"], s["v_cache"]
    for name in ("k", "v"):
        code, e = _codes(s[name])
        s[name + "_cache"].view(torch.uint8)[p, o] = code.view(torch.uint8)
        s[name + "_exp"][p, o] = e
    return _gather(s, s["cu_q"], s["first"]) + (s["k_exp"], s["v_exp"])


def _gather(s, cu, first):
    b, pos = _tokens(cu, s["T"])
    p, o = _slots(s, b, pos if first is None else first[b] + pos)
    return _values(s, "k", (p, o)).bfloat16(), _values(s, "v", (p, o)).bfloat16()


def _values(s, name, at):
    """Rows of a cache in fp32: the codes times their scales where it holds 8 bits."""
    if s[name + "_exp"] is None:
        return s[name + "_cache"][at].float()
    code = s[name + "_cache"].view(torch.uint8)[at].view(E4M3).float()
    return torch.ldexp(code, s[name + "_exp"][at].int()[..., None] - 127)


def _attend(s):
    c = s["case"]
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G, per = Hq // Hkv, s["table"].shape[1]
    L, M = per * page, s["max_q"]
    at = (s["table"].clamp(min=0).long(),)
    K = _values(s, "k", at).reshape(B, L, Hkv, d).permute(0, 2, 3, 1)
    V = _values(s, "v", at).reshape(B, L, Hkv, d).permute(0, 2, 1, 3)
    n = (s["cu_q"][1:] - s["cu_q"][:-1])[:, None]
    i = torch.arange(M, device="cuda")[None]
    row = (s["cu_q"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    pos = s["k_lens"][:, None] - n + i  # (B, M)
    q = s["q"][row].float().view(B, M, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * M, d)
    S = (q @ K).view(B, Hkv, G, M, L) * (d ** -0.5)
    j = torch.arange(L, device="cuda")
    keep = j <= pos[..., None]
    if c["window"]:
        keep &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    S.masked_fill_(~keep[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    P = S.sub_(m).exp_()
    total = P.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)  # (B, Hkv, G, M)
    # keys that nobody sees may hold anything: their weight is zero and so is their product
    V = torch.where((j < s["k_lens"][:, None])[:, None, :, None], V, 0)
    O = (P.view(B, Hkv, G * M, L) @ V).view(B, Hkv, G, M, d) / total
    b, t = _tokens(s["cu_q"], s["q"].shape[0])
    out = O.permute(0, 3, 1, 2, 4).reshape(B, M, Hq, d)[b, t.long()].bfloat16()
    return out, lse.permute(0, 3, 1, 2).reshape(B, M, Hq)[b, t.long()].T.contiguous()


# ------------------------------------------------------------------------------------------------ work
def work(case):
    new, keys = _lengths(case)
    Hkv, d = case["Hkv"], case["d"]
    stored = Hkv * 2 * (d + 1 if case["fp8"] else 2 * d)  # one token's K and V rows in the cache
    plain = Hkv * 2 * 2 * d
    table = 4 * sum(-(-k // case["page"]) for k in keys)
    if case["op"] == "append":
        T = sum(new)
        # rows in, rows stored; the quantised rows are read back once more to return their values
        return dict(bytes=T * (plain + stored) + (T * (plain + stored) if case["fp8"] else 0), flops=T * Hkv * 2 * d)
    if case["op"] == "gather":
        return dict(bytes=sum(keys) * (plain + stored) + table, flops=sum(keys) * Hkv * 2 * d)
    w, z, Hq = case["window"], case["sinks"], case["Hq"]
    seen, pairs = 0, 0
    for n, k in zip(new, keys):
        if not w:
            seen += k
            pairs += n * (k - n) + n * (n + 1) // 2
            continue
        low = max(0, k - n - w + 1)
        seen += k - low + min(z, low)
        for p in range(k - n, k):
            low = max(0, p - w + 1)
            pairs += p + 1 - low + min(z, low)
    T = sum(new)
    return dict(bytes=T * Hq * (4 * d + 4) + seen * stored, flops=pairs * Hq * 4 * d)


# ------------------------------------------------------------------------------------------------ 64 bits
def _e4m3(x):
    """x (64 bits) rounded to the nearest number of e4m3, ties to even, at most 448 in size."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _stored(s, name, b):
    """The first keys[b] rows of sequence b, in 64 bits."""
    c, n = s["case"], s["keys"][b]
    ids = s["table"][b, : -(-n // c["page"])].long()
    x = s[name + "_cache"]
    if c["fp8"]:
        x = x.view(torch.uint8)[ids].view(E4M3).double() * torch.exp2(s[name + "_exp"][ids].double() - 127)[..., None]
    else:
        x = x[ids].double()
    return x.reshape(-1, c["Hkv"], c["d"])[:n]


def exact(case, seed):
    s = prepare(case, seed)
    new, keys = _lengths(case)
    if case["op"] == "gather":
        return tuple(torch.cat([_stored(s, x, b) for b in range(case["B"])]) for x in ("k", "v"))
    cu = s["cu_q"].tolist()
    if case["op"] == "append":
        rows, scales = [], []
        for name in ("k", "v"):
            x = s[name].double()
            if case["fp8"]:
                top = x.abs().amax(-1, keepdim=True)
                e = torch.floor(torch.log2(top / 448))  # raised by one where 448 of it do not reach
                e = torch.where(torch.exp2(e) * 448 < top, e + 1, e).clamp(-126, 119)
                x = _e4m3(x / torch.exp2(e)) * torch.exp2(e)
                to, vals = torch.zeros(s[name + "_exp"].shape, device="cuda"), e.squeeze(-1) + 127
            else:
                to, vals = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device="cuda"), x
            for b in range(case["B"]):
                at = torch.arange(keys[b] - new[b], keys[b], device="cuda")
                to[s["table"][b, at // case["page"]].long(), at % case["page"]] = vals[cu[b]:cu[b + 1]].to(to.dtype)
            rows.append(x)
            scales.append(to)
        return tuple(rows) + tuple(x.to(torch.uint8) for x in scales) if case["fp8"] else tuple(scales)
    Hq, Hkv, d, w, z = case["Hq"], case["Hkv"], case["d"], case["window"], case["sinks"]
    G, T = Hq // Hkv, s["q"].shape[0]
    out = torch.empty(T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(Hq, T, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        K, V = _stored(s, "k", b), _stored(s, "v", b)
        j = torch.arange(keys[b], device="cuda")
        p = torch.arange(keys[b] - new[b], keys[b], device="cuda")[:, None]
        hidden = j > p
        if w:
            hidden |= (j <= p - w) & (j >= z)
        for h in range(Hq):
            x = (s["q"][cu[b]:cu[b + 1], h].double() @ K[:, h // G].T) / math.sqrt(d)
            x[hidden] = -math.inf
            lse[h, cu[b]:cu[b + 1]] = torch.logsumexp(x, -1)
            out[cu[b]:cu[b + 1], h] = torch.softmax(x, -1) @ V[:, h // G]
    return out, lse
