"""What the operators of capped, document- and prefix-masked attention and of the 8-bit key/value cache cost.

Four operators, each in its plain form (``own`` false: elementary torch
operations in 32 bits) and as the library's calls (``own`` true):

* ``fwd``    attention forward whose scores are capped by a tanh and / or whose
             mask keeps a query inside its document, with a prefix that every
             token of the document sees: O and the log-sum-exp;
* ``bwd``    its backward: dQ, dK, dV from O, dO and the log-sum-exp;
* ``append`` new keys and values quantised into a paged cache of e4m3 values
             with one power-of-two scale per (page, head);
* ``cache``  attention of the last tokens of each sequence over that cache.

The layouts are the library's: q, k, v [B, S, H, D]; the cache's keys
[pages, Hkv, page, D], its values [pages, Hkv, D, page].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3_MAX = 448.0
LOWEST_EXP = -120   # the scale's exponent for an all-zero page


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a capped-score layer in training: the repository's 2k causal shape
        dict(name="fwd_cap_2k", op="fwd", B=4, Hq=16, Hkv=16, S=2048, D=128, dtype="bf16", cap=50.0,
             causal=True, docs=0, prefix=0, pad=0, mix=1),
        # documents packed into one 8k sequence, the benchmark's 32 / 8 heads
        dict(name="fwd_docs_8k", op="fwd", B=1, Hq=32, Hkv=8, S=8192, D=128, dtype="bf16", cap=0.0,
             causal=True, docs=1000, prefix=0, pad=100, mix=2),
        # a short ragged batch with instruction prefixes: latency counts
        dict(name="fwd_prefix_333", op="fwd", B=3, Hq=4, Hkv=2, S=333, D=64, dtype="fp16", cap=30.0,
             causal=True, docs=0, prefix=80, pad=0, mix=3),
        # the same three in the backward direction
        dict(name="bwd_cap_2k", op="bwd", B=4, Hq=16, Hkv=16, S=2048, D=128, dtype="bf16", cap=50.0,
             causal=True, docs=0, prefix=0, pad=0, mix=4),
        dict(name="bwd_docs_8k", op="bwd", B=1, Hq=32, Hkv=8, S=8192, D=128, dtype="bf16", cap=0.0,
             causal=True, docs=1000, prefix=0, pad=100, mix=5),
        dict(name="bwd_prefix_333", op="bwd", B=3, Hq=4, Hkv=2, S=333, D=64, dtype="fp16", cap=30.0,
             causal=True, docs=90, prefix=30, pad=0, mix=6),
        # one decoding step of 64 requests: one token each
        dict(name="append_step", op="append", B=64, Hkv=8, D=128, dtype="bf16", page=64, longest=2000,
             spread=32, new=1, mix=7),
        # prompts of mixed lengths entering the cache behind what is there
        dict(name="append_prompts", op="append", B=8, Hkv=8, D=128, dtype="bf16", page=64, longest=700,
             spread=32, new=2048, mix=8),
        # few heads, small pages
        dict(name="append_small", op="append", B=3, Hkv=2, D=64, dtype="fp16", page=16, longest=50,
             spread=32, new=37, mix=9),
        # a decoding step of 64 requests of mixed lengths
        dict(name="cache_step_64", op="cache", B=64, Hq=32, Hkv=8, D=128, dtype="bf16", page=64,
             longest=8192, spread=32, Sq=1, cap=0.0, window=-1, mix=10),
        # two long contexts, capped scores: the work of few rows is split along the keys
        dict(name="cache_long_64k", op="cache", B=2, Hq=32, Hkv=8, D=128, dtype="bf16", page=64,
             longest=65536, spread=2, Sq=1, cap=50.0, window=-1, mix=11),
        # a small batch that verifies three tokens at a time in a local window
        dict(name="cache_small", op="cache", B=3, Hq=8, Hkv=2, D=64, dtype="fp16", page=16, longest=200,
             spread=32, Sq=3, cap=30.0, window=64, mix=12),
    ]


def _log(rng, lo, hi):
    """A whole number spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "append", "cache"])
    dtype = rng.choice(["bf16", "fp16"])
    mix = rng.randrange(1 << 20)
    if op in ("fwd", "bwd"):
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4])
        S = _log(rng, 40, 6000)
        B = _log(rng, 1, max(1, min(8, (32 * 8192 * 8192) // (4 * Hq * S * S))))
        kind = rng.choice(["none", "docs", "docs_prefix", "prefix"])
        cap = rng.choice([0.0, 20.0, 30.0, 50.0]) if kind != "none" else rng.choice([20.0, 30.0, 50.0])
        causal = True if "prefix" in kind else rng.random() < 0.7
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, S=S, D=rng.choice([64, 128]), dtype=dtype, cap=cap, causal=causal,
                    docs=_log(rng, 10, max(11, S)) if "docs" in kind else 0,
                    prefix=_log(rng, 4, max(5, S // 2)) if "prefix" in kind else 0,
                    pad=rng.choice([0, 0, S // 7]) if "docs" in kind else 0, mix=mix)
    if op == "append":
        B = _log(rng, 1, 100)
        return dict(op=op, B=B, Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), dtype=dtype,
                    page=rng.choice([16, 32, 64, 128]), longest=_log(rng, 1, 2000), spread=32,
                    new=rng.choice([1, 1, _log(rng, 2, max(3, 4000 // B))]), mix=mix)
    B = _log(rng, 1, 100)
    Hkv = rng.choice([1, 2, 4, 8])
    return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, D=rng.choice([64, 128]), dtype=dtype,
                page=rng.choice([16, 32, 64, 128]), longest=_log(rng, 1, min(30000, 400000 // B)),
                spread=rng.choice([1, 8, 32]),
                Sq=rng.choice([1, 1, 1, 2, 4]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                window=rng.choice([-1, -1, -1, 100, 1000]), mix=mix)


# ----------------------------------------- what a case's numbers say in full
def _documents(case):
    """Per sequence the (start, end, prefix length) of its documents; tokens
    behind the last one are padding."""
    rng = random.Random(case["mix"])
    S, out = case["S"], []
    for _ in range(case["B"]):
        rows, at, end = [], 0, S - (rng.randint(0, case["pad"]) if case["pad"] else 0)
        while at < end:
            n = end - at if not case["docs"] else min(end - at, _log(rng, max(1, case["docs"] // 4), 3 * case["docs"]))
            rows.append((at, at + n, rng.randint(0, min(n, 2 * case["prefix"])) if case["prefix"] else 0))
            at += n
        out.append(rows)
    return out


def _pairs(case):
    """Visible (query, key) pairs of one head over the batch."""
    total = 0
    for rows in _documents(case):
        for s, e, p in rows:
            n = e - s
            total += n * (n + 1) // 2 + p * (p - 1) // 2 if case["causal"] else n * n
    return total


def _lengths(case):
    """Tokens in the cache per sequence (for ``append``: before the call), and
    the new tokens per sequence."""
    rng = random.Random(case["mix"])
    top = case["longest"]
    lens = [_log(rng, max(1, top // case["spread"]), top) for _ in range(case["B"])]
    if case["op"] == "cache":
        return [max(n, case["Sq"]) for n in lens], [case["Sq"]] * case["B"]
    new = [1 if case["new"] == 1 else rng.randint(max(1, case["new"] // 16), case["new"]) for _ in lens]
    return lens, new


def work(case):
    if case["op"] in ("fwd", "bwd"):
        B, Hq, Hkv, S, D = (case[n] for n in ("B", "Hq", "Hkv", "S", "D"))
        q, k, lse = B * S * Hq * D * 2, B * S * Hkv * D * 2, B * Hq * S * 4
        mask = B * S * 4 * (1 if case["docs"] else 0) + B * S * 4 * (1 if case["docs"] and case["prefix"] else 0)
        n = Hq * D * _pairs(case)
        if case["op"] == "fwd":   # reads q, k, v; writes o and the log-sum-exp
            return {"bytes": 2 * q + 2 * k + lse + mask, "flops": 4 * n}
        return {"bytes": 4 * q + 4 * k + lse + mask, "flops": 10 * n}   # reads q, k, v, o, dO; writes dq, dk, dv
    lens, new = _lengths(case)
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "append":   # 16-bit tokens read, 8-bit ones written, two scales per page touched
        t = sum(new)
        pages = sum((n + m - 1) // case["page"] - n // case["page"] + 1 for n, m in zip(lens, new))
        return {"bytes": 2 * t * Hkv * D * 3 + 2 * pages * Hkv * 4, "flops": 4 * t * Hkv * D}
    w, pairs, seen = case["window"], 0, 0
    for n in lens:
        first = max(0, n - case["Sq"] - w) if w >= 0 else 0
        seen += n - first
        pairs += sum(min(n - case["Sq"] + i, w if w >= 0 else n) + 1 for i in range(case["Sq"]))
    rows = case["B"] * case["Sq"] * case["Hq"]
    return {"bytes": 2 * seen * Hkv * D + 8 * (seen // case["page"]) * Hkv + 2 * rows * D * 2 + 4 * rows,
            "flops": 4 * case["Hq"] * D * pairs}


# ------------------------------------------------------------------ inputs
def _rand(shape, gen, scale, dtype):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def _pow2(e):
    """2^e in 32 bits, from its exponent field."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": dict(case), "scale": case["D"] ** -0.5}
    if case["op"] in ("fwd", "bwd"):
        B, S, D = case["B"], case["S"], case["D"]
        # capped layers meet scores of several units; otherwise N(0, 1)
        a = 2.0 if case["cap"] else 1.0
        st["q"] = _rand((B, S, case["Hq"], D), gen, a, dt)
        st["k"] = _rand((B, S, case["Hkv"], D), gen, a, dt)
        st["v"] = _rand((B, S, case["Hkv"], D), gen, 1.0, dt)
        st["doc"] = st["prefix"] = None
        docs = _documents(case)
        if case["docs"] or case["pad"]:
            ids = [[i for i, (s, e, _) in enumerate(rows) for _ in range(e - s)] for rows in docs]
            st["doc"] = _int([r + [-1] * (S - len(r)) for r in ids])
            if case["prefix"]:
                pre = [[p for s, e, p in rows for _ in range(e - s)] for rows in docs]
                st["prefix"] = _int([r + [0] * (S - len(r)) for r in pre])
        elif case["prefix"]:
            st["prefix"] = _int([rows[0][2] for rows in docs])
        if case["op"] == "bwd":
            st["dout"] = _rand((B, S, case["Hq"], D), gen, 1.0, dt)
            st["o"], st["lse"] = _plain_fwd(st)
        return st
    lens, new = _lengths(case)
    rng = random.Random(seed)
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    need = [-(-(n + (m if case["op"] == "append" else 0)) // page) for n, m in zip(lens, new)]
    pages = list(range(sum(need) + 3))   # a pool with a few free pages
    rng.shuffle(pages)
    width, table, at = max(need), [], 0
    for n in need:
        table.append(pages[at:at + n] + [0] * (width - n))
        at += n
    P = len(pages)
    st["table"] = _int(table)
    st["len"] = _int(lens)
    st["kc"] = _rand((P, Hkv, page, D), gen, 16.0, torch.float8_e4m3fn)
    st["vc"] = _rand((P, Hkv, D, page), gen, 16.0, torch.float8_e4m3fn)
    for name in ("ks", "vs"):   # per (page, head) 2^-5 .. 2^-3: keys and values of about N(0, 1)
        st[name] = _pow2(torch.randint(-5, -2, (P, Hkv), generator=gen, device="cuda"))
    if case["op"] == "append":
        total = sum(new)
        st["k"] = _rand((total, Hkv, D), gen, 2.0, dt)
        st["v"] = _rand((total, Hkv, D), gen, 1.0, dt)
        st["cu"] = _int([sum(new[:i]) for i in range(len(new) + 1)])
        st["max_new"] = max(new)
        # what the plain form's indexing takes: the sequence and place of every new token
        st["seq"] = _int([b for b, n in enumerate(new) for _ in range(n)]).long()
    else:
        st["q"] = _rand((case["B"], case["Sq"], case["Hq"], D), gen, 2.0 if case["cap"] else 1.0, dt)
    return st


# -------------------------------------------------------------- plain forms
def _doc_starts(doc):
    """First position of each token's document (a run of equal ids)."""
    S = doc.shape[1]
    at = torch.arange(S, device=doc.device).expand_as(doc)
    new = torch.ones_like(doc, dtype=torch.bool)
    new[:, 1:] = doc[:, 1:] != doc[:, :-1]
    return torch.where(new, at, torch.zeros_like(at)).cummax(dim=1).values


def _visible(st):
    """[B or 1, 1, 1, S, S] truth values: which keys a query sees."""
    case = st["case"]
    S = case["S"]
    i = torch.arange(S, device="cuda")[:, None]
    j = torch.arange(S, device="cuda")[None, :]
    doc, pre = st["doc"], st["prefix"]
    if doc is not None:
        start = _doc_starts(doc)
        same = (start[:, :, None] == start[:, None, :]) & (doc >= 0)[:, :, None]
    else:
        start, same = torch.zeros((1, S), dtype=torch.long, device="cuda"), torch.ones((1, 1, 1), dtype=torch.bool, device="cuda")
    order = (j <= i)[None] if case["causal"] else torch.ones((1, 1, 1), dtype=torch.bool, device="cuda")
    if pre is not None:
        length = pre[:, None].expand(-1, S).long() if pre.dim() == 1 else pre.gather(1, start).long()
        order = order | (j[None] < (start + length)[:, :, None])
    return (same & order)[:, None, None]


def _split(x, Hkv):
    """[B, S, H, D] as [B, Hkv, H / Hkv, S, D] in 32 bits."""
    B, S, H, D = x.shape
    return x.float().view(B, S, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)


def _join(x, dtype):
    B, Hkv, G, S, D = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, S, Hkv * G, D).to(dtype)


def _scores(st):
    """Masked scores, and what the cap's tanh gave (None without a cap)."""
    case = st["case"]
    Hkv = case["Hkv"]
    s = _split(st["q"], Hkv) @ _split(st["k"], Hkv).transpose(-1, -2) * st["scale"]
    t = None
    if case["cap"]:
        t = torch.tanh(s / case["cap"])
        s = t * case["cap"]
    return s.masked_fill_(~_visible(st), -math.inf) if t is None else s.masked_fill(~_visible(st), -math.inf), t


def _softmax(s):
    """exp(s - log-sum-exp) and the log-sum-exp; rows that see nothing give 0 and -inf."""
    m = s.amax(dim=-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m0)
    l = p.sum(dim=-1, keepdim=True)
    return p / torch.where(l == 0, torch.ones_like(l), l), (m0 + torch.log(l)).squeeze(-1)


def _plain_fwd(st):
    case = st["case"]
    s, _ = _scores(st)
    p, lse = _softmax(s)
    del s
    o = p @ _split(st["v"], case["Hkv"])
    return _join(o, st["q"].dtype), lse.reshape(case["B"], case["Hq"], case["S"])


def _plain_bwd(st):
    case = st["case"]
    Hkv, dt = case["Hkv"], st["q"].dtype
    s, t = _scores(st)
    lse = st["lse"].view(case["B"], Hkv, -1, case["S"], 1)
    p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
    del s
    do = _split(st["dout"], Hkv)
    dv = (p.transpose(-1, -2) @ do).sum(dim=2, keepdim=True)
    delta = (do * _split(st["o"], Hkv)).sum(dim=-1, keepdim=True)
    ds = p * (do @ _split(st["v"], Hkv).transpose(-1, -2) - delta)
    del p
    if t is not None:
        ds = ds * (1.0 - t * t)
    dq = ds @ _split(st["k"], Hkv) * st["scale"]
    dk = (ds.transpose(-1, -2) @ _split(st["q"], Hkv)).sum(dim=2, keepdim=True) * st["scale"]
    return _join(dq, dt), _join(dk, dt), _join(dv, dt)


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    frac, e = torch.frexp(amax)
    e = e - 9 + (frac > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, LOWEST_EXP)).clamp(LOWEST_EXP, -LOWEST_EXP)


def _plain_append(st):
    case = st["case"]
    page, Hkv = case["page"], case["Hkv"]
    seq, table, old_len = st["seq"], st["table"].long(), st["len"].long()
    place = torch.arange(seq.numel(), device="cuda") - st["cu"].long()[seq] + old_len[seq]
    at, slot = table[seq, place // page], place % page
    # the page each sequence goes on in: it holds tokens of before where the length is not a whole number of pages
    part = (old_len % page > 0).nonzero().squeeze(1)
    going_on = table[part, old_len[part] // page]
    for_heads = at[:, None].expand(-1, Hkv)
    for cache, scale, new, values in ((st["kc"], st["ks"], st["k"], False), (st["vc"], st["vs"], st["v"], True)):
        x = new.float()
        amax = torch.zeros_like(scale).scatter_reduce(0, for_heads, x.abs().amax(dim=-1), "amax")
        wanted = _pow2(_exponent(amax))
        before = scale[going_on]
        wanted[going_on] = torch.maximum(wanted[going_on], before)
        scale[at] = wanted[at]
        raw = cache.view(torch.uint8)
        held = raw[going_on].view(torch.float8_e4m3fn).float() * (before / scale[going_on])[:, :, None, None]
        raw[going_on] = held.to(torch.float8_e4m3fn).view(torch.uint8)
        put = (x / scale[at][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        if values:
            raw.permute(0, 3, 1, 2)[at, slot] = put
        else:
            raw.transpose(1, 2)[at, slot] = put
    return st["kc"], st["vc"], st["ks"], st["vs"]


def _plain_cache(st):
    case = st["case"]
    B, Hkv, D, Sq, page = (case[n] for n in ("B", "Hkv", "D", "Sq", "page"))
    table, n = st["table"].long(), st["len"].long()
    L = table.shape[1] * page
    k = st["kc"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * st["ks"][table][..., None, None]
    v = st["vc"].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * st["vs"][table][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, L, D)
    v = v.permute(0, 2, 1, 4, 3).reshape(B, Hkv, 1, L, D)
    s = _split(st["q"], Hkv) @ k.transpose(-1, -2) * st["scale"]
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    j = torch.arange(L, device="cuda")[None, None]
    pos = (n[:, None] - Sq + torch.arange(Sq, device="cuda"))[:, :, None]
    seen = j <= pos
    if case["window"] >= 0:
        seen = seen & (j >= pos - case["window"])
    p, lse = _softmax(s.masked_fill(~seen[:, None, None], -math.inf))
    return _join(p @ v, st["q"].dtype), lse.reshape(B, case["Hq"], Sq)


# ---------------------------------------------------------- the library's
def _own(st):
    import attention_backward_preprocess_gb300 as fa
    case = st["case"]
    if case["op"] in ("fwd", "bwd"):
        ranges = None
        if st["doc"] is not None or st["prefix"] is not None:
            ranges = fa.mask_ranges(case["B"], case["S"], doc_ids=st["doc"], prefix_len=st["prefix"],
                                    causal=case["causal"])
        opt = dict(causal=case["causal"] and ranges is None, softmax_scale=st["scale"], softcap=case["cap"],
                   mask_ranges=ranges)
        if case["op"] == "fwd":
            return fa.fa_fwd(st["q"], st["k"], st["v"], **opt)
        return fa.fa_bwd(st["q"], st["k"], st["v"], st["o"], st["dout"], st["lse"], **opt)
    cache = fa.KvCache(st["kc"], st["vc"], st["ks"], st["vs"], st["table"])
    if case["op"] == "append":
        fa.kvcache_append(cache, st["len"], st["k"], st["v"], cu_new=st["cu"], max_new=st["max_new"])
        return st["kc"], st["vc"], st["ks"], st["vs"]
    return fa.fa_fwd_kvcache(st["q"], cache, st["len"], softmax_scale=st["scale"], softcap=case["cap"],
                             window_left=case["window"])


PLAIN = {"fwd": _plain_fwd, "bwd": _plain_bwd, "append": _plain_append, "cache": _plain_cache}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------- in 64 bits
def _exact_rows(st, b, h, lo, hi, n_prefix):
    """Scores of one head of one document [lo, hi) of sequence b in 64 bits
    (-inf where a key is not visible), the tanh of the cap, and q, k, v."""
    case = st["case"]
    hk = h * case["Hkv"] // case["Hq"]
    q, k, v = st["q"][b, lo:hi, h].double(), st["k"][b, lo:hi, hk].double(), st["v"][b, lo:hi, hk].double()
    s = torch.einsum("id,jd->ij", q, k) * st["scale"]
    t = torch.tanh(s / case["cap"]) if case["cap"] else None
    if t is not None:
        s = case["cap"] * t
    if case["causal"]:
        hidden = torch.ones(hi - lo, hi - lo, dtype=torch.bool, device="cuda").triu(1)
        hidden[:, :n_prefix] = False
        s[hidden] = -math.inf
    return s, t, q, k, v


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "cache":
        return _exact_cache(case, st)
    B, S, Hq, Hkv, D = (case[n] for n in ("B", "S", "Hq", "Hkv", "D"))
    docs = _documents(case)
    zeros = lambda H: torch.zeros((B, S, H, D), dtype=torch.float64, device="cuda")   # noqa: E731
    o, lse = zeros(Hq), torch.full((B, Hq, S), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = zeros(Hq), zeros(Hkv), zeros(Hkv)
    for b in range(B):
        for lo, hi, n_prefix in docs[b]:
            for h in range(Hq):
                s, t, q, k, v = _exact_rows(st, b, h, lo, hi, n_prefix)
                if case["op"] == "fwd":
                    lse[b, h, lo:hi] = torch.logsumexp(s, dim=1)
                    o[b, lo:hi, h] = torch.exp(s - lse[b, h, lo:hi, None]) @ v
                    continue
                hk = h * Hkv // Hq
                p = torch.exp(s - st["lse"][b, h, lo:hi, None].double())
                g = st["dout"][b, lo:hi, h].double()
                row = torch.einsum("id,id->i", g, st["o"][b, lo:hi, h].double())
                ds = p * (g @ v.T - row[:, None])
                if t is not None:
                    ds *= 1.0 - t.square()
                dq[b, lo:hi, h] = st["scale"] * (ds @ k)
                dk[b, lo:hi, hk] += st["scale"] * (ds.T @ q)
                dv[b, lo:hi, hk] += p.T @ g
    return (o, lse) if case["op"] == "fwd" else (dq, dk, dv)


def _exact_append(case, st):
    lens, new = _lengths(case)
    page, Hkv = case["page"], case["Hkv"]
    kc, vc = st["kc"].double(), st["vc"].double().transpose(2, 3).contiguous()
    scales = [st["ks"].double(), st["vs"].double()]
    first = 0
    for b in range(case["B"]):
        for p in range(lens[b] // page, (lens[b] + new[b] - 1) // page + 1):
            at = int(st["table"][b, p])
            a, z = max(lens[b], p * page), min(lens[b] + new[b], (p + 1) * page)   # places of the new tokens
            rows = slice(first + a - lens[b], first + z - lens[b])
            for cache, scale, x in ((kc, scales[0], st["k"]), (vc, scales[1], st["v"])):
                x = x[rows].double().transpose(0, 1)   # [Hkv, tokens, D]
                need = x.abs().amax(dim=(1, 2)) / E4M3_MAX
                e = torch.where(need > 0, torch.ceil(torch.log2(need)), torch.full_like(need, LOWEST_EXP))
                e += (torch.exp2(e) < need).double() - (torch.exp2(e - 1) >= need).double() * (need > 0)
                e = e.clamp(LOWEST_EXP, -LOWEST_EXP)
                if a > p * page:   # tokens of before stay, on the larger of the two scales
                    e = torch.maximum(e, torch.log2(scale[at]).round())
                    ratio = scale[at] / torch.exp2(e)
                    cache[at] = _round_e4m3(cache[at] * ratio[:, None, None])
                scale[at] = torch.exp2(e)
                cache[at, :, a - p * page:z - p * page] = _round_e4m3(x / scale[at][:, None, None])
        first += new[b]
    return kc, vc.transpose(2, 3), scales[0], scales[1]


def _round_e4m3(x):
    """To the nearest value with three fraction bits and exponents of -6 and up, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))).clamp_min(-6)
    e += (x.abs() >= torch.exp2(e + 1)).double()   # log2 rounded down at a power of two
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_cache(case, st):
    lens, _ = _lengths(case)
    B, Sq, Hq, Hkv, page = (case[n] for n in ("B", "Sq", "Hq", "Hkv", "page"))
    o = torch.zeros((B, Sq, Hq, case["D"]), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        at = st["table"][b, :-(-n // page)].long()
        k = st["kc"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * st["ks"][at].double()[:, :, None, None]
        v = st["vc"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * st["vs"][at].double()[:, :, None, None]
        k = k.transpose(0, 1).flatten(1, 2)[:, :n].repeat_interleave(Hq // Hkv, dim=0)   # [Hq, n, D]
        v = v.permute(1, 0, 3, 2).flatten(1, 2)[:, :n].repeat_interleave(Hq // Hkv, dim=0)
        for i in range(Sq):
            last = n - Sq + i
            a = max(0, last - case["window"]) if case["window"] >= 0 else 0
            s = torch.einsum("hd,hjd->hj", st["q"][b, i].double(), k[:, a:last + 1]) * st["scale"]
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            lse[b, :, i] = torch.logsumexp(s, dim=1)
            o[b, i] = torch.einsum("hj,hjd->hd", torch.exp(s - lse[b, :, i, None]), v[:, a:last + 1])
    return o, lse
