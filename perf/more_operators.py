"""What rotary positions and the 4-bit key/value cache cost.

Four operators, each in its plain form (``own`` false: elementary torch
operations in 32 bits, the angles in 64) and as the library's calls (``own``
true):

* ``rope``    queries and keys turned by their positions, forward and backward;
* ``append4`` new keys and values quantised into a paged cache of 4-bit codes
              with a scale and a middle per 64 dims of a token;
* ``cache4``  attention of the last tokens of each sequence over that cache;
* ``read4``   tokens of that cache read back as 16-bit tensors, for the dense
              attention of a prompt's next chunk.

The layouts are the library's: q, k [B, S, H, D]; the cache's codes
[pages, Hkv, page, D / 2] (dim 2i in the low four bits of byte i), its scales
[pages, Hkv, page, D / 64, 2] (scale, middle) in bf16.  A code c stands for
middle + scale (c - 8).
"""
import math
import random
from fractions import Fraction

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LEAST_SCALE = 2.0 ** -60
FIFTEENTHS = 8947849 / 2.0 ** 26   # 2 / 15 in 32 bits
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582")


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the benchmark's training layer: 2 x 8192 tokens, 32 / 8 heads
        dict(name="rope_8k", op="rope", back=False, B=2, S=8192, Hq=32, Hkv=8, D=128, R=128, dtype="bf16",
             inter=False, scaling="none", pos="rows", longest=0, mix=1),
        # its backward over packed documents, positions from the start of each, frequencies stretched by 8
        dict(name="rope_bwd_docs_8k", op="rope", back=True, B=1, S=8192, Hq=32, Hkv=8, D=128, R=128, dtype="bf16",
             inter=False, scaling="stretch", pos="given", longest=1000, mix=2),
        # one decoding step of 64 requests, each at its own place: latency counts
        dict(name="rope_step_64", op="rope", back=False, B=64, S=1, Hq=32, Hkv=8, D=128, R=128, dtype="bf16",
             inter=False, scaling="none", pos="offsets", longest=8192, mix=3),
        # a short batch far into a long context: part of the head, interleaved pairs, fp16
        dict(name="rope_part_333", op="rope", back=False, B=3, S=333, Hq=4, Hkv=2, D=64, R=20, dtype="fp16",
             inter=True, scaling="linear", pos="offsets", longest=500000, mix=4),
        # one decoding step of 64 requests: one token each enters the cache
        dict(name="append4_step", op="append4", B=64, Hkv=8, D=128, dtype="bf16", page=64, longest=2000,
             spread=32, new=1, mix=7),
        # prompts of mixed lengths entering the cache behind what is there
        dict(name="append4_prompts", op="append4", B=8, Hkv=8, D=128, dtype="bf16", page=64, longest=700,
             spread=32, new=2048, mix=8),
        # few heads, small pages
        dict(name="append4_small", op="append4", B=3, Hkv=2, D=64, dtype="fp16", page=16, longest=50,
             spread=32, new=37, mix=9),
        # a decoding step of 64 requests of mixed lengths
        dict(name="cache4_step_64", op="cache4", B=64, Hq=32, Hkv=8, D=128, dtype="bf16", page=64,
             longest=8192, spread=32, Sq=1, cap=0.0, window=-1, mix=10),
        # two long contexts, capped scores: the work of few rows is split along the keys
        dict(name="cache4_long_64k", op="cache4", B=2, Hq=32, Hkv=8, D=128, dtype="bf16", page=64,
             longest=65536, spread=2, Sq=1, cap=50.0, window=-1, mix=11),
        # a small batch that verifies three tokens at a time in a local window
        dict(name="cache4_small", op="cache4", B=3, Hq=8, Hkv=2, D=64, dtype="fp16", page=16, longest=200,
             spread=32, Sq=3, cap=30.0, window=64, mix=12),
        # the contexts of eight prompts read back for the dense attention of their next chunks
        dict(name="read4_contexts", op="read4", B=8, Hkv=8, D=128, dtype="bf16", page=64, longest=8192,
             spread=32, skip=0, mix=13),
        # the last tokens of a few short ones
        dict(name="read4_small", op="read4", B=3, Hkv=2, D=64, dtype="fp16", page=16, longest=200,
             spread=32, skip=30, mix=14),
    ]


def _log(rng, lo, hi):
    """A whole number spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append4", "cache4", "cache4", "read4"])
    dtype = rng.choice(["bf16", "fp16"])
    mix = rng.randrange(1 << 20)
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "rope":
        Hq = Hkv * rng.choice([1, 2, 4, 8])
        D = rng.choice([64, 80, 96, 128, 256])
        tokens = _log(rng, 1, max(2, min(60000, 2 * 8192 * 40 * 128 // (D * (Hq + Hkv)))))
        B = _log(rng, 1, min(tokens, 64))
        pos = rng.choice(["rows", "given", "offsets"])
        return dict(op=op, back=rng.random() < 0.5, B=B, S=max(1, tokens // B), Hq=Hq, Hkv=Hkv, D=D,
                    R=rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)]), dtype=dtype,
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "stretch"]), pos=pos,
                    longest=0 if pos == "rows" else _log(rng, 10, 1000000), mix=mix)
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    B = _log(rng, 1, 100)
    if op == "append4":
        return dict(op=op, B=B, Hkv=Hkv, D=D, dtype=dtype, page=page, longest=_log(rng, 1, 2000), spread=32,
                    new=rng.choice([1, 1, _log(rng, 2, max(3, 8000 // B))]), mix=mix)
    if op == "read4":
        return dict(op=op, B=B, Hkv=Hkv, D=D, dtype=dtype, page=page, longest=_log(rng, 1, max(2, 40000 // B)),
                    spread=rng.choice([1, 8, 32]), skip=rng.choice([0, 0, 20, 500]), mix=mix)
    return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, D=D, dtype=dtype, page=page,
                longest=_log(rng, 1, min(30000, 400000 // B)), spread=rng.choice([1, 8, 32]),
                Sq=rng.choice([1, 1, 1, 2, 4]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                window=rng.choice([-1, -1, -1, 100, 1000]), mix=mix)


# ----------------------------------------- what a case's numbers say in full
def _frequencies(case):
    """Radians per position of every pair, and what the rotation is multiplied by."""
    R = case["R"]
    freq = [10000.0 ** (-2.0 * i / R) for i in range(R // 2)]
    if case["scaling"] == "linear":
        return [f / 4.0 for f in freq], 1.0
    if case["scaling"] == "stretch":   # pairs that turn less than once in 4096 positions by 8, those of over 32 not
        out = []
        for f in freq:
            keep = min(1.0, max(0.0, (4096.0 * f / (2 * math.pi) - 1.0) / 31.0))
            out.append(f / 8.0 * (1.0 - keep) + f * keep)
        return out, 0.1 * math.log(8.0) + 1.0
    return freq, 1.0


def _positions(case):
    """For ``given``: per sequence the positions of its rows, from 0 in each of
    its documents; for ``offsets``: the position of each sequence's first row."""
    rng = random.Random(case["mix"])
    top = case["longest"]
    if case["pos"] == "offsets":
        return [rng.randint(top // 32, top) for _ in range(case["B"])]
    out = []
    for _ in range(case["B"]):
        row = []
        while len(row) < case["S"]:
            row += range(min(_log(rng, max(1, top // 4), 3 * top), case["S"] - len(row)))
        out.append(row)
    return out


def _lengths(case):
    """Tokens in the cache per sequence (for ``append4``: before the call), and
    per sequence the new tokens, the queries, or the tokens not read."""
    rng = random.Random(case["mix"])
    top = case["longest"]
    lens = [_log(rng, max(1, top // case["spread"]), top) for _ in range(case["B"])]
    if case["op"] == "cache4":
        return [max(n, case["Sq"]) for n in lens], [case["Sq"]] * case["B"]
    if case["op"] == "read4":
        return lens, [min(n - 1, rng.randint(0, case["skip"])) for n in lens]
    return lens, [1 if case["new"] == 1 else rng.randint(max(1, case["new"] // 16), case["new"]) for _ in lens]


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "rope":
        rows, heads = case["B"] * case["S"], case["Hq"] + Hkv
        place = {"rows": 0, "given": 4 * rows, "offsets": 4 * case["B"]}[case["pos"]]
        return {"bytes": 4 * rows * heads * D + place, "flops": 3 * rows * heads * case["R"]}
    lens, other = _lengths(case)
    held = D // 2 + D // 16   # bytes of a token's codes, scales and middles: one head's K or V
    if case["op"] in ("append4", "read4"):
        t = sum(other) if case["op"] == "append4" else sum(lens) - sum(other)
        return {"bytes": 2 * t * Hkv * (2 * D + held), "flops": 4 * t * Hkv * D}
    w, pairs, seen = case["window"], 0, 0
    for n in lens:
        seen += n - (max(0, n - case["Sq"] - w) if w >= 0 else 0)
        pairs += sum(min(n - case["Sq"] + i, w if w >= 0 else n) + 1 for i in range(case["Sq"]))
    rows = case["B"] * case["Sq"] * case["Hq"]
    return {"bytes": 2 * seen * Hkv * held + 4 * rows * D + 4 * rows, "flops": 4 * case["Hq"] * D * pairs}


# ------------------------------------------------------------------ inputs
def _rand(shape, gen, scale, dtype):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _codes(shape, gen):
    """Two codes to a byte, as quantised N(0, 1) values have them."""
    c = [torch.randn(shape, generator=gen, device="cuda").mul_(3.2).add_(7.5).round_().clamp_(0, 15).byte()
         for _ in range(2)]
    return c[0] | c[1] << 4


def _scales(shape, gen):
    s = torch.rand(shape, generator=gen, device="cuda") * 0.3 + 0.15
    return torch.stack([s, torch.randn(shape, generator=gen, device="cuda") * 0.3], dim=-1).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": dict(case)}
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "rope":
        B, S = case["B"], case["S"]
        st["q"] = _rand((B, S, case["Hq"], D), gen, 1.0, dt)
        st["k"] = _rand((B, S, Hkv, D), gen, 1.0, dt)
        freq, st["factor"] = _frequencies(case)
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        # the same as parts of a turn per position, in 2^-64ths
        turns = [int(Fraction(f) / TWO_PI * 2 ** 64) % 2 ** 64 for f in freq]
        st["steps"] = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], device="cuda")
        at = None if case["pos"] == "rows" else _int(_positions(case))
        st["positions"] = at if case["pos"] == "given" else None
        st["offsets"] = at if case["pos"] == "offsets" else None
        return st
    lens, other = _lengths(case)
    rng = random.Random(seed)
    page = case["page"]
    need = [-(-(n + (m if case["op"] == "append4" else 0)) // page) for n, m in zip(lens, other)]
    pages = list(range(sum(need) + 3))   # a pool with a few free pages
    rng.shuffle(pages)
    width, table, at = max(need), [], 0
    for n in need:
        table.append(pages[at:at + n] + [0] * (width - n))
        at += n
    P = len(pages)
    st["table"] = _int(table)
    st["len"] = _int(lens)
    for name in ("k", "v"):
        st[name + "c"] = _codes((P, Hkv, page, D // 2), gen)
        st[name + "s"] = _scales((P, Hkv, page, D // 64), gen)
    if case["op"] == "cache4":
        st["q"] = _rand((case["B"], case["Sq"], case["Hq"], D), gen, 2.0 if case["cap"] else 1.0, dt)
        st["scale"] = D ** -0.5
        return st
    count = other if case["op"] == "append4" else [n - m for n, m in zip(lens, other)]
    st["cu"] = _int([sum(count[:i]) for i in range(len(count) + 1)])
    st["rows"] = sum(count)
    # what the plain form's indexing takes: the sequence of every row
    st["seq"] = _int([b for b, n in enumerate(count) for _ in range(n)]).long()
    if case["op"] == "read4":
        st["first"] = _int(other) if case["skip"] else None
        return st
    # a head's dims lie around values of their own, as keys do
    around = _rand((1, Hkv, D), gen, 0.5, torch.float32)
    st["k"] = (_rand((st["rows"], Hkv, D), gen, 1.5, torch.float32) + around).to(dt)
    st["v"] = _rand((st["rows"], Hkv, D), gen, 1.0, dt)
    st["max_new"] = max(count)
    return st


# -------------------------------------------------------------- plain forms
def _plain_rope(st):
    case = st["case"]
    R, S = case["R"], case["S"]
    if st["positions"] is not None:
        pos = st["positions"]
    else:
        pos = torch.arange(S, device="cuda").expand(case["B"], S)
        if st["offsets"] is not None:
            pos = pos + st["offsets"][:, None]
    angle = pos.double()[:, :, None, None] * st["freq"]
    c = (angle.cos() * st["factor"]).float()
    s = (angle.sin() * (-st["factor"] if case["back"] else st["factor"])).float()
    out = []
    for x in (st["q"], st["k"]):
        y = x.float()
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if case["inter"] else (y[..., :R // 2], y[..., R // 2:R])
        u, v = a * c - b * s, b * c + a * s
        turned = torch.stack([u, v], dim=-1).flatten(-2) if case["inter"] else torch.cat([u, v], dim=-1)
        out.append(torch.cat([turned, y[..., R:]], dim=-1).to(x.dtype))
    return tuple(out)


def _values(codes, scales):
    """What codes [..., D / 2] with scales [..., D / 64, 2] stand for, in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8.0
    s = scales.float()
    return (c.unflatten(-1, (-1, 64)) * s[..., :1] + s[..., 1:]).flatten(-2)


def _places(st, start):
    """Pages and slots of the rows of a call, the first of sequence b at token start[b]."""
    seq = st["seq"]
    at = torch.arange(seq.numel(), device="cuda") - st["cu"].long()[seq]
    if start is not None:
        at = at + start.long()[seq]
    page = st["case"]["page"]
    return st["table"].long()[seq, at // page], at % page


def _plain_append4(st):
    at, slot = _places(st, st["len"])
    for codes, scales, new in ((st["kc"], st["ks"], st["k"]), (st["vc"], st["vs"], st["v"])):
        x = new.float().unflatten(-1, (-1, 64))
        lo, hi = x.amin(dim=-1, keepdim=True), x.amax(dim=-1, keepdim=True)
        mid = (0.5 * lo + 0.5 * hi).bfloat16()
        m = mid.float()
        far = torch.maximum(hi - m, m - lo) * FIFTEENTHS
        up = ((far.view(torch.int32) + 0xffff) & -0x10000).view(torch.float32).clamp_min(LEAST_SCALE)   # up to bf16
        c = (torch.round((x - m) * (1.0 / up)).clamp(-8.0, 7.0) + 8.0).byte().flatten(-2)
        codes.transpose(1, 2)[at, slot] = c[..., 0::2] | c[..., 1::2] << 4
        scales.transpose(1, 2)[at, slot] = torch.stack([up.bfloat16(), mid], dim=-1).squeeze(-2)
    return st["kc"], st["vc"], st["ks"], st["vs"]


def _plain_read4(st):
    at, slot = _places(st, st["first"])
    dt = DTYPES[st["case"]["dtype"]]
    return tuple(_values(st[n + "c"].transpose(1, 2)[at, slot], st[n + "s"].transpose(1, 2)[at, slot]).to(dt)
                 for n in "kv")


def _plain_cache4(st):
    case = st["case"]
    B, Hq, Hkv, D, Sq, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "Sq", "page"))
    table, n = st["table"].long(), st["len"].long()
    L = table.shape[1] * page
    k, v = (_values(st[x + "c"][table], st[x + "s"][table]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, L, D)
            for x in "kv")
    q = st["q"].float().view(B, Sq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    s = q @ k.transpose(-1, -2) * st["scale"]
    if case["cap"]:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    j = torch.arange(L, device="cuda")[None, None]
    pos = (n[:, None] - Sq + torch.arange(Sq, device="cuda"))[:, :, None]
    seen = j <= pos
    if case["window"] >= 0:
        seen = seen & (j >= pos - case["window"])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)   # (every query sees its own token)
    p = torch.exp(s - m)
    l = p.sum(dim=-1, keepdim=True)
    o = (p / l) @ v
    return (o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D).to(st["q"].dtype),
            (m + torch.log(l)).reshape(B, Hq, Sq))


# ---------------------------------------------------------- the library's
def _own(st):
    import attention_backward_preprocess_gb300 as fa
    case = st["case"]
    if case["op"] == "rope":
        call = fa.rope_bwd if case["back"] else fa.rope
        return call(st["q"], st["k"], fa.RopeTable(st["steps"], st["factor"]), positions=st["positions"],
                    offsets=st["offsets"], interleaved=case["inter"])
    cache = fa.KvCache4(st["kc"], st["vc"], st["ks"], st["vs"], st["table"])
    if case["op"] == "append4":
        fa.kvcache4_append(cache, st["len"], st["k"], st["v"], cu_new=st["cu"], max_new=st["max_new"])
        return st["kc"], st["vc"], st["ks"], st["vs"]
    if case["op"] == "read4":
        return fa.kvcache4_read(cache, st["len"], st["cu"], st["rows"], DTYPES[case["dtype"]], first=st["first"])
    return fa.fa_fwd_kvcache4(st["q"], cache, st["len"], softmax_scale=st["scale"], softcap=case["cap"],
                              window_left=case["window"])


PLAIN = {"rope": _plain_rope, "append4": _plain_append4, "read4": _plain_read4, "cache4": _plain_cache4}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append4": _exact_append4, "read4": _exact_read4,
            "cache4": _exact_cache4}[case["op"]](case, st)


def _exact_rope(case, st):
    B, S, R, D = (case[n] for n in ("B", "S", "R", "D"))
    row = torch.arange(S, dtype=torch.float64, device="cuda")
    out = [x.double() for x in (st["q"], st["k"])]
    for b in range(B):
        at = st["positions"][b].double() if case["pos"] == "given" else row
        if case["pos"] == "offsets":
            at = at + float(st["offsets"][b])
        turn = torch.polar(torch.full((S, R // 2), st["factor"], dtype=torch.float64, device="cuda"),
                           torch.outer(at, st["freq"]))
        if case["back"]:
            turn = turn.conj()
        first, second = (slice(0, R, 2), slice(1, R, 2)) if case["inter"] else (slice(0, R // 2), slice(R // 2, R))
        for x in out:   # a pair as one complex number
            z = torch.complex(x[b, :, :, first], x[b, :, :, second]) * turn[:, None]
            x[b, :, :, first], x[b, :, :, second] = z.real, z.imag
    return tuple(out)


def _exact_values(st, name, b, lo, hi):
    """Tokens [lo, hi) of sequence b in 64 bits, [Hkv, hi - lo, D]."""
    at = st["table"][b, :-(-hi // st["case"]["page"])].long()
    codes = st[name + "c"][at].transpose(0, 1).flatten(1, 2)[:, lo:hi].long()   # [Hkv, tokens, D / 2]
    s = st[name + "s"][at].transpose(0, 1).flatten(1, 2)[:, lo:hi].double()
    x = torch.empty(codes.shape[:2] + (2 * codes.shape[2],), dtype=torch.float64, device="cuda")
    x[..., 0::2], x[..., 1::2] = (codes % 16).double(), (codes // 16).double()
    wide = s.repeat_interleave(64, dim=2)
    return wide[..., 1] + wide[..., 0] * (x - 8)


def _exact_read4(case, st):
    lens, skip = _lengths(case)
    return tuple(torch.cat([_exact_values(st, n, b, skip[b], lens[b]).transpose(0, 1) for b in range(case["B"])])
                 for n in "kv")


def _exact_append4(case, st):
    """The rule's steps in 64 bits, each then rounded to 32 as the rule says."""
    def r32(x):
        return x.float().double()

    lens, new = _lengths(case)
    first = 0
    for b in range(case["B"]):
        for i in range(lens[b] // case["page"], (lens[b] + new[b] - 1) // case["page"] + 1):
            a = max(lens[b], i * case["page"])
            z = min(lens[b] + new[b], (i + 1) * case["page"])   # places of the new tokens
            at, slots = int(st["table"][b, i]), slice(a - i * case["page"], z - i * case["page"])
            for n in "kv":
                x = st[n][first + a - lens[b]:first + z - lens[b]].double().transpose(0, 1)
                for g in range(case["D"] // 64):
                    y = x[..., 64 * g:64 * g + 64]
                    lo, hi = y.min(dim=2).values, y.max(dim=2).values
                    mid = r32(lo / 2 + hi / 2).bfloat16().double()
                    far = r32(torch.maximum(r32(hi - mid), r32(mid - lo)) * FIFTEENTHS)
                    step = torch.exp2(torch.frexp(far.clamp_min(LEAST_SCALE)).exponent.double() - 8)   # bf16's steps there
                    scale = (torch.ceil(far / step) * step).clamp_min(LEAST_SCALE)
                    c = torch.round(r32(r32(y - mid[..., None]) * r32(1 / scale)[..., None])).clamp(-8, 7) + 8
                    st[n + "c"][at, :, slots, 32 * g:32 * g + 32] = (c[..., 0::2] + 16 * c[..., 1::2]).byte()
                    st[n + "s"][at, :, slots, g, 0] = scale.bfloat16()
                    st[n + "s"][at, :, slots, g, 1] = mid.bfloat16()
        first += new[b]
    return st["kc"], st["vc"], st["ks"].double(), st["vs"].double()


def _exact_cache4(case, st):
    lens, _ = _lengths(case)
    B, Sq, Hq, Hkv = (case[n] for n in ("B", "Sq", "Hq", "Hkv"))
    o = torch.zeros((B, Sq, Hq, case["D"]), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        k, v = (_exact_values(st, x, b, 0, n).repeat_interleave(Hq // Hkv, dim=0) for x in "kv")   # [Hq, n, D]
        for i in range(Sq):
            last = n - Sq + i
            a = max(0, last - case["window"]) if case["window"] >= 0 else 0
            s = torch.einsum("hd,hjd->hj", st["q"][b, i].double(), k[:, a:last + 1]) * st["scale"]
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            lse[b, :, i] = torch.logsumexp(s, dim=1)
            o[b, i] = torch.einsum("hj,hjd->hd", torch.exp(s - lse[b, :, i, None]), v[:, a:last + 1])
    return o, lse
