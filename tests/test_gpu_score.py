"""Capped scores and interval masks (documents, prefixes, windows): forward,
backward and fa_mask_ranges against plain 64-bit forms; refusals on the CPU."""
import ctypes
import math

import pytest
import torch

from score_ref import attend, backward, band, check, lse_bound, visible

F16, BF = torch.float16, torch.bfloat16


def _doc_ids(B, S, kind, seed=0):
    """Documents: 'mixed' lengths from one token up, 'pad' with padding in the
    middle and at the end, 'ones' one token each, 'none' all padding, 'again'
    ids that come back."""
    g = torch.Generator().manual_seed(seed)
    out = torch.zeros((B, S), dtype=torch.int32)
    for b in range(B):
        at, i = 0, 0
        while at < S:
            n = {"ones": 1, "none": S}.get(kind) or 1 + int(torch.randint(0, 130, (1,), generator=g)) * (i % 3)
            out[b, at:at + n] = {"none": -1, "again": i % 2}.get(kind, i)
            if kind == "pad" and i % 4 == 2:
                out[b, at:at + n] = -7
            at, i = at + n, i + 1
    return out


def _inputs(B, Sq, Sk, Hq, Hkv, D, dt, seed, a=1.5):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)   # noqa: E731
    q, k = (r(B, Sq, Hq, D) * a).to(dt), (r(B, Sk, Hkv, D) * a).to(dt)
    return q, k, r(B, Sk, Hkv, D).to(dt), r(B, Sq, Hq, D).to(dt)


def _check_all(fa, x, oks, scale, cap, kw, lens=None, **bwd_kw):
    """Forward, then backward on the forward's own outputs, against 64 bits per
    sequence.  ``lens``: used (query, key) lengths."""
    q, k, v, dout = x
    B, dt, D = q.shape[0], q.dtype, q.shape[-1]
    dev = [t.cuda() for t in x]
    o, lse = fa.fa_fwd(dev[0], dev[1], dev[2], softmax_scale=scale, softcap=cap, **kw)
    grads = fa.fa_bwd(dev[0], dev[1], dev[2], o, dev[3], lse, softmax_scale=scale, softcap=cap, **kw, **bwd_kw)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    for b in range(B):
        nq, nk = lens[b] if lens else (q.shape[1], k.shape[1])
        ok = oks[b][:nq, :nk]
        qb, kb, vb, gb = q[b, :nq], k[b, :nk], v[b, :nk], dout[b, :nq]
        ro, rl, p, t, off = attend(qb, kb, vb, ok, scale, cap)
        check(o[b, :nq], ro, off, "o[%d]" % b)
        lg = lse[b, :, :nq].double().cpu()
        assert torch.equal(torch.isneginf(lg), torch.isneginf(rl)), "empty rows"
        fin = torch.isfinite(rl)
        assert ((lg - rl)[fin].abs() <= lse_bound(cap, rl)[fin]).all(), "lse"
        assert (o[b, :nq].cpu()[torch.isneginf(rl).T] == 0).all()
        og = o[b, :nq].cpu()
        refs = backward(qb, kb, vb, og, gb, ok, p, t, scale, cap, rounded_p=not cap and D == 64)
        for name, got, n, (r, off) in zip(("dq", "dk", "dv"), grads, (nq, nk, nk), refs):
            check(got[b, :n], r, off, "%s[%d]" % (name, b))
    return o, lse, grads


# ------------------------------------------------------------ fa_mask_ranges
RANGES = [
    dict(B=1, S=1, doc="ones"), dict(B=2, S=63, doc="mixed"), dict(B=3, S=64, doc="pad"),
    dict(B=2, S=129, doc="none"), dict(B=2, S=333, doc="again", causal=False),
    dict(B=1, S=1500, doc="mixed", prefix="doc"), dict(B=3, S=700, prefix="seq"),
    dict(B=2, S=700, doc="pad", prefix="seq"), dict(B=1, S=1025, doc="mixed", window=(40, -1)),
    dict(B=1, S=400, window=(0, 0), causal=False), dict(B=1, S=400, window=(2 ** 31 - 1, 2 ** 31 - 1), causal=False),
    dict(B=2, S=300, doc="ones"), dict(B=2, S=8192, doc="mixed"), dict(B=2, S=8193, doc="pad", prefix="seq"),
    dict(B=1, S=9000, window=(700, 5), causal=False),
]


def _mask(c):
    B, S = c["B"], c["S"]
    doc = _doc_ids(B, S, c["doc"], S) if c.get("doc") else None
    prefix = None
    if c.get("prefix"):
        g = torch.Generator().manual_seed(S)   # below 0, inside and past the document
        prefix = torch.randint(-20, 200, (B,) if c["prefix"] == "seq" else (B, S), generator=g).int()
    causal, window = c.get("causal", True), c.get("window")
    ok = visible(B, S, doc, prefix, causal, window)
    return dict(doc_ids=doc, prefix_len=prefix, causal=causal, window=window), ok


def _build(fa, B, S, m, **kw):
    on = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in m.items()}
    return fa.mask_ranges(B, S, **on, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("c", RANGES, ids=lambda c: "_".join("%s%s" % kv for kv in c.items()))
def test_mask_ranges_buffer(fa, cuda_device, c):
    """The rows' intervals are the definition's visible keys, and the tables
    hold every (row block, key block) pair that meets."""
    B, S = c["B"], c["S"]
    m, ok = _mask(c)
    r = _build(fa, B, S, m)
    R = (S + 127) // 128 * 128
    w = r.buffer.cpu().view(torch.int32)
    at = 0

    def take(n):
        nonlocal at
        x = w[at:at + n]
        at += (n + 63) // 64 * 64
        return x
    row, block = take(B * R * 2).view(B, R, 2), take(B * R // 64 * 4).view(B, R // 64, 4)
    key, first = take(B * R // 128 * 4).view(B, R // 128, 4), take(B * R // 64).view(B, R // 64)
    take(B * R // 64)
    order = take(B * R // 128).view(B, R // 128).long()
    for b in range(B):   # each key block once, the most row blocks first
        assert torch.equal(order[b].sort().values, torch.arange(R // 128))
        size = (key[b, :, 1] - key[b, :, 0])[order[b]]
        assert (size[1:] <= size[:-1]).all()
    j = torch.arange(S)
    got = (j >= row[:, :S, :1]) & (j < row[:, :S, 1:])
    assert torch.equal(got, ok)
    assert (row[:, S:] == 0).all()
    pad = torch.zeros((B, R, R), dtype=torch.bool)
    pad[:, :S, :S] = ok
    tiles = pad.view(B, R // 64, 64, R // 128, 128).any(dim=4).any(dim=2)
    n = torch.arange(R // 128)
    # row blocks below S that see a key block whole: the run holds none other
    rows = torch.arange(R) < S
    whole = (pad | ~rows[None, :, None]).view(B, R // 64, 64, R // 128, 128).all(dim=4).all(dim=2)
    m = torch.arange(R // 64)
    for b in range(B):
        for i in range(R // 128):
            run = (m >= key[b, i, 2]) & (m < key[b, i, 3])
            assert (whole[b, run, i]).all()
            inside = whole[b, :, i] & (m >= key[b, i, 0]) & (m < key[b, i, 1])
            assert torch.equal(run, inside), (b, i)   # one run for every mask built here
    for b in range(B):
        for mb in range(R // 64):
            works = (key[b, :, 0] <= mb) & (mb < key[b, :, 1])
            assert (works | ~tiles[b, mb]).all()
            if works.any():   # contiguous from `first`, for the ordered adds
                assert torch.equal(works.nonzero().flatten(),
                                   torch.arange(int(first[b, mb]), int(first[b, mb]) + int(works.sum())))
            lo, hi = row[b, mb * 64:mb * 64 + 64, 0][:max(0, S - 64 * mb)], row[b, mb * 64:mb * 64 + 64, 1][:max(0, S - 64 * mb)]
            some = hi > lo
            want = [int(lo[some].min()) if some.any() else 2 ** 31 - 1, int(hi[some].max()) if some.any() else 0]
            assert block[b, mb, :2].tolist() == want
            if len(lo):
                assert block[b, mb, 2:].tolist() == [int(lo.max()), int(hi.min())]
    assert n.numel() == key.shape[1]


@pytest.mark.gpu
def test_mask_ranges_one_long_document(fa, cuda_device):
    """A document that crosses many tiles, and one begun far back."""
    S = 40000
    doc = torch.zeros((2, S), dtype=torch.int32)
    doc[0, 17:] = 3
    doc[1, S - 1:] = -1
    r = fa.mask_ranges(2, S, doc_ids=doc.cuda(), causal=False)
    R = (S + 127) // 128 * 128
    row = r.buffer.cpu().view(torch.int32)[:2 * R * 2].view(2, R, 2)
    assert (row[0, :17] == torch.tensor([0, 17])).all() and (row[0, 17:S] == torch.tensor([17, S])).all()
    assert (row[1, :S - 1] == torch.tensor([0, S - 1])).all() and (row[1, S - 1:] == 0).all()


# --------------------------------------------------- capped scores, the band
BAND = [
    # B, Sq, Sk, Hq, Hkv, D, dtype, causal, window, cap, scale factor
    (1, 1, 1, 1, 1, 64, BF, True, None, 30.0, 1),
    (1, 1, 300, 2, 2, 128, F16, True, None, 20.0, 1),
    (2, 130, 130, 4, 2, 64, BF, True, None, 50.0, 1),
    (2, 257, 257, 4, 1, 128, BF, True, None, 50.0, 1),
    (1, 200, 333, 2, 2, 128, F16, False, None, 0.5, 1),
    (1, 333, 200, 2, 1, 64, F16, True, None, 30.0, 1),      # rows that see nothing
    (2, 300, 300, 2, 2, 72, BF, True, (60, -1), 30.0, 1),
    (1, 500, 500, 2, 2, 120, F16, False, (33, 70), 15.0, 1),
    (1, 260, 260, 2, 2, 128, BF, True, None, 1000.0, 1),
    (1, 260, 260, 2, 2, 64, F16, True, None, 0.01, 8),      # every score at the cap
    (1, 4200, 4200, 1, 1, 64, BF, True, (200, -1), 30.0, 1),   # D = 64 in the 128-wide tile
]


@pytest.mark.gpu
@pytest.mark.parametrize("c", BAND, ids=lambda c: "b%d_%dx%d_h%d_%d_d%d_%s_c%d_w%s_cap%g_x%d" % (
    c[:6] + (str(c[6])[6:], c[7], c[8], c[9], c[10])))
def test_softcap(fa, cuda_device, c):
    B, Sq, Sk, Hq, Hkv, D, dt, causal, window, cap, mul = c
    x = _inputs(B, Sq, Sk, Hq, Hkv, D, dt, Sq + D)
    ok = band(Sq, Sk, causal, window)
    _check_all(fa, x, [ok] * B, mul / math.sqrt(D), cap, dict(causal=causal, window=window))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_softcap_used_lengths_and_order(fa, cuda_device, D):
    """seqused, deterministic order bit for bit, rows behind the used ones left
    as they were."""
    B, S = 3, 300
    x = _inputs(B, S, S, 4, 2, D, BF, 5)
    lens = [(300, 280), (0, 300), (129, 0)]
    use = dict(seqused_q=torch.tensor([n for n, _ in lens], dtype=torch.int32).cuda(),
               seqused_k=torch.tensor([n for _, n in lens], dtype=torch.int32).cuda())
    oks = []
    for nq, nk in lens:
        ok = torch.zeros((S, S), dtype=torch.bool)
        ok[:nq, :nk] = band(nq, nk, True)
        oks.append(ok)
    out = []
    for _ in range(2):
        g = [torch.full(t.shape, 7.0, dtype=BF, device="cuda") for t in (x[0], x[1], x[2])]
        _check_all(fa, x, oks, 1 / math.sqrt(D), 25.0, dict(causal=True, **use), lens, deterministic=True,
                   dq=g[0], dk=g[1], dv=g[2])
        out.append(g)
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert (out[0][0][1] == 7).all() and (out[0][0][2, 129:] == 7).all() and (out[0][1][2] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D,dt", [(64, F16), (128, BF)])
def test_softcap_varlen(fa, cuda_device, D, dt):
    lens = [(1, 1), (200, 333), (77, 5), (64, 128)]
    x = [_inputs(1, a, b, 4, 2, D, dt, a + b) for a, b in lens]
    cat = [torch.cat([y[i][0] for y in x]) for i in range(4)]
    cu = [torch.tensor([sum(n[i] for n in lens[:j]) for j in range(len(lens) + 1)], dtype=torch.int32).cuda()
          for i in (0, 1)]
    q, k, v, g = (t.cuda() for t in cat)
    kw = dict(causal=True, cu_seqlens_q=cu[0], cu_seqlens_k=cu[1], max_seqlen_q=200, max_seqlen_k=333,
              totals=(q.shape[0], k.shape[0]), softcap=30.0)
    o, lse = fa.fa_fwd(q, k, v, **kw)
    grads = fa.fa_bwd(q, k, v, o, g, lse, **kw)
    torch.cuda.synchronize()
    aq = ak = 0
    for (nq, nk), y in zip(lens, x):
        ok = band(nq, nk, True)
        ro, rl, p, t, off = attend(y[0][0], y[1][0], y[2][0], ok, D ** -0.5, 30.0)
        check(o[aq:aq + nq], ro, off, "o")
        og = o[aq:aq + nq].cpu()
        refs = backward(y[0][0], y[1][0], y[2][0], og, y[3][0], ok, p, t, D ** -0.5, 30.0, False)
        check(grads[0][aq:aq + nq], *refs[0], "dq")
        check(grads[1][ak:ak + nk], *refs[1], "dk")
        check(grads[2][ak:ak + nk], *refs[2], "dv")
        aq, ak = aq + nq, ak + nk


# --------------------------------------------------------- interval masks
MASKED = [
    # mask, Hq, Hkv, D, dtype, cap
    (dict(B=1, S=1, doc="ones"), 1, 1, 64, BF, 0.0),
    (dict(B=2, S=129, doc="none"), 2, 1, 128, BF, 30.0),
    (dict(B=2, S=130, doc="ones"), 2, 2, 128, F16, 0.0),
    (dict(B=2, S=333, doc="mixed"), 4, 2, 128, BF, 0.0),
    (dict(B=2, S=333, doc="mixed"), 4, 1, 64, BF, 0.0),
    (dict(B=2, S=500, doc="pad"), 2, 1, 64, F16, 30.0),
    (dict(B=2, S=500, doc="pad"), 2, 2, 128, F16, 50.0),
    (dict(B=1, S=640, doc="again", causal=False), 2, 2, 128, BF, 0.0),
    (dict(B=1, S=333, doc="mixed", causal=False), 2, 1, 64, F16, 20.0),
    (dict(B=2, S=400, doc="mixed", prefix="doc"), 2, 1, 128, BF, 50.0),
    (dict(B=3, S=270, prefix="seq"), 2, 2, 64, BF, 0.0),
    (dict(B=2, S=256, doc="pad", prefix="seq"), 4, 2, 96, F16, 30.0),
    (dict(B=1, S=700, doc="mixed", window=(40, -1)), 2, 1, 128, BF, 0.0),
    (dict(B=1, S=300, window=(9, 3), causal=False), 2, 1, 128, F16, 5.0),
    (dict(B=1, S=4200, doc="mixed"), 1, 1, 64, BF, 0.0),
    (dict(B=1, S=8200, doc="pad"), 1, 1, 64, BF, 0.0),      # intervals of more than 8192 rows
]


@pytest.mark.gpu
@pytest.mark.parametrize("c", MASKED, ids=lambda c: "_".join("%s%s" % kv for kv in c[0].items()) +
                         "_h%d_%d_d%d_%s_cap%g" % (c[1:4] + (str(c[4])[6:], c[5])))
def test_interval_masks(fa, cuda_device, c):
    mask, Hq, Hkv, D, dt, cap = c
    B, S = mask["B"], mask["S"]
    m, ok = _mask(mask)
    x = _inputs(B, S, S, Hq, Hkv, D, dt, S + D, a=1.5 if cap else 1.0)
    _check_all(fa, x, ok, D ** -0.5, cap, dict(mask_ranges=_build(fa, B, S, m)))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_interval_masks_used_lengths_and_order(fa, cuda_device, D):
    B, S = 2, 520
    m, ok = _mask(dict(B=B, S=S, doc="pad"))
    lens = [(500, 300), (130, 520)]
    use = dict(seqused_q=torch.tensor([n for n, _ in lens], dtype=torch.int32).cuda(),
               seqused_k=torch.tensor([n for _, n in lens], dtype=torch.int32).cuda())
    x = _inputs(B, S, S, 4, 2, D, BF, 6)
    r = _build(fa, B, S, m)
    a = _check_all(fa, x, ok, D ** -0.5, 40.0, dict(mask_ranges=r, **use), lens, deterministic=True)[2]
    b = _check_all(fa, x, ok, D ** -0.5, 40.0, dict(mask_ranges=r, **use), lens, deterministic=True)[2]
    for i, (s, t) in enumerate(zip(a, b)):
        for j in range(B):
            n = lens[j][0 if i == 0 else 1]
            assert torch.equal(s[j, :n], t[j, :n])


@pytest.mark.gpu
def test_interval_masks_equal_the_band(fa, cuda_device):
    """Causal intervals give what the causal flag gives, bit for bit where both
    run the same blocks: capped scores, forward and ordered backward.  (Without
    a cap the flag runs 128-key blocks, the intervals 64-key ones: sums in
    another order.)"""
    x = [t.cuda() for t in _inputs(2, 400, 400, 4, 2, 128, BF, 11)]
    r = fa.mask_ranges(2, 400)
    a, b = (fa.fa_fwd(*x[:3], softcap=30.0, **kw) for kw in (dict(causal=True), dict(mask_ranges=r)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = (fa.fa_bwd(*x[:3], a[0], x[3], a[1], deterministic=True, softcap=30.0, **kw)
              for kw in (dict(causal=True), dict(mask_ranges=r)))
    for s, t in zip(ga, gb):
        assert torch.equal(s, t)


@pytest.mark.gpu
def test_gradients_against_differences(fa, cuda_device):
    """A directional difference of the 64-bit forward of sum(o * dout) agrees
    with the kernel's gradients (documents, a prefix and a cap at once)."""
    B, S, D, cap, scale = 1, 150, 64, 10.0, 0.125
    m, ok = _mask(dict(B=B, S=S, doc="mixed", prefix="doc"))
    x = _inputs(B, S, S, 2, 1, D, F16, 21)
    dev = [t.cuda() for t in x]
    r = _build(fa, B, S, m)
    o, lse = fa.fa_fwd(*dev[:3], softmax_scale=scale, softcap=cap, mask_ranges=r)
    grads = fa.fa_bwd(*dev[:3], o, dev[3], lse, softmax_scale=scale, softcap=cap, mask_ranges=r)
    g = torch.Generator().manual_seed(3)

    def loss(q, k, v):
        s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(2, dim=1)) * scale
        s = (cap * torch.tanh(s / cap)).masked_fill(~ok[0], -1e300)
        p = torch.softmax(s, dim=2) * ok[0].any(dim=1)[None, :, None]
        return (torch.einsum("hij,jhd->ihd", p, v.repeat_interleave(2, dim=1)) * x[3][0].double()).sum()

    base = [t[0].double() for t in x[:3]]
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        at = lambda h: loss(*[t + h * d if n == i else t for n, t in enumerate(base)])   # noqa: B023, E731
        want = float(at(1e-4) - at(-1e-4)) / 2e-4
        got = float((grads[i][0].double().cpu() * d).sum())
        # each element is off by about 2^-11 of its size: sum of independent errors
        size = float((grads[i][0].double().cpu() * d).norm())
        assert abs(got - want) <= 2.0 ** -11 * 8 * size + 1e-6, (name, got, want)


@pytest.mark.gpu
def test_training_step_in_a_graph(fa, cuda_device):
    """Intervals, forward and the staged backward captured once, replayed on
    other documents and other inputs, on a stream of its own."""
    B, S, Hq, Hkv, D = 2, 300, 4, 2, 128
    x = [t.cuda() for t in _inputs(B, S, S, Hq, Hkv, D, BF, 31)]
    doc = _doc_ids(B, S, "mixed", 1).cuda()
    ws = torch.empty(fa.workspace_bytes(B, S, S, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    g = [torch.empty_like(t) for t in x[:3]]
    r = fa.mask_ranges(B, S, doc_ids=doc)

    def step():
        fa.mask_ranges(B, S, doc_ids=doc, out=r)
        o, lse = fa.fa_fwd(*x[:3], softcap=30.0, mask_ranges=r)
        fa.fa_bwd(*x[:3], o, x[3], lse, softcap=30.0, mask_ranges=r, workspace=ws, dq=g[0], dk=g[1], dv=g[2])
        return o, lse
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o, lse = step()
    for seed in (41, 42):
        y = _inputs(B, S, S, Hq, Hkv, D, BF, seed)
        ids = _doc_ids(B, S, "pad", seed)
        for dst, src in zip(x, y):
            dst.copy_(src)
        doc.copy_(ids)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ok = visible(B, S, ids)
        for b in range(B):
            ro, rl, p, t, off = attend(y[0][b], y[1][b], y[2][b], ok[b], D ** -0.5, 30.0)
            check(o[b], ro, off, "o")
            refs = backward(y[0][b], y[1][b], y[2][b], o[b].cpu(), y[3][b], ok[b], p, t, D ** -0.5, 30.0, False)
            for got, (want, off), name in zip(g, refs, ("dq", "dk", "dv")):
                check(got[b], want, off, name)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [149, 150])
def test_nan_scores_stay_nan(fa, cuda_device, D, bad):
    """A NaN query row gives NaN output and gradient rows under a cap; other
    rows, and rows that do not see a NaN key (next to their last one, an
    even and an odd one), give what they gave."""
    q, k, v, g = (t.cuda() for t in _inputs(1, 200, 200, 2, 2, D, BF, 51))
    kw = dict(causal=True, softcap=30.0)
    want, wl = fa.fa_fwd(q, k, v, **kw)
    dq, _, _ = fa.fa_bwd(q, k, v, want, g, wl, deterministic=True, **kw)
    q2, k2 = q.clone(), k.clone()
    q2[0, 77, 1] = float("nan")
    k2[0, bad, 0] = float("nan")
    got, lse = fa.fa_fwd(q2, k2, v, **kw)
    assert torch.isnan(got[0, 77, 1]).all() and torch.isnan(lse[0, 1, 77])
    assert torch.isnan(got[0, bad:, 0]).all()
    assert torch.equal(got[0, :bad, 0], want[0, :bad, 0])
    rest = [i for i in range(200) if i != 77]
    assert torch.equal(got[0, rest, 1], want[0, rest, 1])
    # in the backward dK and dV of the head are NaN then; dQ of the row, and of
    # the one it shares a reciprocal with
    dq2, _, _ = fa.fa_bwd(q2, k, v, want, g, wl, deterministic=True, **kw)
    assert torch.isnan(dq2[0, 77, 1]).all()
    rest = [i for i in rest if i != 76]
    assert torch.equal(dq2[0, :, 0], dq[0, :, 0]) and torch.equal(dq2[0, rest, 1], dq[0, rest, 1])


# ------------------------------- problems of more query tiles than the GPU has SMs
# (the forward's two CTAs per SM; tests above mostly have fewer tiles)
MANY = [
    # B, S (Sq, Sk), Hq, Hkv, D, dtype, mask keywords (None: the band), causal, window, cap
    (3, (300, 300), 20, 4, 128, BF, None, True, None, 50.0),
    (3, (300, 300), 20, 20, 64, F16, None, True, None, 30.0),
    (2, (333, 200), 40, 8, 64, BF, None, True, None, 20.0),        # rows that see nothing
    (80, (1, 130), 2, 1, 128, F16, None, True, None, 15.0),        # single queries
    (2, (257, 390), 32, 8, 120, BF, None, False, (33, 70), 25.0),
    (2, (400, 400), 24, 2, 72, F16, None, True, (60, -1), 1000.0),
    (3, (300, 300), 20, 4, 128, F16, dict(doc="mixed"), True, None, 0.0),
    (3, (300, 300), 20, 4, 64, BF, dict(doc="pad"), True, None, 0.0),
    (3, (300, 300), 20, 4, 128, BF, dict(doc="pad", prefix="doc"), True, None, 50.0),
    (160, (65, 65), 2, 1, 64, F16, dict(doc="ones"), True, None, 30.0),
    (160, (64, 64), 1, 1, 128, BF, dict(doc="none"), True, None, 0.0),
    (2, (420, 420), 24, 8, 96, BF, dict(doc="again", causal=False), True, None, 0.0),
    (2, (420, 420), 24, 8, 128, F16, dict(doc="mixed", window=(40, -1)), True, None, 10.0),
    (1, (2500, 2500), 8, 2, 64, BF, dict(doc="mixed", prefix="seq"), True, None, 0.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("c", MANY, ids=lambda c: "b%d_%dx%d_h%d_%d_d%d_%s_%s_c%d_w%s_cap%g" % (
    c[0], *c[1], *c[2:5], str(c[5])[6:], "_".join("%s%s" % kv for kv in (c[6] or {"band": ""}).items()), *c[7:]))
def test_many_tiles(fa, cuda_device, c):
    B, (Sq, Sk), Hq, Hkv, D, dt, mask, causal, window, cap = c
    assert B * Hq * ((Sq + 127) // 128) > torch.cuda.get_device_properties(0).multi_processor_count
    x = _inputs(B, Sq, Sk, Hq, Hkv, D, dt, Sq + D, a=1.5 if cap else 1.0)
    if mask is None:
        oks, kw = [band(Sq, Sk, causal, window)] * B, dict(causal=causal, window=window)
    else:
        m, oks = _mask(dict(B=B, S=Sq, **mask))
        kw = dict(mask_ranges=_build(fa, B, Sq, m))
    _check_all(fa, x, oks, D ** -0.5, cap, kw)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_many_tiles_used_lengths(fa, cuda_device, D):
    B, S = 4, 520
    m, ok = _mask(dict(B=B, S=S, doc="pad"))
    lens = [(500, 300), (130, 520), (0, 64), (520, 0)]
    use = dict(seqused_q=torch.tensor([n for n, _ in lens], dtype=torch.int32).cuda(),
               seqused_k=torch.tensor([n for _, n in lens], dtype=torch.int32).cuda())
    x = _inputs(B, S, S, 12, 3, D, BF, 9)
    _check_all(fa, x, ok, D ** -0.5, 40.0, dict(mask_ranges=_build(fa, B, S, m), **use), lens)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dt", [(64, BF), (128, F16)])
def test_many_tiles_varlen(fa, cuda_device, D, dt):
    lens = [(1, 1), (200, 333), (77, 5), (64, 128), (0, 40), (129, 129)] * 8
    x = [_inputs(1, a, b, 8, 2, D, dt, a + b + i) for i, (a, b) in enumerate(lens)]
    cat = [torch.cat([y[i][0] for y in x]) for i in range(4)]
    cu = [torch.tensor([sum(n[i] for n in lens[:j]) for j in range(len(lens) + 1)], dtype=torch.int32).cuda()
          for i in (0, 1)]
    q, k, v, g = (t.cuda() for t in cat)
    kw = dict(causal=True, cu_seqlens_q=cu[0], cu_seqlens_k=cu[1], max_seqlen_q=200, max_seqlen_k=333,
              totals=(q.shape[0], k.shape[0]), softcap=30.0)
    o, lse = fa.fa_fwd(q, k, v, **kw)
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    aq = 0
    for (nq, nk), y in zip(lens, x):
        ro, rl, _, _, off = attend(y[0][0], y[1][0], y[2][0], band(nq, nk, True), D ** -0.5, 30.0)
        check(o[aq:aq + nq], ro, off, "o")
        lg, fin = lse[:, aq:aq + nq].double().cpu(), torch.isfinite(rl)
        assert ((lg - rl)[fin].abs() <= lse_bound(30.0, rl)[fin]).all()
        assert torch.equal(torch.isneginf(lg), torch.isneginf(rl))
        aq += nq


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [149, 150])
def test_many_tiles_nan_scores(fa, cuda_device, D, bad):
    q, k, v, _ = (t.cuda() for t in _inputs(1, 200, 200, 90, 90, D, BF, 52))
    for kw in (dict(causal=True, softcap=30.0), dict(mask_ranges=fa.mask_ranges(1, 200))):
        want, _ = fa.fa_fwd(q, k, v, **kw)
        q2, k2 = q.clone(), k.clone()
        q2[0, 77, 1] = float("nan")
        k2[0, bad, 0] = float("nan")
        got, lse = fa.fa_fwd(q2, k2, v, **kw)
        assert torch.isnan(got[0, 77, 1]).all() and torch.isnan(lse[0, 1, 77])
        assert torch.isnan(got[0, bad:, 0]).all()
        assert torch.equal(got[0, :bad, 0], want[0, :bad, 0])
        rest = [i for i in range(200) if i != 77]
        assert torch.equal(got[0, rest, 1], want[0, rest, 1]) and torch.equal(got[0, :, 2:], want[0, :, 2:])


@pytest.mark.gpu
def test_two_streams_at_once(fa, cuda_device):
    """Calls in flight together on two streams give what each gives alone."""
    r = fa.mask_ranges(3, 300, doc_ids=_doc_ids(3, 300, "pad").cuda())
    runs = [([t.cuda() for t in _inputs(3, 300, 300, 20, 4, 128, BF, 81)], dict(mask_ranges=r, softcap=30.0)),
            ([t.cuda() for t in _inputs(2, 333, 333, 40, 8, 64, F16, 82)], dict(causal=True, softcap=20.0))]

    def step(x, kw):
        o, lse = fa.fa_fwd(*x[:3], **kw)
        return (o, lse) + fa.fa_bwd(*x[:3], o, x[3], lse, deterministic=True, **kw)
    want = [step(*a) for a in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[], []]
    for _ in range(5):
        for i, a in enumerate(runs):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(*a))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        for one in many:
            assert all(torch.equal(a, b) for a, b in zip(w, one))


@pytest.mark.gpu
def test_other_strides(fa, cuda_device):
    """Tensors that lie head by head, or as slices of a wider one, give what
    their contiguous copies give; non-contiguous outputs are refused."""
    x = [t.cuda() for t in _inputs(2, 150, 150, 4, 2, 64, BF, 61)]
    o, lse = fa.fa_fwd(*x[:3], causal=True, softcap=30.0)
    want = fa.fa_bwd(*x[:3], o, x[3], lse, causal=True, softcap=30.0, deterministic=True)
    y = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in x[:2]]
    wide = torch.cat([x[2], x[2]], dim=3)
    y.append(wide[..., 64:])
    o2, lse2 = fa.fa_fwd(*y, causal=True, softcap=30.0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    lying = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (o, x[3])]
    got = fa.fa_bwd(*y, *lying, lse, causal=True, softcap=30.0, deterministic=True)
    for a, b in zip(got, want):
        assert a.is_contiguous() and torch.equal(a, b)
    with pytest.raises(ValueError):
        fa.fa_bwd(*x[:3], o, x[3], lse, dq=y[0])
    # lying off the 16-byte steps of the tensor loads: copied, on the current stream only
    odd = [torch.cat([t, t], dim=3)[..., 1:65].copy_(t) for t in x[:3]]
    o3, _ = fa.fa_fwd(*odd, causal=True, softcap=30.0)
    assert torch.equal(o, o3)
    o4, _ = fa.fa_fwd(*y, causal=True, softcap=30.0, stream=torch.cuda.current_stream())
    assert torch.equal(o, o4)
    with pytest.raises(ValueError):
        fa.fa_fwd(*odd, stream=torch.cuda.current_stream())
    # head dims of the wide backward kernel, slices of a joint projection
    w = torch.cat(_inputs(1, 140, 140, 2, 2, 192, BF, 62), dim=2).cuda()
    parts = [w[:, :, 2 * i:2 * i + 2] for i in range(4)]
    whole = [t.contiguous() for t in parts]
    a, b = fa.fa_fwd(*parts[:3], causal=True), fa.fa_fwd(*whole[:3], causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = fa.fa_bwd(*parts[:3], a[0], parts[3], a[1], causal=True), fa.fa_bwd(*whole[:3], a[0], whole[3], a[1], causal=True)
    assert torch.equal(ga[1], gb[1]) and torch.equal(ga[2], gb[2])
    # packed varlen slices of a joint projection
    cu = torch.tensor([0, 60, 150], dtype=torch.int32).cuda()
    kw = dict(cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=90, max_seqlen_k=90, causal=True, totals=(150, 150))
    joint = torch.cat([x[0][0, :, :2], x[1][0], x[2][0]], dim=1)
    parts = [joint[:, :2], joint[:, 2:4], joint[:, 4:]]
    a = fa.fa_fwd(*parts, **kw)
    b = fa.fa_fwd(*(t.contiguous() for t in parts), **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------- refusals (no GPU)
def _fwd_ext(fa, ext, B=1, Sq=128, Sk=128, D=64, causal=0, cu=None, scale=0.125):
    vp = ctypes.c_void_p
    return fa.lib().fa_fwd_ext(*[vp(0x1000 * (i + 1)) for i in range(5)], B, Sq, Sk, 2, 2, D, scale, causal, cu, cu,
                               ctypes.pointer(ext), 0, None)


def _bwd_ext(fa, ext, B=1, Sq=128, Sk=128, D=64, causal=0, cu=None, scale=0.125):
    vp = ctypes.c_void_p
    return fa.lib().fa_bwd_ext(*[vp(0x1000 * (i + 1)) for i in range(9)], B, Sq, Sk, 2, 2, D, scale, causal, cu, cu,
                               ctypes.pointer(ext), 0, 0, vp(0x100000), 1 << 40, None)


def _ext(fa, **over):
    e = fa.FaExt(window_left=-1, window_right=-1)
    for n, v in over.items():
        setattr(e, n, v)
    return e


REFUSED = [
    (dict(softcap=-1.0), {}, 1), (dict(softcap=float("nan")), {}, 1), (dict(softcap=float("inf")), {}, 1),
    (dict(softcap=1e-4), {}, 1), (dict(softcap=2000.0), {}, 1), (dict(softcap=0.001), dict(scale=3e38), 1),
    (dict(softcap=30.0, alibi_slopes=0x7000), {}, 2), (dict(softcap=30.0, dropout_p=0.5), {}, 2),
    (dict(softcap=30.0, bias=0x7000, bias_row_stride=128), {}, 2), (dict(softcap=30.0), dict(D=256), 2),
    (dict(softcap=30.0, head_dim_v=64), dict(D=128), 2),
    (dict(mask_ranges=0x10000, mask_ranges_bytes=1 << 30), dict(causal=1), 1),
    (dict(mask_ranges=0x10000, mask_ranges_bytes=1 << 30, window_left=5), {}, 1),
    (dict(mask_ranges=0x10000, mask_ranges_bytes=1 << 30), dict(Sq=100), 1),
    (dict(mask_ranges=0x10010, mask_ranges_bytes=1 << 30), {}, 1),
    (dict(mask_ranges=0x10000, mask_ranges_bytes=100), {}, 1),
    (dict(mask_ranges=0x10000, mask_ranges_bytes=1 << 30), dict(cu=0xA000), 2),
    (dict(mask_ranges=0x10000, mask_ranges_bytes=1 << 30), dict(D=192), 2),
    (dict(mask_ranges=0x10000, mask_ranges_bytes=1 << 30, alibi_slopes=0x7000), {}, 2),
    (dict(q_stride=(8192, 100, 64)), {}, 1), (dict(k_stride=(0, 128, 64)), {}, 1),
    (dict(v_stride=(8192, 128, -64)), {}, 1), (dict(q_stride=(8192, 1 << 39, 64)), {}, 1),
]


@pytest.mark.parametrize("over,call,status", REFUSED)
def test_refused_before_any_launch(fa, over, call, status):
    assert _fwd_ext(fa, _ext(fa, **over), **call) == status
    assert _bwd_ext(fa, _ext(fa, **over), **call) == status


@pytest.mark.parametrize("over", [
    dict(B=0), dict(S=0), dict(S=-3), dict(ranges=0), dict(ranges=0x100010), dict(nbytes=16), dict(doc=0x2002),
    dict(prefix=0x3001), dict(wl=-2), dict(wr=-5), dict(prefix=0x3000, causal=0), dict(prefix=0x3000, wl=4),
    dict(B=1 << 16, S=1 << 16)])
def test_mask_ranges_refused(fa, over):
    a = dict(doc=0x2000, prefix=0, per=0, B=2, S=100, causal=1, wl=-1, wr=-1, ranges=0x100000, nbytes=1 << 40)
    a.update(over)
    vp = ctypes.c_void_p
    assert fa.lib().fa_mask_ranges(vp(a["doc"]), vp(a["prefix"]), a["per"], a["B"], a["S"], a["causal"], a["wl"],
                                   a["wr"], vp(a["ranges"]), a["nbytes"], None) == 1


def test_mask_ranges_sizes(fa):
    n = fa.lib().fa_mask_ranges_bytes
    assert n(0, 5) == 0 and n(5, -1) == 0 and n(1 << 20, 1 << 20) == 0
    # rows of 8 bytes, blocks of 16, key blocks of 8, two words per row block
    assert n(2, 129) == 2 * 256 * 8 + 5 * 256
    assert n(1, 1 << 20) > 8 << 20


def test_python_refusals(fa):
    doc = torch.zeros((2, 10), dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.mask_ranges(2, 10, doc_ids=doc)                 # not on the GPU
    with pytest.raises(ValueError):
        fa.mask_ranges(2, 10, doc_ids=doc.long())
    q = torch.zeros((1, 64, 2, 64), dtype=BF)
    with pytest.raises(ValueError):
        fa.fa_fwd(q, q, q, mask_ranges=doc)
    with pytest.raises(ValueError):
        fa.fa_fwd(q, q, q, mask_ranges=fa.MaskRanges(doc, 1, 65))
