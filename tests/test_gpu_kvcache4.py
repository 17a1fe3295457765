"""The 4-bit paged cache: appending (codes, scales and middles exact), reading
back and attention over it, against plain forms in 64 bits; a serving run with
rotary positions; refusals on the CPU.

Bounds of the attention.  With S = 16 scale + |middle| at least as large as any value
the kernel's sums go through, a score is off by e = 2^-21 sum |q| S c (32-bit sums of the
tensor core: within 2^-22 of the sum of magnitudes, and the few operations behind
it) + softcap 2^-21.  That is a relative error of the weights, twice (numerator
and row sum); exp2, the sums and the division add less than 2^-17.  P times a
scale is rounded to f16, 2^-11 relative and 2^-25 of the largest in absolute
terms, and meets codes of at most 8 in size once 8 times their sum is taken off;
the output is rounded once.
"""
import ctypes
import math

import pytest
import torch

from score_ref import SUB, U, check

F16, BF = torch.float16, torch.bfloat16
LEAST = 2.0 ** -60


# ------------------------------------------------------------ plain forms
def unpack(codes, scales):
    """(c - 8, scale, middle) in 64 bits, each [..., D], of codes [..., D / 2] and scales [..., D / 64, 2]."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double() - 8
    s = scales.double().repeat_interleave(64, dim=-2)
    return c, s[..., 0], s[..., 1]


def values(codes, scales):
    c, s, m = unpack(codes, scales)
    return m + s * c


def r32(x):
    return x.float().double()


def quantise(x):
    """codes [..., D / 2] and scales [..., D / 64, 2] of x [..., D] by the rule, each
    operation in 64 bits and then rounded to 32 (which is what a 32-bit one gives)."""
    y = x.double().unflatten(-1, (-1, 64))
    lo, hi = y.amin(dim=-1), y.amax(dim=-1)
    mid = r32(lo / 2 + hi / 2).bfloat16().double()
    far = r32(torch.maximum(r32(hi - mid), r32(mid - lo)) * (8947849 / 2.0 ** 26))
    step = torch.exp2(torch.frexp(far.clamp_min(LEAST)).exponent.double() - 8)
    scale = (torch.ceil(far / step) * step).clamp_min(LEAST)
    c = torch.round(r32(r32(y - mid[..., None]) * r32(1 / scale)[..., None])).clamp(-8, 7) + 8
    bad = ~torch.isfinite(y).all(dim=-1)
    c = torch.where(bad[..., None], torch.full_like(c, 8), c).flatten(-2).to(torch.uint8)
    scale = torch.where(bad, torch.full_like(scale, LEAST), scale)
    mid = torch.where(bad, torch.full_like(mid, math.nan), mid)
    return c[..., 0::2] | c[..., 1::2] << 4, torch.stack([scale, mid], dim=-1).to(BF)


def make_cache(pages, H, page, D, seed, spread=(0.15, 0.45)):
    """Random caches on the CPU: codes k, v, scales ks, vs."""
    g = torch.Generator().manual_seed(seed)
    c = [torch.randint(0, 256, (pages, H, page, D // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
    s = []
    for _ in range(2):
        w = torch.rand((pages, H, page, D // 64), generator=g) * (spread[1] - spread[0]) + spread[0]
        s.append(torch.stack([w, torch.randn(w.shape, generator=g) * 0.3], dim=-1).to(BF))
    return c[0], c[1], s[0], s[1]


def block_table(lens, page, extra=0, seed=0):
    need = [max(0, -(-n // page)) for n in lens]
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(sum(need) + extra, generator=g).int()
    t = torch.full((len(lens), max(need + [1])), -5, dtype=torch.int32)   # unused entries: no page
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, sum(need) + extra


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def sums(n):
    return ints([sum(n[:i]) for i in range(len(n) + 1)])


def plain_attention(q, k, v, ks, vs, table, lens, page, scale, cap, window):
    """(o, lse, bounds of both) in 64 bits, per sequence, query and head."""
    B, Sq, Hq, D = q.shape
    Hkv = k.shape[1]
    o = torch.zeros((B, Sq, Hq, D), dtype=torch.float64)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64)
    off, lse_off = torch.zeros_like(o), torch.zeros((B, Hq, Sq), dtype=torch.float64)
    for b, n in enumerate(lens):
        for i in range(Sq):
            pos = n - Sq + i
            if pos < 0:
                continue
            rows = torch.arange(max(0, pos - window) if window >= 0 else 0, pos + 1)
            at, slot = table[b].long()[rows // page], rows % page
            for h in range(Hq):
                hk = h * Hkv // Hq
                kc, kw, km = unpack(k[at, hk, slot], ks[at, hk, slot])
                vc, vw, vm = unpack(v[at, hk, slot], vs[at, hk, slot])
                x = q[b, i, h].double()
                s = (km + kw * kc) @ x * scale
                e = 2.0 ** -21 * float(((16 * kw + km.abs()) @ x.abs()).max()) * scale + cap * 2.0 ** -21
                if cap:
                    s = cap * torch.tanh(s / cap)
                lse[b, h, i] = torch.logsumexp(s, dim=0)
                p = torch.exp(s - lse[b, h, i])
                o[b, i, h] = p @ (vm + vw * vc)
                top = (p[:, None] * vw).amax(dim=0)
                off[b, i, h] = 2.0 ** -11 * (p @ (vw * vc.abs())) + 2.0 ** -25 * 8 * top * len(rows) \
                    + (2 * e + 2.0 ** -17) * (p @ (16 * vw + vm.abs()))
                lse_off[b, h, i] = e + 2.0 ** -17 + abs(float(lse[b, h, i])) * 2.0 ** -20
    return o, lse, off + U[q.dtype] * o.abs() + SUB[q.dtype], lse_off


def check_lse(lse, want, off):
    lse = lse.double().cpu()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(want))
    fin = torch.isfinite(want)
    assert ((lse - want)[fin].abs() <= off[fin]).all(), float(((lse - want)[fin].abs() - off[fin]).max())


# --------------------------------------------------------------- appending
APPEND = [
    # lens, new tokens, page, Hkv, D, dtype, magnitude of the new values, around which value
    ([0], [1], 16, 1, 64, BF, 1.0, 0.0),
    ([0, 15, 16, 17], [1, 1, 1, 1], 16, 2, 128, F16, 1.0, 0.0),
    ([0, 63, 64, 100, 5], [200, 2, 64, 1, 0], 64, 2, 128, BF, 3.0, 0.0),
    ([3, 30], [40, 77], 32, 1, 64, F16, 100.0, 0.0),
    ([7, 120, 250], [1, 9, 130], 128, 3, 128, BF, 1e-3, 5.0),
    ([9, 40], [3, 30], 48, 2, 64, BF, 1e30, 0.0),
    ([9, 40], [3, 30], 16, 1, 128, BF, 1e-38, 0.0),    # below the least scale
    ([5, 5], [4, 4], 16, 1, 64, F16, 0.0, 0.0),        # all zeros
    ([5, 5], [4, 4], 16, 1, 128, F16, 0.0, -1.25),     # all the same
    ([0, 7], [700, 900], 64, 8, 128, BF, 1.0, 0.5),    # several rows a CTA
    ([i % 33 for i in range(300)], [i % 3 for i in range(300)], 16, 1, 64, BF, 1.0, 0.0),   # more sequences than threads
]


def _ids(c):
    return "_".join(("-".join(map(str, x[:6])) if isinstance(x, list) else str(x)) for x in c).replace("torch.", "")


@pytest.mark.gpu
@pytest.mark.parametrize("c", APPEND, ids=_ids)
def test_append(fa, cuda_device, c):
    lens, new, page, H, D, dt, size, around = c
    table, pages = block_table([a + n for a, n in zip(lens, new)], page, extra=3, seed=page)
    host = make_cache(pages, H, page, D, 1)
    g = torch.Generator().manual_seed(2)
    rows = sum(new)
    kn, vn = ((torch.randn((rows + 2, H, D), generator=g) * size + around).to(dt) for _ in range(2))   # two rows of nobody
    if size == 1.0 and not around:
        kn[-3, 0, 3] = float("inf")
        vn[-3, 0, 5] = float("nan")
        vn[0, 0, D - 1] = -float("inf")
    dev = [t.cuda() for t in host]
    cache = fa.KvCache4(*dev, table.cuda())
    fa.kvcache4_append(cache, ints(lens), kn.cuda(), vn.cuda(), cu_new=sums(new), max_new=max(new))
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    want = [t.clone() for t in host]
    at = 0
    for b, n in enumerate(new):
        for x, codes, scales in ((kn, want[0], want[2]), (vn, want[1], want[3])):
            c4, s4 = quantise(x[at:at + n])
            for t in range(n):
                p, slot = int(table[b, (lens[b] + t) // page]), (lens[b] + t) % page
                codes[p, :, slot], scales[p, :, slot] = c4[t], s4[t]
        at += n
    for got, w, name in zip(dev, want, ("k", "v", "k_scale", "v_scale")):
        got = got.cpu()
        same = (got == w) | ((got != got) & (w != w))
        assert same.all(), (name, int((~same).sum()), got[~same][:5], w[~same][:5])


def test_rule_keeps_half_a_scale():
    """The rule itself: a value is off by at most half a scale, and by what rounding its
    distance from the middle and 1 / scale in 32 bits adds (2^-22 of up to 8 scales)."""
    g = torch.Generator().manual_seed(3)
    for dt, size, around in ((BF, 1.0, 0.0), (F16, 1.0, 0.0), (BF, 1e-3, 7.0), (F16, 0.01, -100.0), (BF, 1e25, 0.0)):
        x = (torch.randn((50, 2, 128), generator=g) * size + around).to(dt)
        c, s, m = unpack(*quantise(x))
        assert ((m + s * c - x.double()).abs() <= s * (0.5 + 2.0 ** -19)).all()


@pytest.mark.gpu
def test_append_every_sequence_the_same(fa, cuda_device):
    """The [B, T, Hkv, D] form, on a stream of its own, from a strided tensor."""
    lens, T, page, H, D = [10, 0, 31], 5, 16, 2, 64
    table, pages = block_table([n + T for n in lens], page)
    host = make_cache(pages, H, page, D, 3)
    kv = torch.randn((3, T, 2, H, D), generator=torch.Generator().manual_seed(4)).to(BF)
    dev = [t.cuda() for t in host]
    cache, on, n = fa.KvCache4(*dev, table.cuda()), kv.cuda(), ints(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.kvcache4_append(cache, n, on[:, :, 0], on[:, :, 1])
    side.synchronize()
    want = [t.clone() for t in host]
    for b in range(3):
        for i, (codes, scales) in enumerate(((want[0], want[2]), (want[1], want[3]))):
            c4, s4 = quantise(kv[b, :, i])
            for t in range(T):
                p, slot = int(table[b, (lens[b] + t) // page]), (lens[b] + t) % page
                codes[p, :, slot], scales[p, :, slot] = c4[t], s4[t]
    for got, w in zip(dev, want):
        assert torch.equal(got.cpu(), w)
    with pytest.raises(ValueError):
        fa.kvcache4_append(cache, n, on[:, :, 0], on[:, :, 1], stream=side)
    fa.kvcache4_append(cache, n, on[:, :, 0].contiguous(), on[:, :, 1].contiguous(), stream=side)   # the same again
    side.synchronize()
    for got, w in zip(dev, want):
        assert torch.equal(got.cpu(), w)


# ------------------------------------------------------------ reading back
READ = [
    # lens, first, page, Hkv, D, dtype
    ([1], None, 16, 1, 64, BF),
    ([40, 0, 17, 1], [3, 0, 17, 0], 16, 2, 128, F16),
    ([300, 64, 65], [299, 0, 64], 64, 8, 128, BF),
    ([700, 900, 5], None, 128, 4, 64, F16),
    ([i % 37 for i in range(300)], [i % 37 // 2 for i in range(300)], 48, 1, 64, BF),
    ([2000, 3000], [1, 7], 64, 8, 128, BF),
]


@pytest.mark.gpu
@pytest.mark.parametrize("c", READ, ids=_ids)
def test_read(fa, cuda_device, c):
    lens, first, page, H, D, dt = c
    table, pages = block_table(lens, page, extra=2, seed=page)
    host = make_cache(pages, H, page, D, 5)
    host[2][..., 0] *= 3.0
    cache = fa.KvCache4(*(t.cuda() for t in host), table.cuda())
    start = first or [0] * len(lens)
    count = [n - f for n, f in zip(lens, start)]
    rows = sum(count) + 3   # three rows of nobody
    out = tuple(torch.full((rows, H, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    got = fa.kvcache4_read(cache, ints(lens), sums(count), rows, dt, first=None if first is None else ints(first), out=out)
    assert got is out and fa.device_status() == fa.FA_OK
    new = fa.kvcache4_read(cache, ints(lens), sums(count), rows, dt, first=None if first is None else ints(first))
    for i in range(2):
        x = values(host[i], host[2 + i])
        want = torch.cat([x[table[b].long()[torch.arange(f, n) // page], :, torch.arange(f, n) % page]
                          for b, (f, n) in enumerate(zip(start, lens))])
        assert torch.equal(got[i][:-3].cpu(), want.float().to(dt))   # one rounding to 32 bits, then one to 16
        assert (got[i][-3:] == 7).all()
        assert torch.equal(new[i][:-3], got[i][:-3])


# --------------------------------------------------------------- attention
ATTEND = [
    # lens, Sq, Hq, Hkv, D, page, dtype, cap, window
    ([1], 1, 1, 1, 64, 16, BF, 0.0, -1),
    ([1, 0, 2, 63, 64, 65], 1, 4, 2, 128, 64, F16, 0.0, -1),
    ([17, 300, 0, 129], 1, 8, 1, 128, 16, BF, 30.0, -1),
    ([500, 40, 7], 1, 16, 1, 64, 32, F16, 0.0, -1),
    ([200, 3, 90], 5, 8, 2, 128, 16, BF, 0.0, -1),          # 20 rows per kv head; a length below Sq
    ([700, 64], 3, 32, 2, 64, 128, BF, 50.0, -1),           # 48 rows
    ([1000, 20, 333], 1, 4, 4, 128, 64, BF, 0.0, 100),
    ([400, 130, 6], 4, 4, 1, 64, 16, F16, 20.0, 0),         # a window of the token alone
    ([300, 4], 2, 2, 1, 128, 48, F16, 0.0, 2 ** 31 - 1),
    ([5000], 1, 2, 1, 128, 64, BF, 0.0, -1),                # cut between many workers
    ([16] * 90 + [0] * 10, 1, 2, 2, 64, 16, BF, 0.0, -1),
    ([250, 33], 1, 16, 1, 128, 96, F16, 0.0, -1),           # 16 rows; pages of three half tiles
    ([900, 5, 64], 2, 8, 1, 128, 128, F16, 25.0, 300),
    ([333, 112, 113], 1, 3, 1, 64, 112, BF, 0.0, -1),
    ([(7 * i) % 41 for i in range(700)], 1, 1, 1, 64, 16, F16, 0.0, -1),   # more sequences than threads
    ([(5 * i) % 23 for i in range(1300)], 1, 1, 1, 128, 16, BF, 0.0, -1),  # with tables in shared memory for all
    ([(5 * i) % 67 for i in range(3000)], 1, 2, 1, 64, 64, F16, 0.0, -1),  # more still
    ([400, 31, 9], 2, 4, 2, 128, 16, F16, 20.0, 70),        # four rows: capped, in a window, small pages
    ([400, 31, 9], 1, 4, 1, 64, 32, BF, 50.0, -1),
    ([77, 300], 4, 2, 2, 64, 128, F16, 0.0, 33),
]


def _attend(fa, c, seed=0, a=1.0, spread=(0.15, 0.45)):
    lens, Sq, Hq, Hkv, D, page, dt, cap, window = c
    table, pages = block_table(lens, page, extra=2, seed=seed)
    host = make_cache(pages, Hkv, page, D, seed, spread)
    # behind the last token, and in free pages, middles and scales of NaN
    used = torch.zeros((pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[int(table[b, t // page]), t % page] = True
    for s in host[2:]:
        s.copy_(torch.where(used[:, None, :, None, None], s, torch.full_like(s, math.nan)))
    q = (torch.randn((len(lens), Sq, Hq, D), generator=torch.Generator().manual_seed(seed + 1)) * a).to(dt)
    return q, fa.KvCache4(*(t.cuda() for t in host), table.cuda()), ints(lens), host + (table, lens, page)


@pytest.mark.gpu
@pytest.mark.parametrize("c", ATTEND, ids=_ids)
def test_attention_over_the_cache(fa, cuda_device, c):
    q, cache, n, plain = _attend(fa, c, a=2.0 if c[7] else 1.0)
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=c[7], window_left=c[8])
    again = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=c[7], window_left=c[8])
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    ro, rl, off, lse_off = plain_attention(q, *plain, c[4] ** -0.5, c[7], c[8])
    check(o, ro, off, "o")
    check_lse(lse, rl, lse_off)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(40))
def test_attention_of_any_sizes(fa, cuda_device, seed):
    """Sizes, pages, masks and types drawn at random."""
    r = torch.Generator().manual_seed(100 + seed)
    pick = lambda *x: x[int(torch.randint(0, len(x), (), generator=r))]   # noqa: E731
    Hkv, cap = pick(1, 2, 3), pick(0.0, 0.0, 15.0)
    lens = [int(n) for n in torch.randint(0, pick(20, 200, 900), (pick(1, 2, 5),), generator=r)]
    c = (lens, pick(1, 1, 2, 3, 5), Hkv * pick(1, 2, 3, 4, 8), Hkv, pick(64, 128), pick(16, 32, 48, 64, 80, 128), pick(BF, F16),
         cap, pick(-1, -1, 0, 15, 100))
    q, cache, n, plain = _attend(fa, c, seed, a=2.0 if cap else 1.0)
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=cap, window_left=c[8])
    assert fa.device_status() == fa.FA_OK
    ro, rl, off, lse_off = plain_attention(q, *plain, c[4] ** -0.5, cap, c[8])
    check(o, ro, off, "o of %r" % (c,))
    check_lse(lse, rl, lse_off)


@pytest.mark.gpu
def test_a_heavy_scale_nobody_looks_at(fa, cuda_device):
    """Tokens with V scales 2^40 above the others' and scores far below: their weight
    is nothing, and the others keep theirs."""
    c = ([500, 64], 1, 4, 1, 128, 16, BF, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 31, 3.0)
    ks, vs, table = plain[2], plain[3], plain[4]
    for b, tokens in enumerate(c[0]):
        for t in range(0, tokens, 7):   # a key that is a large multiple of -q: its score is about -2 |q|^2 c < -150
            at, slot = int(table[b, t // 16]), t % 16
            x = -q[b, 0].double().mean(dim=0) * 2
            code, s = _keys_like(x)
            plain[0][at, 0, slot], ks[at, 0, slot] = code, s
            vs[at, 0, slot, :, 0] *= 2.0 ** 40
    cache.k.copy_(plain[0])
    cache.k_scale.copy_(ks)
    cache.v_scale.copy_(vs)
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n)
    ro, rl, off, lse_off = plain_attention(q, *plain, 128 ** -0.5, 0.0, -1)
    check(o, ro, off, "o")
    check_lse(lse, rl, lse_off)


def _keys_like(x):
    c, s = quantise(x.float()[None])
    return c[0], s[0]


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(20))
def test_append_and_read_of_any_sizes(fa, cuda_device, seed):
    """Appends of random sizes behind each other, then everything read back."""
    r = torch.Generator().manual_seed(200 + seed)
    pick = lambda *x: x[int(torch.randint(0, len(x), (), generator=r))]   # noqa: E731
    B, H, D, page, dt = pick(1, 3, 40, 270), pick(1, 2, 5, 8), pick(64, 128), pick(16, 48, 64, 128), pick(BF, F16)
    steps = [[int(n) for n in torch.randint(0, pick(2, 9, 60), (B,), generator=r)] for _ in range(3)]
    total = [sum(x) for x in zip(*steps)]
    table, pages = block_table(total, page, extra=1, seed=seed)
    cache = fa.KvCache4(*(t.cuda() for t in make_cache(pages, H, page, D, seed)), table.cuda())
    held, want = [0] * B, [([], []) for _ in range(B)]
    for new in steps:
        if sum(new) == 0:
            continue
        kv = [torch.randn((sum(new), H, D), generator=r).to(dt) for _ in range(2)]
        fa.kvcache4_append(cache, ints(held), kv[0].cuda(), kv[1].cuda(), cu_new=sums(new), max_new=max(new))
        at = 0
        for b, n in enumerate(new):
            for i in range(2):
                want[b][i].append(kv[i][at:at + n])
            at += n
        held = [a + n for a, n in zip(held, new)]
    if sum(held) == 0:
        return
    got = fa.kvcache4_read(cache, ints(held), sums(held), sum(held), dt)
    assert fa.device_status() == fa.FA_OK
    for i in range(2):
        x = torch.cat([t for b in range(B) for t in want[b][i]])
        assert torch.equal(got[i].cpu(), values(*quantise(x)).float().to(dt))


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi,a", [(-60, 20, 1.0), (-3, 6, 20.0), (-100, -90, 1.0), (90, 100, 1.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_far_apart(fa, cuda_device, lo, hi, a, D):
    """V scales many binades apart from token to token, and zeros; sharp scores."""
    c = ([700, 33], 1, 4, 1, D, 16, BF, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 5, a)
    vs = plain[3]
    g = torch.Generator().manual_seed(6)
    w = torch.exp2(torch.randint(lo, hi, vs.shape[:-1], generator=g).float()) * (torch.rand(vs.shape[:-1], generator=g) + 0.5)
    w[torch.rand(w.shape, generator=g) < 0.1] = 0.0
    mid = w * torch.randn(w.shape, generator=g)
    live = torch.isfinite(vs[..., 0].float())
    vs.copy_(torch.where(live[..., None], torch.stack([w, mid], dim=-1).to(BF), vs))
    cache.v_scale.copy_(vs)
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n)
    ro, rl, off, lse_off = plain_attention(q, *plain, D ** -0.5, 0.0, -1)
    check(o, ro, off, "o")
    check_lse(lse, rl, lse_off)


@pytest.mark.gpu
def test_no_scale_at_all(fa, cuda_device):
    """Scales of zero everywhere: the middles alone."""
    c = ([200, 1], 1, 4, 2, 128, 32, F16, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 9)
    for s, on in ((plain[2], cache.k_scale), (plain[3], cache.v_scale)):
        s[..., 0] = 0.0
        on.copy_(s)
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n)
    ro, rl, off, lse_off = plain_attention(q, *plain, 128 ** -0.5, 0.0, -1)
    check(o, ro, off, "o")
    check_lse(lse, rl, lse_off)


@pytest.mark.gpu
def test_nan_and_range_of_queries(fa, cuda_device):
    """bf16 queries far outside f16's range, and a NaN one."""
    c = ([100, 100], 1, 2, 1, 64, 16, BF, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 7)
    q[0, 0, 0] = (q[0, 0, 0].float() * 1e-30).to(BF)
    q[0, 0, 1] = (q[0, 0, 1].float() * 1e6).to(BF)
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softmax_scale=1e-6)
    ro, rl, off, _ = plain_attention(q, *plain, 1e-6, 0.0, -1)
    check(o, ro, off, "o")
    q[1, 0, 1, 3] = float("nan")
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softmax_scale=1e-6)
    assert torch.isnan(o[1, 0, 1]).all() and torch.isnan(lse[1, 1, 0])
    check(torch.cat([o[0, 0], o[1, 0, :1]]), torch.cat([ro[0, 0], ro[1, 0, :1]]), torch.cat([off[0, 0], off[1, 0, :1]]), "o")


@pytest.mark.gpu
def test_nan_in_the_cache(fa, cuda_device):
    """A token appended with a NaN: rows that see it are NaN, others are not."""
    c = ([50, 60], 2, 2, 1, 64, 16, BF, 0.0, 3)
    q, cache, n, plain = _attend(fa, c, 8)
    want, _ = fa.fa_fwd_kvcache4(q.cuda(), cache, n, window_left=3)
    bad = int(plain[4][0, 49 // 16])
    cache.k_scale[bad, 0, 49 % 16, 0, 1] = math.nan   # the last token of sequence 0: its last query's alone
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, window_left=3)
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, :, 1]).all()
    assert torch.equal(o[1], want[1]) and torch.equal(o[0, 0], want[0, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("D,Sq", [(64, 1), (128, 3)])
def test_before_the_window(fa, cuda_device, D, Sq):
    """Tokens no query sees any more are not looked at, nor table entries of pages
    wholly before the window."""
    c = ([300, 41, 64], Sq, 4, 2, D, 32, F16, 0.0, 20)
    q, cache, n, plain = _attend(fa, c, 23)
    want = fa.fa_fwd_kvcache4(q.cuda(), cache, n, window_left=20)
    for b, tokens in enumerate(c[0]):
        for t in range(tokens - Sq - 20):
            at = int(plain[4][b, t // c[5]])
            cache.k_scale[at, :, t % c[5]] = math.nan
            cache.v_scale[at, :, t % c[5]] = math.nan
    cache.block_table[0, :(300 - Sq - 20) // 32] = -1
    got = fa.fa_fwd_kvcache4(q.cuda(), cache, n, window_left=20)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(got[0]).all() and fa.device_status() == fa.FA_OK


@pytest.mark.gpu
def test_streams(fa, cuda_device):
    """Calls for another stream than the current one, and in flight together."""
    c = ([3000, 900, 17], 1, 8, 2, 128, 64, BF, 0.0, -1)
    d = ([100, 2000], 1, 8, 1, 64, 32, F16, 30.0, -1)
    runs = [_attend(fa, c, 14), _attend(fa, d, 15)]
    q = [r[0].cuda() for r in runs]
    rows = [sum(c[0]), sum(d[0])]
    call = [lambda i, x, **kw: fa.fa_fwd_kvcache4(q[i], runs[i][1], runs[i][2], softcap=x[7], **kw),
            lambda i, x, **kw: fa.kvcache4_read(runs[i][1], runs[i][2], cu[i], rows[i], x[6], **kw)]
    cu = [sums(c[0]), sums(d[0])]
    want = [[f(i, x) for f in call] for i, x in enumerate((c, d))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for turn in range(20):
        busy = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]
        for i, x in enumerate((c, d)):
            if turn % 2:
                got[i].append([f(i, x, stream=streams[i]) for f in call])
            else:
                with torch.cuda.stream(streams[i]):
                    got[i].append([f(i, x) for f in call])
        del busy
    torch.cuda.synchronize()
    for i in range(2):
        for both in got[i]:
            for a, b in zip(both, want[i]):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_far_pages(fa, cuda_device):
    """Page offsets past 2^32 bytes, in all three calls."""
    H, page, D = 2, 64, 128
    pages = (1 << 32) // (H * page * D // 2) + 40
    k, v = (torch.zeros((pages, H, page, D // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, H, page, 2, 2), dtype=BF, device="cuda") for _ in range(2))
    lens = [100, 70]
    table = torch.tensor([[pages - 1, 3], [pages - 20, pages - 7]], dtype=torch.int32)
    cache = fa.KvCache4(k, v, ks, vs, table.cuda())
    g = torch.Generator().manual_seed(9)
    kn, vn = (torch.randn((170, H, D), generator=g).to(BF) for _ in range(2))
    fa.kvcache4_append(cache, ints([0, 0]), kn.cuda(), vn.cuda(), cu_new=ints([0, 100, 170]), max_new=100)
    back = fa.kvcache4_read(cache, ints(lens), ints([0, 100, 170]), 170)
    for x, y in zip((kn, vn), back):
        assert torch.equal(values(*quantise(x)).float().to(BF), y.cpu())
    q = torch.randn((2, 1, 4, D), generator=g).to(BF)
    o, _ = fa.fa_fwd_kvcache4(q.cuda(), cache, ints(lens))
    small = [torch.stack([t[p].cpu() for p in table.flatten().tolist()]) for t in (k, v, ks, vs)]
    ro, _, off, _ = plain_attention(q, *small, torch.arange(4, dtype=torch.int32).view(2, 2), lens, page, D ** -0.5, 0.0, -1)
    check(o, ro, off, "o")


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_reported(fa, cuda_device):
    """Found on the device by the kernels' own checks; the other sequences are served."""
    c = ([40, 50, 60], 1, 2, 1, 64, 16, BF, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 10)
    want, _ = fa.fa_fwd_kvcache4(q.cuda(), cache, n)
    table = cache.block_table.clone()
    for bad in (-1, 10 ** 6, 65):   # 65: beyond the table of 4 pages
        n2 = n.clone()
        n2[1] = bad
        o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n2)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG and fa.device_status() == fa.FA_OK
        assert torch.equal(o[[0, 2]], want[[0, 2]]) and (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    cu = ints([0, 5, 10, 15])
    full = fa.kvcache4_read(cache, n, cu, 15)
    for bad in (-1, cache.k.shape[0], 2 ** 31 - 1):
        cache.block_table[1, 0] = bad
        o, _ = fa.fa_fwd_kvcache4(q.cuda(), cache, n)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
        assert torch.equal(o[[0, 2]], want[[0, 2]]) and torch.isfinite(o).all()
        got = fa.kvcache4_read(cache, n, cu, 15, out=tuple(torch.zeros_like(t) for t in full))
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
        for a, b in zip(got, full):
            assert torch.equal(a[:5], b[:5]) and (a[5:10] == 0).all() and torch.equal(a[10:], b[10:])
        cache.block_table.copy_(table)
    # reading what is not held: too many rows, a start below 0 or behind the end, a length past the table, sums that fall
    for lens, first, cu_bad, left in (([40, 4, 60], None, [0, 5, 10, 15], [1]), ([40, 50, 60], [0, -1, 0], [0, 5, 10, 15], [1]),
                                      ([40, 50, 60], [0, 46, 0], [0, 5, 10, 15], [1]), ([40, 65, 60], None, [0, 5, 10, 15], [1]),
                                      ([40, 50, 60], None, [0, 5, 10, 16], [2])):
        got = fa.kvcache4_read(cache, ints(lens), ints(cu_bad), 15, first=None if first is None else ints(first),
                               out=tuple(torch.zeros_like(t) for t in full))
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG and fa.device_status() == fa.FA_OK
        for a, b in zip(got, full):
            for s in range(3):
                assert torch.equal(a[5 * s:5 * s + 5], b[5 * s:5 * s + 5] * (s not in left))
    for cu_bad in ([0, 7, 3, 15], [-5, 5, 10, 15], [2 ** 31 - 1, -2 ** 31, 5, 15]):
        fa.kvcache4_read(cache, n, ints(cu_bad), 15)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
    x = torch.ones((3, 5, 1, 64), dtype=BF, device="cuda")
    before = [t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]

    def untouched():
        for t, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
            assert torch.equal(t.view(torch.uint8), w)
    # a length below 0, a bad page, tokens past the table
    for lens in ([-1, 55, 63], [62, 63, 64]):
        if lens[0] < 0:
            cache.block_table[1, 3] = 77
        fa.kvcache4_append(cache, ints(lens), x, x)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
        cache.block_table.copy_(table)
        untouched()
    # rows past the tensor, more than max_new, sums that fall
    y = x.view(15, 1, 64)
    for cu_bad, most in (([0, 0, 0, 16], 16), ([0, 6, 6, 6], 5), ([16, 16, 16, 16], 5)):
        fa.kvcache4_append(cache, ints([0, 0, 0]), y, y, cu_new=ints(cu_bad), max_new=most)
        assert fa.device_status() == (fa.FA_ERR_INVALID_ARG)
        untouched()


@pytest.mark.gpu
@pytest.mark.parametrize("D,cap,dt,scaling", [(128, 30.0, BF, None), (64, 0.0, F16, ("yarn", 8.0, 4096))])
def test_serving_run(fa, cuda_device, D, cap, dt, scaling):
    """Prompts and then tokens one at a time: q and k turned by their positions, k and v
    into the cache, attention over it; a step captured once and replayed.  Then a chunk of
    prompt: the cache read back and the dense attention over it."""
    prompts, steps, page, Hq, Hkv = [37, 1, 64], 20, 16, 4, 2
    B, more = len(prompts), 10
    g = torch.Generator().manual_seed(11)
    r = lambda n, h: torch.randn((n, h, D), generator=g).to(dt)   # noqa: E731
    ks_, vs_, qs = ([r(n + steps + more, h) for n in prompts] for h in (Hkv, Hkv, Hq))
    table, pages = block_table([n + steps + more for n in prompts], page, seed=12)
    cache = fa.KvCache4(*(t.cuda() for t in make_cache(pages, Hkv, page, D, 13)), table.cuda())
    turns = fa.rope_table(D, scaling=scaling)
    pos = torch.cat([torch.arange(m) for m in prompts]).int().cuda()
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    pk, pv = (torch.cat([x[:m] for x, m in zip(t, prompts)]).cuda() for t in (ks_, vs_))
    pk, _ = fa.rope(pk, None, turns, positions=pos, out=(pk, None))   # in place
    fa.kvcache4_append(cache, n, pk, pv, cu_new=sums(prompts), max_new=64)
    n += ints(prompts)
    newk, newv = (torch.empty((B, 1, Hkv, D), dtype=dt, device="cuda") for _ in range(2))
    q = torch.empty((B, 1, Hq, D), dtype=dt, device="cuda")
    turned = torch.empty_like(q), torch.empty_like(newk)
    ws = torch.empty(fa.fa_fwd_kvcache4_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")

    def step():
        fa.rope(q, newk, turns, offsets=n, out=turned)
        fa.kvcache4_append(cache, n, turned[1], newv)
        n.add_(1)
        fa.fa_fwd_kvcache4(turned[0], cache, n, softcap=cap, workspace=ws, out=out)
    graph = None
    for t in range(steps):
        for dst, src in ((newk, ks_), (newv, vs_), (q, qs)):
            dst.copy_(torch.stack([x[m + t] for x, m in zip(src, prompts)])[:, None])
        if t == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay() if graph else step()
        torch.cuda.synchronize()
        lens = [m + t + 1 for m in prompts]
        assert n.tolist() == lens
        w, f = fa.rope_frequencies(D, scaling=scaling)
        for b in range(B):
            angle = (lens[b] - 1) * w
            for x, y in ((qs[b][lens[b] - 1], turned[0][b, 0]), (ks_[b][lens[b] - 1], turned[1][b, 0])):
                c, s = f * angle.cos(), f * angle.sin()
                a, d = x.double().chunk(2, dim=-1)
                want = torch.cat([a * c - d * s, d * c + a * s], dim=-1)
                size = f * (torch.cat([a, a], dim=-1).abs() + torch.cat([d, d], dim=-1).abs())
                check(y, want, U[dt] * want.abs() + 2.0 ** -22 * size + SUB[dt], "turned")
        ro, _, off, _ = plain_attention(turned[0].cpu(), cache.k.cpu(), cache.v.cpu(), cache.k_scale.cpu(),
                                        cache.v_scale.cpu(), table, lens, page, D ** -0.5, cap, -1)
        check(out[0], ro, off, "step %d" % t)
    # a chunk of `more` tokens a sequence
    chunk = [torch.stack([x[m + steps:m + steps + more] for x, m in zip(t, prompts)]).cuda() for t in (qs, ks_, vs_)]
    cq, ck = fa.rope(chunk[0], chunk[1], turns, offsets=n)
    fa.kvcache4_append(cache, n, ck, chunk[2])
    n += more
    lens = [m + steps + more for m in prompts]
    k, v = fa.kvcache4_read(cache, n, sums(lens), sum(lens), dt)
    dense, lse = fa.fa_fwd(cq.view(-1, Hq, D), k, v, causal=True, softcap=cap, cu_seqlens_q=sums([more] * B),
                           cu_seqlens_k=sums(lens), max_seqlen_q=more, max_seqlen_k=max(lens))
    over, olse = fa.fa_fwd_kvcache4(cq, cache, n, softcap=cap)
    assert fa.device_status() == fa.FA_OK
    ro, rl, off, lse_off = plain_attention(cq.cpu(), cache.k.cpu(), cache.v.cpu(), cache.k_scale.cpu(), cache.v_scale.cpu(),
                                           table, lens, page, D ** -0.5, cap, -1)
    check(over, ro, off, "chunk over the cache")
    check_lse(olse, rl, lse_off)
    # the dense attention reads values rounded to 16 bits: each score moves by u sum |q||k| c, twice in the
    # weights, which average |v| < 16 scale + |middle| < 9; P and V are rounded as well
    u = U[dt]
    moved = u * float((cq.double().abs().amax(dim=(0, 1, 2)).cpu() * k.double().abs().amax(dim=(0, 1)).cpu()).sum()) * D ** -0.5
    assert (dense.view(B, more, Hq, D).double().cpu() - ro).abs().max() <= (2 * moved + 3 * u) * float(v.abs().max())


# ------------------------------------------------------- refusals (no GPU)
def _struct(fa, **over):
    a = dict(k=0x1000, v=0x2000, k_scale=0x3000, v_scale=0x4000, block_table=0x5000, num_pages=10, page_size=64,
             max_pages=4, Hkv=2, D=128)
    a.update(over)
    return fa._KvCacheStruct(**a)


def _append4(fa, s, **over):
    a = dict(len=0x6000, k=0x7000, v=0x8000, cu=0, rows=15, B=3, max_new=5, dtype=0)
    a.update(over)
    vp = ctypes.c_void_p
    return fa.lib().fa_kvcache4_append(ctypes.byref(s), vp(a["len"]), vp(a["k"]), vp(a["v"]), vp(a["cu"]), a["rows"],
                                       a["B"], a["max_new"], a["dtype"], None)


def _read4(fa, s, **over):
    a = dict(len=0x6000, first=0, cu=0x9000, rows=15, B=3, k=0x7000, v=0x8000, dtype=0)
    a.update(over)
    vp = ctypes.c_void_p
    return fa.lib().fa_kvcache4_read(ctypes.byref(s), vp(a["len"]), vp(a["first"]), vp(a["cu"]), a["rows"], a["B"],
                                     vp(a["k"]), vp(a["v"]), a["dtype"], None)


def _attn4(fa, s, **over):
    a = dict(q=0x7000, len=0x6000, o=0x8000, lse=0, B=3, Sq=1, Hq=4, scale=0.1, cap=0.0, window=-1, dtype=0,
             ws=0x10000, nbytes=1 << 30)
    a.update(over)
    vp = ctypes.c_void_p
    return fa.lib().fa_fwd_kvcache4(vp(a["q"]), ctypes.byref(s), vp(a["len"]), vp(a["o"]), vp(a["lse"]), a["B"],
                                    a["Sq"], a["Hq"], a["scale"], a["cap"], a["window"], a["dtype"], vp(a["ws"]),
                                    a["nbytes"], None)


@pytest.mark.parametrize("over,status", [
    (dict(k=0), 1), (dict(v_scale=0), 1), (dict(k_scale=0), 1), (dict(block_table=0), 1), (dict(k=0x1008), 1),
    (dict(v=0x2004), 1), (dict(k_scale=0x3008), 1), (dict(v_scale=0x4004), 1), (dict(block_table=0x5002), 1),
    (dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(page_size=-64), 1), (dict(max_pages=0), 1), (dict(Hkv=0), 1),
    (dict(page_size=24), 2), (dict(page_size=256), 2), (dict(D=96), 2), (dict(D=256), 2), (dict(max_pages=1 << 30), 1)])
def test_bad_caches_refused(fa, over, status):
    for call in (_append4, _read4, _attn4):
        assert call(fa, _struct(fa, **over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(len=0), 1), (dict(k=0), 1), (dict(v=0x8004), 1), (dict(k=0x7008), 1), (dict(cu=0x9002), 1),
    (dict(len=0x6001), 1), (dict(B=0), 1), (dict(max_new=0), 1), (dict(dtype=5), 2),
    (dict(B=1 << 20, max_new=1 << 20), 1), (dict(rows=14), 1), (dict(rows=16), 1), (dict(rows=0, cu=0x9000), 1)])
def test_append_refused(fa, over, status):
    assert _append4(fa, _struct(fa), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(len=0), 1), (dict(cu=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(k=0x7008), 1), (dict(v=0x8004), 1),
    (dict(first=0x9002), 1), (dict(cu=0x9001), 1), (dict(len=0x6001), 1), (dict(rows=0), 1), (dict(B=0), 1),
    (dict(dtype=7), 2)])
def test_read_refused(fa, over, status):
    assert _read4(fa, _struct(fa), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(q=0), 1), (dict(o=0), 1), (dict(len=0), 1), (dict(q=0x7008), 1), (dict(lse=0x9002), 1),
    (dict(B=-1), 1), (dict(Sq=0), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(cap=-3.0), 1), (dict(cap=1e-5), 1), (dict(cap=float("inf")), 1),
    (dict(cap=0.001, scale=3e38), 1), (dict(window=-2), 1), (dict(ws=0), 1), (dict(ws=0x10080), 1),
    (dict(nbytes=1000), 1), (dict(B=4097), 2), (dict(dtype=9), 2), (dict(Sq=1 << 24), 2)])
def test_attention_refused(fa, over, status):
    assert _attn4(fa, _struct(fa), **over) == status


def test_too_many_rows_refused(fa):
    assert _attn4(fa, _struct(fa, num_pages=1 << 24, page_size=64, Hkv=2)) == 2   # 2^31 rows
    for call in (_append4, _read4):
        assert call(fa, _struct(fa, Hkv=(1 << 20) + 1)) == 2


def test_python_refusals(fa):
    k = torch.zeros((4, 2, 16, 32), dtype=torch.uint8)
    s = torch.ones((4, 2, 16, 1, 2), dtype=BF)
    t = torch.zeros((1, 4), dtype=torch.int32)
    for bad in ((k, k, s, s, t), (k.view(torch.int8), k, s, s, t), (k, k[:3], s, s, t), (k, k, s.half(), s, t),
                (k, k, s[..., :1], s, t)):
        with pytest.raises(ValueError):
            fa.KvCache4(*bad)   # the first: not on the GPU
    assert fa.fa_fwd_kvcache4_workspace_bytes(96) == 0 and fa.fa_fwd_kvcache4_workspace_bytes(128) > 0
    # one kind of cache is not the other: its tensors are of another size
    eight, four = fa.KvCache.__new__(fa.KvCache), fa.KvCache4.__new__(fa.KvCache4)
    x = torch.zeros((1, 1, 2, 64), dtype=BF)
    for cache, calls in ((eight, (fa.kvcache4_append, fa.kvcache4_read)), (four, (fa.kvcache_append,))):
        for call in calls:
            with pytest.raises(ValueError, match="cache: a KvCache"):
                call(cache, t, x, x)
    with pytest.raises(ValueError, match="cache: a KvCache4"):
        fa.fa_fwd_kvcache4(x, eight, t)
    with pytest.raises(ValueError, match="cache: a KvCache"):
        fa.fa_fwd_kvcache(x, four, t)


@pytest.mark.gpu
def test_gpu_side_refusals(fa, cuda_device):
    c = ([40, 50], 1, 2, 1, 64, 16, BF, 0.0, -1)
    q, cache, n, _ = _attend(fa, c, 16)
    with pytest.raises(ValueError):
        fa.fa_fwd_kvcache4(q, cache, n)                                  # q on the CPU
    q = q.cuda()
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[..., :32]), dict(n=n.long()), dict(n=n[:1]), dict(n=n.cpu())):
        with pytest.raises(ValueError):
            fa.fa_fwd_kvcache4(bad.get("q", q), cache, bad.get("n", n))
    with pytest.raises(fa.FaError):
        fa.fa_fwd_kvcache4(q, cache, n, softcap=-1.0)
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    with pytest.raises(fa.FaError):
        fa.fa_fwd_kvcache4(q, cache, n, workspace=small)
    # a strided q is read as it is meant
    wide = torch.cat([q, q], dim=3)[..., 64:]
    a, b = fa.fa_fwd_kvcache4(wide, cache, n), fa.fa_fwd_kvcache4(q, cache, n)
    assert torch.equal(a[0], b[0])
    x = torch.zeros((2, 1, 1, 64), dtype=BF, device="cuda")
    for k, v in ((x, x.half()), (x[:1], x[:1]), (x[..., :32], x[..., :32]), (x, x.cpu()), (x.float(), x.float())):
        with pytest.raises(ValueError):
            fa.kvcache4_append(cache, n, k, v)
    cu = ints([0, 1, 2])
    with pytest.raises(ValueError):
        fa.kvcache4_append(cache, n, x[:, 0], x[:, 0], cu_new=cu)        # max_new
    for bad in (dict(cu=cu[:2]), dict(cu=cu.long()), dict(n=n[:1]), dict(rows=0), dict(dtype=torch.float32),
                dict(first=cu), dict(out=(x, x)), dict(out=(x.view(2, 1, 64), x.view(2, 1, 64).half()))):
        with pytest.raises(ValueError):
            fa.kvcache4_read(cache, bad.get("n", n), bad.get("cu", cu), bad.get("rows", 2), bad.get("dtype", BF),
                             first=bad.get("first"), out=bad.get("out"))
