"""The 8-bit paged cache: appending (bytes and scales exact) and attention over
it, against plain 64-bit forms; a serving run; refusals on the CPU."""
import ctypes
import math

import pytest
import torch

from score_ref import SUB, U, check, eps, lse_bound

F16, BF, F8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


# ------------------------------------------------------------ plain forms
def round_e4m3(x):
    """float64 to the nearest e4m3 value (ties to even), saturating; NaN stays."""
    a = x.abs().clamp(max=448.0)
    e = torch.frexp(a).exponent.double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.where(torch.isnan(x), x, torch.sign(x) * torch.clamp(torch.round(a / step) * step, max=448.0))


def exponent(amax):
    """Smallest e in [-120, 120] with amax <= 448 2^e."""
    e = -120
    while e < 120 and amax > math.ldexp(448.0, e):
        e += 1
    return e


def plain_append(kc, vc, ks, vs, table, lens, news, page):
    """In place on float64 caches kc / vc, both [pages, H, page, D], and scales.
    ``news``: per sequence (k, v), [n, H, D]."""
    for b, pair in enumerate(news):
        for cache, scale, x in zip((kc, vc), (ks, vs), pair):
            x = x.double()
            for p in range(lens[b] // page, (lens[b] + len(x) + page - 1) // page):
                a, z = max(lens[b], p * page), min(lens[b] + len(x), (p + 1) * page)
                if a >= z:
                    continue
                at = int(table[b, p])
                for h in range(x.shape[1]):
                    new = x[a - lens[b]:z - lens[b], h]
                    fin = new[torch.isfinite(new)]
                    s = math.ldexp(1.0, exponent(float(fin.abs().max()) if fin.numel() else 0.0))
                    if a > p * page:
                        s = max(s, float(scale[at, h]))
                        held = slice(0, a - p * page)
                        cache[at, h, held] = round_e4m3(cache[at, h, held] * (float(scale[at, h]) / s))
                    scale[at, h] = s
                    cache[at, h, a - p * page:z - p * page] = round_e4m3(new / s)


def make_cache(pages, H, page, D, seed, spread=(-5, -2)):
    """Random caches: float8 CPU tensors k [.., page, D], v [.., D, page] and power-of-two scales."""
    g = torch.Generator().manual_seed(seed)
    k = (torch.randn((pages, H, page, D), generator=g) * 16).to(F8)
    v = (torch.randn((pages, H, D, page), generator=g) * 16).to(F8)
    s = [torch.exp2(torch.randint(spread[0], spread[1], (pages, H), generator=g).float()) for _ in range(2)]
    return k, v, s[0], s[1]


def block_table(lens, page, extra=0, seed=0, width=None):
    need = [max(0, -(-n // page)) for n in lens]
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(sum(need) + extra, generator=g).int()
    t = torch.full((len(lens), width or max(need + [1])), -5, dtype=torch.int32)   # unused entries: no page
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, sum(need) + extra


def f64(x):
    return x.float().double()


def plain_attention(q, k, v, ks, vs, table, lens, page, scale, cap, window):
    """(o, lse, bound) in 64 bits, per sequence and head; float8 caches."""
    B, Sq, Hq, D = q.shape
    Hkv, k, v = k.shape[1], f64(k), f64(v)
    o = torch.zeros((B, Sq, Hq, D), dtype=torch.float64)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64)
    bound = torch.zeros_like(o)
    for b, n in enumerate(lens):
        for i in range(Sq):
            pos = n - Sq + i
            if pos < 0:
                continue
            lo = max(0, pos - window) if window >= 0 else 0
            rows = torch.arange(lo, pos + 1)
            at, slot = table[b].long()[rows // page], rows % page
            for h in range(Hq):
                hk = h * Hkv // Hq
                kk = k[at, hk, slot] * ks[at, hk].double()[:, None]
                vb = v[at, hk, :, slot]
                vv = vb * vs[at, hk].double()[:, None]
                s = kk @ q[b, i, h].double() * scale
                if cap:
                    s = cap * torch.tanh(s / cap)
                lse[b, h, i] = torch.logsumexp(s, dim=0)
                p = torch.exp(s - lse[b, h, i])
                o[b, i, h] = p @ vv
                # P in f16 (2^-11 relative, 2^-25 of the largest P x scale in absolute terms)
                top = float((p * vs[at, hk].double()).max())
                bound[b, i, h] = (2.0 ** -11 + eps(cap)) * (p @ vv.abs()) + 2.0 ** -25 * top * vb.abs().sum(dim=0)
    return o, lse, bound + U[q.dtype] * o.abs() + SUB[q.dtype]


# --------------------------------------------------------------- appending
APPEND = [
    # lens, new tokens, page, Hkv, D, dtype, magnitude of the new values
    ([0], [1], 16, 1, 64, BF, 1.0),
    ([0, 15, 16, 17], [1, 1, 1, 1], 16, 2, 128, F16, 1.0),
    ([0, 63, 64, 100, 5], [200, 2, 64, 1, 0], 64, 2, 128, BF, 3.0),
    ([3, 30], [40, 77], 32, 1, 64, F16, 100.0),
    ([7, 120, 250], [1, 9, 130], 128, 3, 128, BF, 1e-3),
    ([9, 40], [3, 30], 48, 2, 64, BF, 1e30),     # the held tokens' scale grows by many steps
    ([9, 40], [3, 30], 16, 1, 128, BF, 1e-38),   # the smallest scale
    ([5, 5], [4, 4], 16, 1, 64, F16, 0.0),       # all zeros
]


@pytest.mark.gpu
@pytest.mark.parametrize("c", APPEND, ids=lambda c: "len%s_new%s_p%d_h%d_d%d_%s_x%g" % (
    "-".join(map(str, c[0])), "-".join(map(str, c[1])), c[2], c[3], c[4], str(c[5])[6:], c[6]))
def test_append(fa, cuda_device, c):
    lens, new, page, H, D, dt, size = c
    table, pages = block_table([a + n for a, n in zip(lens, new)], page, extra=3, seed=page)
    k, v, ks, vs = make_cache(pages, H, page, D, 1)
    g = torch.Generator().manual_seed(2)
    news = [tuple((torch.randn((n, H, D), generator=g) * size).to(dt) for _ in range(2)) for n in new]
    if size == 1.0:
        news[-1][0][0, 0, 3] = float("inf")
        news[-1][1][0, -1, 5] = float("nan")
        news[-1][1][0, 0, 6] = -float("inf")
    dev = [t.cuda() for t in (k, v, ks, vs)]
    cache = fa.KvCache(*dev, table.cuda())
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32).cuda()
    fa.kvcache_append(cache, torch.tensor(lens, dtype=torch.int32).cuda(), torch.cat([n[0] for n in news]).cuda(),
                      torch.cat([n[1] for n in news]).cuda(), cu_new=cu, max_new=max(new))
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    want = [f64(k), f64(v).transpose(2, 3).contiguous(), ks.double(), vs.double()]
    plain_append(*want, table, lens, news, page)
    for got, w, name in zip(dev, (want[0], want[1].transpose(2, 3), want[2], want[3]), ("k", "v", "k_scale", "v_scale")):
        got = f64(got.cpu())
        same = (got == w) | (torch.isnan(got) & torch.isnan(w))
        assert same.all(), (name, int((~same).sum()), got[~same][:5], w[~same][:5])


@pytest.mark.gpu
def test_append_every_sequence_the_same(fa, cuda_device):
    """The [B, T, Hkv, D] form, on a stream of its own, from a strided tensor."""
    lens, T, page, H, D = [10, 0, 31], 5, 16, 2, 64
    table, pages = block_table([n + T for n in lens], page)
    k, v, ks, vs = make_cache(pages, H, page, D, 3)
    g = torch.Generator().manual_seed(4)
    kv = torch.randn((3, T, 2, H, D), generator=g).to(BF)
    dev = [t.cuda() for t in (k, v, ks, vs)]
    cache = fa.KvCache(*dev, table.cuda())
    on, n = kv.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.kvcache_append(cache, n, on[:, :, 0], on[:, :, 1])
    side.synchronize()
    want = [f64(k), f64(v).transpose(2, 3).contiguous(), ks.double(), vs.double()]
    plain_append(*want, table, lens, [(kv[b, :, 0], kv[b, :, 1]) for b in range(3)], page)
    for got, w in zip(dev, (want[0], want[1].transpose(2, 3), want[2], want[3])):
        assert torch.equal(f64(got.cpu()), w)
    with pytest.raises(ValueError):
        fa.kvcache_append(cache, n, on[:, :, 0], on[:, :, 1], stream=side)


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
    ([250, 33], 1, 16, 1, 128, 96, F16, 0.0, -1),           # 16 rows, three parts of Q; pages of three half tiles
    ([900, 5, 64], 2, 8, 1, 128, 128, F16, 25.0, 300),
    ([333, 112, 113], 1, 3, 1, 64, 112, BF, 0.0, -1),
    ([(7 * i) % 41 for i in range(700)], 1, 1, 1, 64, 16, F16, 0.0, -1),   # more sequences than threads
]


def _attend(fa, c, seed=0, spread=(-5, -2), a=1.0):
    lens, Sq, Hq, Hkv, D, page, dt, cap, window = c
    table, pages = block_table(lens, page, extra=2, seed=seed)
    k, v, ks, vs = make_cache(pages, Hkv, page, D, seed, spread)
    # what lies behind the last token, and in free pages: NaN, with scales of NaN in the latter
    used = torch.zeros((pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[int(table[b, t // page]), t % page] = True
    nan = torch.tensor(0x7F, dtype=torch.uint8)
    k.view(torch.uint8)[:] = torch.where(used[:, None, :, None], k.view(torch.uint8), nan)
    v.view(torch.uint8)[:] = torch.where(used[:, None, None, :], v.view(torch.uint8), nan)
    ks[~used.any(dim=1)] = float("nan")
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((len(lens), Sq, Hq, D), generator=g) * a).to(dt)
    cache = fa.KvCache(*(t.cuda() for t in (k, v, ks, vs)), table.cuda())
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    return q, cache, n, (k, v, ks, vs, table, lens, page)


@pytest.mark.gpu
@pytest.mark.parametrize("c", ATTEND, ids=lambda c: "len%s_q%d_h%d_%d_d%d_p%d_%s_cap%g_w%d" % (
    ("-".join(map(str, c[0][:6])),) + c[1:6] + (str(c[6])[6:],) + c[7:]))
def test_attention_over_the_cache(fa, cuda_device, c):
    q, cache, n, plain = _attend(fa, c, a=2.0 if c[7] else 1.0)
    scale = c[4] ** -0.5
    o, lse = fa.fa_fwd_kvcache(q.cuda(), cache, n, softcap=c[7], window_left=c[8])
    again = fa.fa_fwd_kvcache(q.cuda(), cache, n, softcap=c[7], window_left=c[8])
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    ro, rl, bound = plain_attention(q, *plain, scale, c[7], c[8])
    check(o, ro, bound, "o")
    lg = lse.double().cpu()
    assert torch.equal(torch.isneginf(lg), torch.isneginf(rl))
    fin = torch.isfinite(rl)
    assert ((lg - rl)[fin].abs() <= lse_bound(c[7], rl)[fin]).all()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("spread,a", [((-40, 20), 1.0), ((-3, -2), 20.0), ((-110, -90), 1.0)])
def test_scales_far_apart(fa, cuda_device, spread, a):
    """V scales many binades apart in one sequence, sharp scores, tiny scales.
    K scales stay ordinary in the first two: scores beyond f32 are not the point."""
    c = ([700, 33], 1, 4, 1, 128, 16, BF, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 5, (-6, -4), a)
    k, v, ks, vs = plain[:4]
    g = torch.Generator().manual_seed(6)
    vs[:] = torch.exp2(torch.randint(spread[0], spread[1], vs.shape, generator=g).float())
    cache.v_scale.copy_(vs)
    o, lse = fa.fa_fwd_kvcache(q.cuda(), cache, n)
    ro, rl, bound = plain_attention(q, *plain, 128 ** -0.5, 0.0, -1)
    # sharp scores: the 32-bit score error grows with them (2^-21 of sum |q||k| c, below 64 a here)
    check(o, ro, bound * max(1.0, a / 2), "o")
    fin = torch.isfinite(rl)
    assert ((lse.double().cpu() - rl)[fin].abs() <= max(1.0, a / 2) * lse_bound(0.0, rl)[fin]).all()


@pytest.mark.gpu
def test_nan_and_range_of_queries(fa, cuda_device):
    """bf16 queries far outside f16's range, and a NaN one."""
    c = ([100, 100], 1, 2, 1, 64, 16, BF, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 7)
    q[0, 0, 0] = (q[0, 0, 0].float() * 1e-30).to(BF)
    q[0, 0, 1] = (q[0, 0, 1].float() * 1e6).to(BF)
    o, lse = fa.fa_fwd_kvcache(q.cuda(), cache, n, softmax_scale=1e-6)
    ro, rl, bound = plain_attention(q, *plain, 1e-6, 0.0, -1)
    check(o, ro, bound, "o")
    q[1, 0, 1, 3] = float("nan")
    o, lse = fa.fa_fwd_kvcache(q.cuda(), cache, n, softmax_scale=1e-6)
    assert torch.isnan(o[1, 0, 1]).all() and torch.isnan(lse[1, 1, 0])
    check(torch.cat([o[0, 0], o[1, 0, :1]]), torch.cat([ro[0, 0], ro[1, 0, :1]]), torch.cat([bound[0, 0], bound[1, 0, :1]]), "o")


@pytest.mark.gpu
def test_window_leaves_old_pages_alone(fa, cuda_device):
    """Table entries of pages wholly before the window are not read."""
    c = ([400], 1, 4, 2, 64, 16, BF, 0.0, 50)
    q, cache, n, plain = _attend(fa, c, 8)
    want = fa.fa_fwd_kvcache(q.cuda(), cache, n, window_left=50)
    cache.block_table[0, :(399 - 50) // 16] = -1
    got = fa.fa_fwd_kvcache(q.cuda(), cache, n, window_left=50)
    assert torch.equal(want[0], got[0]) and fa.device_status() == fa.FA_OK


@pytest.mark.gpu
def test_other_scales(fa, cuda_device):
    """A cache filled elsewhere: scales that are no powers of two, and zeros."""
    c = ([300, 41, 64], 1, 4, 2, 64, 32, BF, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 21)
    g = torch.Generator().manual_seed(22)
    for s, on in ((plain[2], cache.k_scale), (plain[3], cache.v_scale)):
        s.mul_(torch.rand(s.shape, generator=g) + 0.5)
        s[torch.rand(s.shape, generator=g) < 0.3] = 0.0
        on.copy_(s)
    o, lse = fa.fa_fwd_kvcache(q.cuda(), cache, n)
    ro, rl, bound = plain_attention(q, *plain, 64 ** -0.5, 0.0, -1)
    # the V scale enters P through its logarithm, |log2| < 8 and off by 2^-22 of that: inside eps
    check(o, ro, bound, "o")
    assert ((lse.double().cpu() - rl).abs() <= lse_bound(0.0, rl)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D,Sq", [(64, 1), (128, 3)])
def test_nan_before_the_window(fa, cuda_device, D, Sq):
    """Keys and values of tokens no query sees any more are not looked at."""
    c = ([300, 41, 64], Sq, 4, 2, D, 32, F16, 0.0, 20)
    q, cache, n, plain = _attend(fa, c, 23)
    want = fa.fa_fwd_kvcache(q.cuda(), cache, n, window_left=20)
    page = c[5]
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    for b, tokens in enumerate(c[0]):
        for t in range(tokens - Sq - 20):
            at = int(plain[4][b, t // page])
            k[at, :, t % page] = 0x7F
            v[at, :, :, t % page] = 0x7F
    got = fa.fa_fwd_kvcache(q.cuda(), cache, n, window_left=20)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(got[0]).all()


@pytest.mark.gpu
def test_given_stream(fa, cuda_device):
    """A call for another stream than the current one, its workspace and outputs
    allocated by the call, while the current stream works and allocates."""
    c = ([3000, 900, 17], 1, 8, 2, 128, 64, BF, 0.0, -1)
    q, cache, n, _ = _attend(fa, c, 24)
    q = q.cuda()
    want = fa.fa_fwd_kvcache(q, cache, n)
    full = [torch.randn((1, 300, 2, 64), device="cuda").to(BF) for _ in range(3)]
    ranges = fa.mask_ranges(1, 300)
    plain = fa.fa_fwd(*full, softcap=9.0, mask_ranges=ranges)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        for _ in range(20):
            busy = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]
            got = fa.fa_fwd_kvcache(q, cache, n, stream=handle)
            r = fa.mask_ranges(1, 300, stream=handle)
            o, lse = fa.fa_fwd(*full, softcap=9.0, mask_ranges=r, stream=handle)
            del busy
            side.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(o, plain[0]) and torch.equal(lse, plain[1])


@pytest.mark.gpu
def test_append_rows_past_the_tensor(fa, cuda_device):
    """Prefix sums that run past the tensors: that sequence is left alone."""
    k, v, ks, vs = make_cache(4, 1, 16, 64, 25)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32).cuda()
    dev = [t.cuda() for t in (k, v, ks, vs)]
    cache = fa.KvCache(*dev, table)
    n = torch.tensor([3, 4], dtype=torch.int32).cuda()
    x = torch.randn((5, 1, 64), device="cuda").to(BF)
    fa.kvcache_append(cache, n, x, x, cu_new=torch.tensor([0, 3, 6], dtype=torch.int32).cuda(), max_new=3)
    torch.cuda.synchronize()
    assert fa.device_status() != fa.FA_OK
    assert fa.device_status() == fa.FA_OK
    assert not torch.equal(dev[0].view(torch.uint8)[0].cpu(), k.view(torch.uint8)[0])
    assert torch.equal(dev[0].view(torch.uint8)[2:].cpu(), k.view(torch.uint8)[2:])
    assert torch.equal(dev[1].view(torch.uint8)[2:].cpu(), v.view(torch.uint8)[2:])


@pytest.mark.gpu
def test_two_calls_at_once(fa, cuda_device):
    """Two streams, a workspace each: what one stream alone gives."""
    c = ([3000, 900, 17], 1, 8, 2, 128, 64, BF, 0.0, -1)
    d = ([100, 2000], 1, 8, 1, 64, 32, F16, 30.0, -1)
    runs = [_attend(fa, c, 14), _attend(fa, d, 15)]
    q = [r[0].cuda() for r in runs]
    want = [fa.fa_fwd_kvcache(q[i], runs[i][1], runs[i][2], softcap=x[7]) for i, x in enumerate((c, d))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, x in enumerate((c, d)):
            with torch.cuda.stream(streams[i]):
                got[i].append(fa.fa_fwd_kvcache(q[i], runs[i][1], runs[i][2], softcap=x[7]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.gpu
def test_gpu_side_refusals(fa, cuda_device):
    c = ([40, 50], 1, 2, 1, 64, 16, BF, 0.0, -1)
    q, cache, n, _ = _attend(fa, c, 16)
    with pytest.raises(ValueError):
        fa.fa_fwd_kvcache(q, cache, n)                                  # q on the CPU
    q = q.cuda()
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[..., :32]), dict(n=n.long()), dict(n=n[:1]), dict(n=n.cpu())):
        with pytest.raises(ValueError):
            fa.fa_fwd_kvcache(bad.get("q", q), cache, bad.get("n", n))
    with pytest.raises(fa.FaError):
        fa.fa_fwd_kvcache(q, cache, n, softcap=-1.0)
    with pytest.raises(ValueError):
        fa.fa_fwd_kvcache(q, cache, n, out=(q, torch.empty(3, device="cuda")))
    # a strided q is read as it is meant
    wide = torch.cat([q, q], dim=3)[..., 64:]
    a, b = fa.fa_fwd_kvcache(wide, cache, n), fa.fa_fwd_kvcache(q, cache, n)
    assert torch.equal(a[0], b[0])
    x = torch.zeros((2, 1, 1, 64), dtype=BF, device="cuda")
    for k, v in ((x, x.half()), (x[:1], x[:1]), (x[..., :32], x[..., :32]), (x, x.cpu()), (x.float(), x.float())):
        with pytest.raises(ValueError):
            fa.kvcache_append(cache, n, k, v)
    with pytest.raises(ValueError):
        fa.kvcache_append(cache, n, x[:, 0], x[:, 0], cu_new=torch.tensor([0, 1, 2], dtype=torch.int32).cuda())
    with pytest.raises(ValueError):
        fa.KvCache(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.block_table.long())
    with pytest.raises(ValueError):
        fa.KvCache(cache.k, cache.k, cache.k_scale, cache.v_scale, cache.block_table)


@pytest.mark.gpu
def test_far_pages(fa, cuda_device):
    """Page offsets past 2^32 bytes."""
    H, page, D = 2, 64, 128
    pages = (1 << 32) // (H * page * D) + 40
    k = torch.zeros((pages, H, page, D), dtype=torch.uint8, device="cuda").view(F8)
    v = torch.zeros((pages, H, D, page), dtype=torch.uint8, device="cuda").view(F8)
    ks, vs = (torch.ones((pages, H), device="cuda") for _ in range(2))
    lens = [100, 70]
    table = torch.tensor([[pages - 1, 3], [pages - 20, pages - 7]], dtype=torch.int32)
    cache = fa.KvCache(k, v, ks, vs, table.cuda())
    g = torch.Generator().manual_seed(9)
    news = [tuple(torch.randn((n, H, D), generator=g).to(BF) for _ in range(2)) for n in lens]
    zero = torch.zeros(2, dtype=torch.int32).cuda()
    cu = torch.tensor([0, 100, 170], dtype=torch.int32).cuda()
    fa.kvcache_append(cache, zero, torch.cat([n[0] for n in news]).cuda(), torch.cat([n[1] for n in news]).cuda(),
                      cu_new=cu, max_new=100)
    q = torch.randn((2, 1, 4, D), generator=g).to(BF)
    o, _ = fa.fa_fwd_kvcache(q.cuda(), cache, torch.tensor(lens, dtype=torch.int32).cuda())
    small = [torch.stack([t[p].cpu() for p in table.flatten().tolist()]) for t in (k.view(torch.uint8), v.view(torch.uint8), ks, vs)]
    near = torch.arange(4, dtype=torch.int32).view(2, 2)
    ro, _, bound = plain_attention(q, small[0].view(F8), small[1].view(F8), small[2], small[3], near, lens, page,
                                   D ** -0.5, 0.0, -1)
    check(o, ro, bound, "o")


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_reported(fa, cuda_device):
    """Found on the device by the kernels' own checks; the other sequences are
    served."""
    c = ([40, 50, 60], 1, 2, 1, 64, 16, BF, 0.0, -1)
    q, cache, n, plain = _attend(fa, c, 10)
    want, _ = fa.fa_fwd_kvcache(q.cuda(), cache, n)
    table = cache.block_table.clone()
    for bad in (-1, 10 ** 6, 65):   # 65: beyond the table of 4 pages
        n2 = n.clone()
        n2[1] = bad
        o, lse = fa.fa_fwd_kvcache(q.cuda(), cache, n2)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG and fa.device_status() == fa.FA_OK
        assert torch.equal(o[[0, 2]], want[[0, 2]]) and (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    for bad in (-1, cache.k.shape[0], 2 ** 31 - 1):
        cache.block_table[1, 1] = bad
        o, _ = fa.fa_fwd_kvcache(q.cuda(), cache, n)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
        assert torch.equal(o[[0, 2]], want[[0, 2]]) and torch.isfinite(o).all()
        cache.block_table.copy_(table)
    x = torch.ones((3, 5, 1, 64), dtype=BF, device="cuda")
    before = [t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    # a length below 0, a bad page, tokens past the table
    for lens in ([-1, 55, 63], [62, 63, 64]):
        if lens[0] < 0:
            cache.block_table[1, 3] = 77
        fa.kvcache_append(cache, torch.tensor(lens, dtype=torch.int32).cuda(), x, x)
        assert fa.device_status() == fa.FA_ERR_INVALID_ARG
        cache.block_table.copy_(table)
        for t, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
            assert torch.equal(t.view(torch.uint8), w)


@pytest.mark.gpu
@pytest.mark.parametrize("D,cap,dt", [(128, 30.0, BF), (64, 0.0, F16)])
def test_serving_run(fa, cuda_device, D, cap, dt):
    """Prompts through fa_fwd and the cache, then tokens one at a time, the
    append and the attention of a step captured once and replayed: every step
    against the definition over the cache's own values, and near fa_fwd's row
    over the unrounded ones."""
    prompts, steps, page, Hq, Hkv = [37, 1, 64], 20, 16, 4, 2
    B = len(prompts)
    g = torch.Generator().manual_seed(11)
    r = lambda n, h: torch.randn((n, h, D), generator=g).to(dt)   # noqa: E731
    ks_, vs_, qs = ([r(n + steps, h) for n in prompts] for h in (Hkv, Hkv, Hq))
    table, pages = block_table([n + steps for n in prompts], page, seed=12)
    k, v, ks, vs = make_cache(pages, Hkv, page, D, 13)
    cache = fa.KvCache(*(t.cuda() for t in (k, v, ks, vs)), table.cuda())
    cu = torch.tensor([0, 37, 38, 102], dtype=torch.int32).cuda()
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    pk, pv = (torch.cat([x[:m] for x, m in zip(t, prompts)]).cuda() for t in (ks_, vs_))
    fa.kvcache_append(cache, n, pk, pv, cu_new=cu, max_new=64)
    n += torch.tensor(prompts, dtype=torch.int32).cuda()
    newk, newv = (torch.empty((B, 1, Hkv, D), dtype=dt, device="cuda") for _ in range(2))
    q = torch.empty((B, 1, Hq, D), dtype=dt, device="cuda")
    ws = torch.empty(fa.fa_fwd_kvcache_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q), torch.empty((B, Hq, 1), device="cuda")

    def step():
        fa.kvcache_append(cache, n, newk, newv)
        n.add_(1)
        fa.fa_fwd_kvcache(q, cache, n, softcap=cap, workspace=ws, out=out)
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
        ro, rl, bound = plain_attention(q.cpu(), cache.k.cpu(), cache.v.cpu(), cache.k_scale.cpu(),
                                        cache.v_scale.cpu(), table, lens, page, D ** -0.5, cap, -1)
        check(out[0], ro, bound, "step %d" % t)
    # the last step next to fa_fwd over 16-bit keys and values: e4m3 rounds each
    # by 2^-4 at most; with N(0, 1) data scores move by about 2^-4 / sqrt(3) and
    # the mean over a softmax by less, so a fifth of the rows' size holds amply
    for b in range(B):
        full = [x[b][None].cuda() for x in (qs, ks_, vs_)]
        o, _ = fa.fa_fwd(*full, causal=True, softcap=cap)
        want = o[0, -1].double()
        assert (out[0][b, 0].double() - want).norm() <= 0.2 * want.norm()


# ------------------------------------------------------- refusals (no GPU)
def _struct(fa, **over):
    a = dict(k=0x1000, v=0x2000, k_scale=0x3000, v_scale=0x4000, block_table=0x5000, num_pages=10, page_size=64,
             max_pages=4, Hkv=2, D=128)
    a.update(over)
    return fa._KvCacheStruct(**a)


CACHE_REFUSED = [
    (dict(k=0), 1), (dict(v_scale=0), 1), (dict(block_table=0), 1), (dict(k=0x1008), 1), (dict(v=0x2004), 1),
    (dict(k_scale=0x3001), 1), (dict(block_table=0x5002), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1),
    (dict(page_size=-64), 1), (dict(max_pages=0), 1), (dict(Hkv=0), 1), (dict(page_size=24), 2),
    (dict(page_size=256), 2), (dict(D=96), 2), (dict(D=256), 2), (dict(max_pages=1 << 30), 1),
]


def _append(fa, s, **over):
    a = dict(len=0x6000, k=0x7000, v=0x8000, cu=0, rows=15, B=3, max_new=5, dtype=0)
    a.update(over)
    vp = ctypes.c_void_p
    return fa.lib().fa_kvcache_append(ctypes.byref(s), vp(a["len"]), vp(a["k"]), vp(a["v"]), vp(a["cu"]), a["rows"],
                                      a["B"], a["max_new"], a["dtype"], None)


def _attn(fa, s, **over):
    a = dict(q=0x7000, len=0x6000, o=0x8000, lse=0, B=3, Sq=1, Hq=4, scale=0.1, cap=0.0, window=-1, dtype=0,
             ws=0x10000, nbytes=1 << 30)
    a.update(over)
    vp = ctypes.c_void_p
    return fa.lib().fa_fwd_kvcache(vp(a["q"]), ctypes.byref(s), vp(a["len"]), vp(a["o"]), vp(a["lse"]), a["B"],
                                   a["Sq"], a["Hq"], a["scale"], a["cap"], a["window"], a["dtype"], vp(a["ws"]),
                                   a["nbytes"], None)


@pytest.mark.parametrize("over,status", CACHE_REFUSED)
def test_bad_caches_refused(fa, over, status):
    assert _append(fa, _struct(fa, **over)) == status
    assert _attn(fa, _struct(fa, **over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(len=0), 1), (dict(k=0), 1), (dict(v=0x8004), 1), (dict(k=0x7008), 1), (dict(cu=0x9002), 1),
    (dict(len=0x6001), 1), (dict(B=0), 1), (dict(max_new=0), 1), (dict(dtype=5), 2),
    (dict(B=1 << 20, max_new=1 << 20), 1), (dict(rows=14), 1), (dict(rows=16), 1), (dict(rows=0, cu=0x9000), 1)])
def test_append_refused(fa, over, status):
    assert _append(fa, _struct(fa), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(q=0), 1), (dict(o=0), 1), (dict(len=0), 1), (dict(q=0x7008), 1), (dict(lse=0x9002), 1),
    (dict(B=-1), 1), (dict(Sq=0), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(cap=-3.0), 1), (dict(cap=1e-5), 1), (dict(cap=float("inf")), 1),
    (dict(cap=0.001, scale=3e38), 1), (dict(window=-2), 1), (dict(ws=0), 1), (dict(ws=0x10080), 1),
    (dict(nbytes=1000), 1), (dict(B=4097), 2), (dict(dtype=9), 2), (dict(Sq=1 << 24), 2)])
def test_attention_refused(fa, over, status):
    assert _attn(fa, _struct(fa), **over) == status


def test_python_refusals(fa):
    k = torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(F8)
    v = torch.zeros((4, 2, 64, 16), dtype=torch.uint8).view(F8)
    s = torch.ones((4, 2))
    t = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.KvCache(k, v, s, s, t)             # not on the GPU
    with pytest.raises(ValueError):
        fa.KvCache(k, k, s, s, t)             # V in K's layout
    with pytest.raises(ValueError):
        fa.KvCache(k.view(torch.uint8), v, s, s, t)
    assert fa.fa_fwd_kvcache_workspace_bytes(96) == 0 and fa.fa_fwd_kvcache_workspace_bytes(128) > 0
