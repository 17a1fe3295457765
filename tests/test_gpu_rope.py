"""Rotary positions: values and gradients against complex numbers in 64 bits, the
frequencies and the fixed-point steps on the CPU, refusals.

Bounds.  The angle's part of a turn is a whole number of 2^-64ths times the
position, cut to 2^-32 of a turn and brought to f32 (2^-24 of at most half a
turn), so an angle is off by less than pi 2^-24 + pi 2^-31; cosine and sine by that
and two steps of their own (2^-23 each), their products with the factor and the
sum of two products by 2^-23 more.  Together less than 2^-20 of |a| + |b| times
the factor, then one rounding to the output's type.
"""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from score_ref import SUB, U, check

F16, BF = torch.float16, torch.bfloat16
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def plain(x, w, factor, pos, interleaved, inverse=False):
    """(turned, bound) of x [.., S, H, D] at positions [.., S], in 64 bits."""
    R = 2 * len(w)
    turn = torch.polar(torch.full_like(w, factor), pos.double()[..., None, None] * w)
    turn = turn.conj() if inverse else turn
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y = x.double()
    z = torch.complex(y[..., a], y[..., b]) * turn
    out, size = y.clone(), torch.zeros_like(y)
    out[..., a], out[..., b] = z.real, z.imag
    size[..., a] = size[..., b] = abs(factor) * (y[..., a].abs() + y[..., b].abs())
    return out, U[x.dtype] * out.abs() * (size > 0) + 2.0 ** -20 * size + SUB[x.dtype] * (size > 0)


CASES = [
    # B, S, Hq, Hkv (0: no k), D, rotary dims, interleaved, dtype, positions, scaling
    (1, 1, 1, 1, 64, 64, False, BF, "rows", None),
    (2, 37, 4, 2, 128, 128, False, BF, "given", None),
    (2, 37, 4, 2, 128, 128, True, F16, "offsets", None),
    (3, 5, 3, 1, 96, 96, False, F16, "offsets", ("linear", 4.0)),
    (3, 5, 3, 0, 80, 20, True, BF, "given", ("ntk", 3.0)),
    (3, 5, 3, 1, 80, 20, False, BF, "given", None),          # halves of ten: a pair at a time
    (1, 333, 8, 8, 64, 2, True, F16, "rows", None),
    (1, 333, 8, 8, 64, 2, False, F16, "rows", None),
    (1, 100, 2, 1, 256, 256, False, BF, "far", ("yarn", 16.0, 4096)),
    (1, 100, 2, 1, 256, 254, True, F16, "far", ("yarn", 16.0, 4096, 16.0, 2.0)),
    (64, 1, 32, 8, 128, 128, False, BF, "offsets", None),
    (5, 700, 32, 8, 128, 64, False, BF, "rows", None),       # several rows a CTA
    (5, 700, 1, 0, 8, 8, True, BF, "rows", None),            # a row of one piece
    (5, 2000, 1, 1, 16, 16, False, F16, "given", None),
    (2, 3, 100, 7, 64, 34, False, F16, "far", None),
]


def _positions(kind, B, S, g):
    """(positions, offsets, the rows' positions) of a case."""
    at = torch.arange(S).expand(B, S)
    if kind == "rows":
        return None, None, at
    top = {"given": 5000, "offsets": 100000, "far": 2 ** 31 - 5000}[kind]
    if kind == "offsets":
        off = torch.randint(-10, top, (B,), generator=g).int()
        return None, off.cuda(), at + off[:, None]
    pos = torch.randint(-top if kind == "far" else -10, top, (B, S), generator=g).int()
    return pos.cuda(), None, pos


@pytest.mark.gpu
@pytest.mark.parametrize("c", CASES, ids=lambda c: "_".join(map(str, c)).replace("torch.", "").replace(" ", ""))
def test_turned(fa, cuda_device, c):
    B, S, Hq, Hkv, D, R, inter, dt, kind, scaling = c
    g = torch.Generator().manual_seed(S)
    q = torch.randn((B, S, Hq, D), generator=g).to(dt)
    k = torch.randn((B, S, Hkv, D), generator=g).to(dt) if Hkv else None
    positions, offsets, pos = _positions(kind, B, S, g)
    w, factor = fa.rope_frequencies(R, scaling=scaling)
    table = fa.rope_table(R, scaling=scaling)
    assert table.rotary_dim == R and table.factor == factor
    on = [None if t is None else t.cuda() for t in (q, k)]
    kw = dict(positions=positions, offsets=offsets, interleaved=inter)
    for call, inverse in ((fa.rope, False), (fa.rope_bwd, True)):
        got = call(*on, table, **kw)
        for name, x, y in (("q", q, got[0]), ("k", k, got[1])):
            if x is None:
                assert y is None
                continue
            want, bound = plain(x, w, factor, pos, inter, inverse)
            check(y, want, bound, name)
            assert torch.equal(y[..., R:].cpu(), x[..., R:])
        # in place: the same
        into = [None if t is None else t.clone() for t in on]
        back = call(*into, table, out=tuple(into), **kw)
        for a, b in zip(got, back):
            assert (a is None and b is None) or torch.equal(a, b)
        assert back[0] is into[0]
    assert fa.device_status() == fa.FA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(30))
def test_any_sizes(fa, cuda_device, seed):
    """Sizes, layouts and positions drawn at random."""
    r = torch.Generator().manual_seed(300 + seed)
    pick = lambda *x: x[int(torch.randint(0, len(x), (), generator=r))]   # noqa: E731
    D = 8 * int(torch.randint(1, 33, (), generator=r))
    R = pick(D, 2 * int(torch.randint(1, D // 2 + 1, (), generator=r)))
    B, S, Hq, Hkv, dt = pick(1, 2, 7), pick(1, 3, 50, 900), pick(1, 2, 6, 20), pick(0, 1, 3), pick(BF, F16)
    inter, kind = pick(True, False), pick("rows", "given", "offsets", "far")
    q, k = (torch.randn((B, S, h, D), generator=r).to(dt) if h else None for h in (Hq, Hkv))
    positions, offsets, pos = _positions(kind, B, S, r)
    w, factor = fa.rope_frequencies(R, 500.0)
    got = fa.rope(q.cuda(), None if k is None else k.cuda(), fa.rope_table(R, 500.0), positions=positions, offsets=offsets,
                  interleaved=inter)
    for x, y in ((q, got[0]), (k, got[1])):
        if x is not None:
            want, bound = plain(x, w, factor, pos, inter)
            check(y, want, bound, "%r" % ((B, S, Hq, Hkv, D, R, inter, kind),))
            assert torch.equal(y[..., R:].cpu(), x[..., R:])


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(fa, cuda_device, inter):
    """<g, rope(x + h) - rope(x - h)> against <rope_bwd(g), 2 h>: rope is linear, so the
    differences are those of its roundings (u of what is rounded, each side)."""
    g_ = torch.Generator().manual_seed(1)
    B, S, H, D, R, dt = 2, 9, 2, 64, 48, F16
    x, h, g = (torch.randn((B, S, H, D), generator=g_).to(dt) for _ in range(3))
    h = (h * 0.5).to(dt)
    table = fa.RopeTable.of([0.3 ** i for i in range(R // 2)], 1.25)
    off = torch.tensor([3, 1000], dtype=torch.int32).cuda()
    f = lambda t: fa.rope(t.to(dt).cuda(), None, table, offsets=off, interleaved=inter)[0].double().cpu()   # noqa: E731
    up, down = (x.double() + h.double()).to(dt), (x.double() - h.double()).to(dt)
    yu, yd = f(up), f(down)
    left = (g.double() * (yu - yd)).sum()
    dx = fa.rope_bwd(g.cuda(), None, table, offsets=off, interleaved=inter)[0].double().cpu()
    step = up.double() - down.double()
    right = (dx * step).sum()
    slack = U[dt] * ((g.double().abs() * (yu.abs() + yd.abs())).sum() + (dx.abs() * step.abs()).sum()) * 1.01
    assert (left - right).abs() <= slack


@pytest.mark.gpu
def test_there_and_back_leaves_scores(fa, cuda_device):
    """What the operator is for: scores of turned q and k depend on the distance alone."""
    g = torch.Generator().manual_seed(2)
    q, k = (torch.randn((1, 1, 1, 128), generator=g).half().cuda() for _ in range(2))
    table = fa.rope_table(128)
    at = lambda x, p: fa.rope(x, None, table, offsets=torch.tensor([p], dtype=torch.int32).cuda())[0].double()   # noqa: E731
    want = (at(q, 7) * at(k, 2)).sum()
    size = (q.double().norm() * k.double().norm()).item()
    for far in (1000, 10 ** 6, 2 ** 31 - 10):
        # each turned value is off by u of itself (and far less for its angle)
        assert abs((at(q, far + 7) * at(k, far + 2)).sum() - want) <= 4 * (U[F16] + 2.0 ** -19) * size


@pytest.mark.gpu
def test_strides_and_packed_rows(fa, cuda_device):
    """Slices of a joint projection, turned where they lie; packed rows; odd strides."""
    g = torch.Generator().manual_seed(3)
    B, S, D = 2, 50, 64
    qkv = torch.randn((B, S, 4 + 2 + 2, D), generator=g).to(BF).cuda()
    table = fa.rope_table(32)
    pos = torch.randint(0, 999, (B, S), generator=g).int().cuda()
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:].clone()
    want = fa.rope(q.contiguous(), k.contiguous(), table, positions=pos)
    got = fa.rope(q, k, table, positions=pos)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].is_contiguous()
    packed = fa.rope(q.reshape(B * S, 4, D), k.reshape(B * S, 2, D), table, positions=pos.view(-1))
    assert torch.equal(packed[0].view_as(q), want[0]) and torch.equal(packed[1].view_as(k), want[1])
    part = fa.rope(qkv.view(B * S, 8, D)[:, :4], None, table, positions=pos.view(-1))[0]
    assert torch.equal(part.view_as(q), want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    by_heads = q.transpose(1, 2).contiguous().transpose(1, 2)   # [B, H, S, D] in memory
    for x in (q, by_heads):
        a = fa.rope(x, k, table, positions=pos, stream=side)
        side.synchronize()
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    odd = torch.zeros((B, S, 4, D + 1), dtype=BF, device="cuda")[..., 1:]
    odd.copy_(q)
    assert torch.equal(fa.rope(odd, None, table, positions=pos)[0], want[0])   # copied, then turned
    with pytest.raises(ValueError):
        fa.rope(odd, None, table, positions=pos, out=(odd, None))
    with pytest.raises(ValueError):
        fa.rope(odd, None, table, positions=pos, stream=side)
    fa.rope(q, k, table, positions=pos, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 6:], v)
    wide = torch.zeros((B, S, 10, D), dtype=BF, device="cuda")
    fa.rope_bwd(q, k, table, positions=pos, out=(wide[:, :, :4], wide[:, :, 5:7]))
    back = fa.rope_bwd(want[0], want[1], table, positions=pos)
    assert torch.equal(wide[:, :, :4], back[0]) and torch.equal(wide[:, :, 5:7], back[1]) and (wide[:, :, [4, 7, 8, 9]] == 0).all()


@pytest.mark.gpu
def test_captured(fa, cuda_device):
    """Captured and replayed, on new values in the captured buffers."""
    table = fa.rope_table(64)
    q = torch.zeros((2, 3, 2, 64), dtype=F16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    fa.rope(q, None, table, offsets=off, out=(out, None))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.rope(q, None, table, offsets=off, out=(out, None))
    for at in (0, 5, 70000):
        q.normal_()
        off.fill_(at)
        graph.replay()
        assert torch.equal(out, fa.rope(q, None, table, offsets=off)[0])


@pytest.mark.gpu
def test_training_step(fa, cuda_device):
    """rope, fa_fwd, fa_bwd and rope_bwd as a layer uses them, over packed documents,
    against one 64-bit form with automatic gradients."""
    g = torch.Generator().manual_seed(6)
    B, S, Hq, Hkv, D, dt = 2, 100, 4, 2, 64, BF
    q, k, v, do = (torch.randn((B, S, h, D), generator=g).to(dt) for h in (Hq, Hkv, Hkv, Hq))
    ids = (torch.arange(S) // 37).expand(B, S).int()
    pos = (torch.arange(S) % 37).expand(B, S).int()
    table = fa.rope_table(D, scaling=("linear", 2.0))
    w, _ = fa.rope_frequencies(D, scaling=("linear", 2.0))
    ranges = fa.mask_ranges(B, S, doc_ids=ids.contiguous().cuda())
    p = pos.contiguous().cuda()
    tq, tk = fa.rope(q.cuda(), k.cuda(), table, positions=p)
    o, lse = fa.fa_fwd(tq, tk, v.cuda(), mask_ranges=ranges)
    dq, dk, dv = fa.fa_bwd(tq, tk, v.cuda(), o, do.cuda(), lse, mask_ranges=ranges)
    dq, dk = fa.rope_bwd(dq, dk, table, positions=p)
    leaves = [t.double().requires_grad_() for t in (q, k, v)]

    def turn(x):
        a, b = x.chunk(2, dim=-1)
        c, s = (f(pos.double()[..., None, None] * w) for f in (torch.cos, torch.sin))
        return torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    x, y, z = (t.transpose(1, 2) for t in (turn(leaves[0]), turn(leaves[1]).repeat_interleave(2, dim=2),
                                           leaves[2].repeat_interleave(2, dim=2)))
    i = torch.arange(S)
    ok = (i[:, None] >= i[None]) & (ids[0][:, None] == ids[0][None])
    want = (torch.softmax((x @ y.transpose(2, 3) * D ** -0.5).masked_fill(~ok, -math.inf), dim=-1) @ z).transpose(1, 2)
    want.backward(do.double())
    # roundings to bf16 on the way: q, k turned (u of each score's magnitudes), P, dS, O and the results; as
    # relative 2-norms they add to a few u, and the library's own bar is 5e-3 for the attention alone
    for got, ref in ((o, want), (dq, leaves[0].grad), (dk, leaves[1].grad), (dv, leaves[2].grad)):
        ref = ref.detach()
        assert (got.double().cpu() - ref).norm() <= 4 * U[dt] * ref.norm()


# ------------------------------------------------------------------- no GPU
def test_frequencies(fa):
    w, f = fa.rope_frequencies(8, 10000.0)
    assert f == 1.0 and torch.allclose(w, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    lin, f = fa.rope_frequencies(8, 10000.0, ("linear", 4.0))
    assert f == 1.0 and torch.equal(lin, w / 4)
    ntk, f = fa.rope_frequencies(8, 10000.0, ("ntk", 16.0))
    # the fastest pair stays, the slowest is slowed by the whole scale
    assert f == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[3], w[3] / 16, rel_tol=1e-14)
    yarn, f = fa.rope_frequencies(8, 10000.0, ("yarn", 4.0, 2000.0))
    assert math.isclose(f, 0.1 * math.log(4.0) + 1.0)
    r = 2000.0 * w / (2 * math.pi)   # 318, 31.8, 3.18, 0.318 turns in the trained length
    g = ((r - 1.0) / 31.0).clamp(0.0, 1.0)
    assert torch.allclose(yarn, w / 4 * (1 - g) + w * g, rtol=1e-14) and yarn[0] == w[0] and yarn[3] == w[3] / 4
    for bad in ((7, 1e4, None), (0, 1e4, None), (258, 1e4, None), (8, 1.0, None), (8, math.nan, None), (8, 1e4, ("linear", 0.5)),
                (2, 1e4, ("ntk", 2.0)), (8, 1e4, ("yarn", 2.0, 0.0)), (8, 1e4, ("yarn", 2.0, 100.0, 1.0, 1.0))):
        with pytest.raises(fa.FaError):
            fa.rope_frequencies(*bad)
    for bad in (("slow", 2.0), ("linear",), ("yarn", 2.0), ("yarn", 2.0, 1.0, 2.0)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(8, 1e4, bad)


def test_steps(fa):
    """Parts of a turn per position in 2^-64ths: nearest to w / (2 pi), whole turns dropped."""
    w = [1.0, 10000.0 ** -0.3, 1e-5, 1e-18, 1e-25, 0.0, 5e-324, 2 * math.pi, 1000.0, math.pi, math.nextafter(1.0, 0.0)]
    got = fa.RopeTable.of(w, device="cpu").steps.tolist()
    for x, n in zip(w, got):
        exact = Fraction(x) / (2 * PI) * 2 ** 64
        # rounded once, from 2^128 / (2 pi) rounded itself and cut to 64 bits below: half a step and a hair
        assert abs((n % 2 ** 64) - exact % 2 ** 64) <= Fraction(1, 2) + Fraction(1, 2 ** 20) or exact % 2 ** 64 > 2 ** 64 - 1
    for bad in ([-1.0], [1024.0], [math.inf], [math.nan], [1.0, -0.5]):
        with pytest.raises(fa.FaError):
            fa.RopeTable.of(bad, device="cpu")
    for bad in ([], [[1.0]]):
        with pytest.raises(ValueError):
            fa.RopeTable.of(bad, device="cpu")
    assert fa.lib().fa_rope_steps(None, 3, None) == 1


def _call(fa, q=None, k=None, **over):
    a = dict(B=2, S=3, D=64, R=64, steps=0x1000, factor=1.0, inter=0, inv=0, pos=0, off=0, dtype=0)
    a.update(over)
    base = dict(in_=0x2000, out=0x3000, heads=2, in_stride=(0, 0, 0), out_stride=(0, 0, 0))

    def tensor(x):
        t = dict(base, **x)
        r = fa._RopeTensor(t["in_"], t["out"], t["heads"])
        r.in_stride[:], r.out_stride[:] = t["in_stride"], t["out_stride"]
        return ctypes.byref(r)
    vp = ctypes.c_void_p
    return fa.lib().fa_rope(None if q == "none" else tensor(q or {}), None if k is None else tensor(k), a["B"], a["S"],
                            a["D"], a["R"], vp(a["steps"]), a["factor"], a["inter"], a["inv"], vp(a["pos"]), vp(a["off"]),
                            a["dtype"], None)


@pytest.mark.parametrize("q,over,status", [
    ("none", {}, 1), (dict(in_=0), {}, 1), (dict(out=0), {}, 1), (dict(in_=0x2008), {}, 1), (dict(out=0x3002), {}, 1),
    (dict(heads=0), {}, 1), (dict(heads=-1), {}, 1), (dict(heads=32768), {}, 2), (dict(in_stride=(192, 64, 4)), {}, 1),
    (dict(in_stride=(192, 0, 64)), {}, 1), (dict(out_stride=(-384, 128, 64)), {}, 1), (dict(out_stride=(1 << 39, 128, 64)), {}, 1),
    (dict(out=0x2000, in_stride=(1536, 512, 64)), {}, 1),      # in place with other strides
    ({}, dict(B=0), 1), ({}, dict(S=0), 1), ({}, dict(D=0), 1), ({}, dict(R=0), 1), ({}, dict(R=63), 1), ({}, dict(R=66), 1),
    ({}, dict(steps=0), 1), ({}, dict(steps=0x1004), 1), ({}, dict(factor=math.nan), 1), ({}, dict(pos=0x4002), 1),
    ({}, dict(off=0x4001), 1), ({}, dict(pos=0x4000, off=0x5000), 1), ({}, dict(D=68, R=64), 2), ({}, dict(D=264), 2),
    ({}, dict(dtype=2), 2), ({}, dict(B=1 << 16, S=1 << 15), 2)])
def test_refused(fa, q, over, status):
    assert _call(fa, q, **over) == status
    if isinstance(q, dict) and q:
        assert _call(fa, {}, q, **over) == status   # of k


def test_python_refusals(fa):
    q = torch.zeros((2, 3, 2, 64), dtype=BF)
    with pytest.raises(ValueError, match="q: not on a GPU"):
        fa.rope(q, None, fa.rope_table(64, device="cpu"))


@pytest.mark.gpu
def test_gpu_side_refusals(fa, cuda_device):
    q = torch.zeros((2, 3, 2, 64), dtype=BF, device="cuda")
    t = fa.rope_table(64)
    pos, off = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for args, kw in (((q.float(), None), {}), ((q[0, 0], None), {}), ((q, q[:1]), {}), ((q, q[..., :32]), {}), ((q, q.half()), {}),
                     ((q, q.cpu()), {}), ((q, None), dict(positions=pos[:1])), ((q, None), dict(positions=pos.long())),
                     ((q, None), dict(positions=pos.cpu())), ((q, None), dict(offsets=off[:1])), ((q, None), dict(out=(q, q))),
                     ((q, q), dict(out=(q, None))), ((q, None), dict(out=(q[:, :, :1], None))), ((q[:0], None), {}),
                     ((q[:, :, :0], None), {}), ((q.view(6, 2, 64), None), dict(positions=pos))):
        with pytest.raises(ValueError):
            fa.rope(*args, t, **kw)
    for bad in (fa.RopeTable(t.steps.int()), fa.RopeTable(t.steps.cpu()), fa.RopeTable(t.steps[::2])):
        with pytest.raises(ValueError):
            fa.rope(q, None, bad)
    for bad in (fa.rope_table(66), fa.RopeTable(t.steps, math.inf)):
        with pytest.raises(fa.FaError):
            fa.rope(q, None, bad)
    with pytest.raises(fa.FaError):
        fa.rope(q, None, t, positions=pos, offsets=off)
