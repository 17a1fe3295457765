"""Plain 64-bit forms of the capped / interval-masked attention, and the bounds
its 16-bit outputs are held to (tests/test_gpu_score.py, tests/test_gpu_kvcache.py).

Bounds.  u is half a rounding step of the 16-bit type relative to the value
(2^-8 bf16, 2^-11 fp16).  P and dS are rounded to that type once before their
products and every output once after them, so with A the product of absolute
values an output is off by at most u |out| + u A, and eps A for everything held
in 32 bits: the score's absolute error (softcap 2^-21 for the cap, and the
32-bit accumulation of q.k, below 2^-21 of sum |q||k| c < 64 here) acts on P as
a relative one, twice (numerator and row sum), eps = softcap 2^-20 + 2^-14.
fp16 has no relative precision below 2^-14: P and dS are then off by up to
2^-25 in absolute terms, `sub` below.  The dS of the 64-wide instance without a
cap is formed from the rounded P: one more u.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SUB = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def visible(B, S, doc=None, prefix=None, causal=True, window=None):
    """[B, S, S] truth values from the definition: same run of equal ids, not
    padding, and inside the order / window or the document's prefix."""
    out = torch.zeros((B, S, S), dtype=torch.bool)
    wl, wr = window or (-1, -1)
    for b in range(B):
        ids = [0] * S if doc is None else doc[b].tolist()
        s = 0
        while s < S:
            e = s
            while e < S and ids[e] == ids[s]:
                e += 1
            if ids[s] >= 0:
                n = 0
                if prefix is not None:
                    n = int(prefix[b]) if prefix.dim() == 1 else int(prefix[b, s])
                i, j = torch.arange(s, e)[:, None], torch.arange(s, e)[None, :]
                ok = (j <= i) if causal else torch.ones((e - s, e - s), dtype=torch.bool)
                if wl >= 0:
                    ok = ok & (j >= i - wl)
                if wr >= 0:
                    ok = ok & (j <= i + wr)
                out[b, s:e, s:e] = ok | (j < s + max(n, 0)) if prefix is not None else ok
            s = e
    return out


def band(Lq, Lk, causal, window=None):
    """[Lq, Lk]: the bottom-right aligned causal mask and window."""
    i, j = torch.arange(Lq)[:, None] + (Lk - Lq), torch.arange(Lk)[None, :]
    ok = (j <= i) if causal else torch.ones((Lq, Lk), dtype=torch.bool)
    wl, wr = window or (-1, -1)
    if wl >= 0:
        ok = ok & (j >= i - wl)
    if wr >= 0:
        ok = ok & (j <= i + wr)
    return ok


def heads(x, H):
    """[S, h, D] -> [H, S, D] double, every kv head repeated over its group."""
    return x.double().transpose(0, 1).repeat_interleave(H // x.shape[1], dim=0)


def attend(q, k, v, ok, scale, cap):
    """One sequence: q [Lq, Hq, D], k / v [Lk, Hkv, D], ok [Lq, Lk].  Returns
    (o [Lq, Hq, D], lse [Hq, Lq], p, t, bound of |o's error| without u |o|)."""
    Hq, dt = q.shape[1], q.dtype
    s = heads(q, Hq) @ heads(k, Hq).transpose(1, 2) * scale
    t = torch.tanh(s / cap) if cap else torch.zeros_like(s)
    s = cap * t if cap else s
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, dim=2)
    p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    vv = heads(v, Hq)
    o = p @ vv
    off = (U[dt] + eps(cap)) * (p @ vv.abs()) + SUB[dt] * (ok.double() @ vv.abs())
    return o.transpose(0, 1), lse, p, t, (U[dt] * o.abs() + off).transpose(0, 1)


def eps(cap):
    return cap * 2.0 ** -20 + 2.0 ** -14


def lse_bound(cap, lse):
    """The log-sum-exp: the score's error, and 32-bit sums and logarithm."""
    fin = torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))
    return cap * 2.0 ** -20 + 2.0 ** -15 + fin.abs() * 2.0 ** -20


def backward(q, k, v, o, dout, ok, p, t, scale, cap, rounded_p):
    """Gradients of one sequence and their bounds: [(dq, off), (dk, off), (dv, off)]."""
    Hq, Hkv, dt = q.shape[1], k.shape[1], q.dtype
    u, e, sub = U[dt], eps(cap), SUB[dt]
    qq, kk, vv, g, oo = heads(q, Hq), heads(k, Hq), heads(v, Hq), heads(dout, Hq), heads(o, Hq)
    dp = g @ vv.transpose(1, 2)
    row = (g * oo).sum(dim=2, keepdim=True)
    f = 1.0 - t * t if cap else torch.ones_like(t)
    ds = p * (dp - row) * f
    # what 32-bit sums of dP and of the row term may be off by, next to dS
    loose = p * f * (g.abs() @ vv.abs().transpose(1, 2) + (g * oo).abs().sum(dim=2, keepdim=True))
    err = (u * (2 if rounded_p else 1) + e) * ds.abs() + (2.0 ** -16 + e * 2.0 ** -3) * loose
    err = err + sub * ok.double() * (1 + (dp - row).abs() * (1 if rounded_p else 0))
    # 1 - tanh^2 = 4 r (1 - r) in 32 bits: absolute error of a few 2^-24
    err = err + (2.0 ** -20 * p * (dp - row).abs() if cap else 0.0)

    def group(x):   # [Hq, S, D] -> [S, Hkv, D]
        return x.view(Hkv, Hq // Hkv, *x.shape[1:]).sum(dim=1).transpose(0, 1)

    dq, dq_off = scale * (ds @ kk), scale * (err @ kk.abs())
    dk, dk_off = scale * group(ds.transpose(1, 2) @ qq), scale * group(err.transpose(1, 2) @ qq.abs())
    dv = group(p.transpose(1, 2) @ g)
    dv_off = group(((u + e) * p + sub * ok.double()).transpose(1, 2) @ g.abs())
    dq, dq_off = dq.transpose(0, 1), dq_off.transpose(0, 1)
    return [(x, y + u * x.abs() + sub) for x, y in ((dq, dq_off), (dk, dk_off), (dv, dv_off))]


def check(got, want, bound, what):
    """|got - want| <= bound everywhere; the message says where and by how much."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what + ": not finite"
    over = (got - want).abs() - bound
    if (over > 0).any():
        at = int(over.argmax())
        raise AssertionError("%s: %d of %d off; worst %r: got %.6g, want %.6g, bound %.3g" % (
            what, int((over > 0).sum()), over.numel(), tuple(torch.unravel_index(torch.tensor(at), over.shape)),
            got.flatten()[at], want.flatten()[at], bound.flatten()[at]))
