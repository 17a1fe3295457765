"""Backward calls without a workspace of their own: in flight together on two
streams, captured into graphs, and what they report."""
import pytest
import torch

from test_gpu_score import _build, _inputs, _mask
from score_ref import attend, backward, band

F16, BF = torch.float16, torch.bfloat16

# B, S, Hq, Hkv, D, dtype, mask keywords (None: causal), cap, more keywords (a window: not the compiled way in)
CALLS = [
    (3, 300, 20, 4, 128, BF, dict(doc="pad"), 30.0, {}),
    (2, 333, 40, 8, 64, F16, None, 20.0, {}),
    (1, 257, 6, 2, 128, BF, None, 0.0, dict(window=(100, 0))),
    (6, 420, 16, 8, 96, F16, dict(doc="mixed", prefix="doc"), 0.0, {}),
]


def _call(fa, i):
    """(call, [(gradient, bound), ..] per sequence in 64 bits on the GPU)"""
    B, S, Hq, Hkv, D, dt, mask, cap, more = CALLS[i]
    x = _inputs(B, S, S, Hq, Hkv, D, dt, 90 + i, a=1.5 if cap else 1.0)
    kw = dict(more, softcap=cap)
    if mask is None:
        kw["causal"], oks = True, [band(S, S, True, more.get("window"))] * B
    else:
        m, oks = _mask(dict(B=B, S=S, **mask))
        kw["mask_ranges"] = _build(fa, B, S, m)
    q, k, v, g = (t.cuda() for t in x)
    o, lse = fa.fa_fwd(q, k, v, **kw)
    og, refs = o.cpu(), []
    for b in range(B):
        _, _, p, t, _ = attend(x[0][b], x[1][b], x[2][b], oks[b], D ** -0.5, cap)
        refs.append(backward(x[0][b], x[1][b], x[2][b], og[b], x[3][b], oks[b], p, t, D ** -0.5, cap,
                             rounded_p=not cap and D == 64))
    want = [[torch.stack([r[n][e] for r in refs]).cuda() for e in (0, 1)] for n in range(3)]
    return (lambda: fa.fa_bwd(q, k, v, o, g, lse, **kw)), want


def _right(grads, want):
    return all(bool(((got.double() - r).abs() <= off).all()) for got, (r, off) in zip(grads, want))


@pytest.mark.gpu
@pytest.mark.parametrize("first,second", [(0, 1), (2, 3), (0, 0)])
def test_backwards_in_flight_together(fa, cuda_device, first, second):
    """Queued on two streams behind a wait, so that they run together: every one of
    them inside its bounds, dK and dV as alone (they are summed in a fixed order)."""
    runs = [_call(fa, first), _call(fa, second)]
    alone = [call() for call, _ in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[], []]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)   # about 10 ms
    for _ in range(12):
        for (call, _), s, out in zip(runs, streams, got):
            with torch.cuda.stream(s):
                out.append(call())
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    for (_, want), out, one in zip(runs, got, alone):
        assert _right(one, want)
        for grads in out:
            assert _right(grads, want)
            assert torch.equal(grads[1], one[1]) and torch.equal(grads[2], one[2])


@pytest.mark.gpu
def test_captured_backward_has_its_own_scratch(fa, cuda_device):
    """Two graphs of backwards without a workspace, replayed on two streams while
    eager calls run on a third."""
    runs = [_call(fa, 0), _call(fa, 3), _call(fa, 1)]
    alone = [call() for call, _ in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call, _ in runs[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        for grads in outs:
            for t in grads:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        eager = []
        for _ in range(4):
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
            with torch.cuda.stream(streams[2]):
                eager.append(runs[2][0]())
        torch.cuda.synchronize()
        for grads, (_, want), one in zip(outs + eager, runs[:2] + [runs[2]] * 4, alone[:2] + [alone[2]] * 4):
            assert _right(grads, want)
            assert torch.equal(grads[1], one[1]) and torch.equal(grads[2], one[2])
    assert fa.device_status() == fa.FA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("det", [False, True])
def test_errors_stay_readable(fa, cuda_device, det):
    """Sequence lengths the device refuses are reported by fa_device_status although
    the call's scratch is gone, also behind a later call that is in order."""
    call, want = _call(fa, 1)
    call()
    T, H, D = 400, 2, 64
    q, k, v, g = (torch.randn((T, H, D), device="cuda").to(BF) for _ in range(4))
    cu = torch.tensor([0, 100, 400], dtype=torch.int32).cuda()
    kw = dict(cu_seqlens_q=cu, cu_seqlens_k=cu, causal=True, totals=(T, T))
    o, lse = fa.fa_fwd(q, k, v, max_seqlen_q=300, max_seqlen_k=300, **kw)
    bad = dict(max_seqlen_q=200, max_seqlen_k=200, deterministic=det, **kw)   # the second sequence has 300
    assert fa.device_status() == fa.FA_OK
    if det:
        with pytest.raises(fa.FaError) as e:
            fa.fa_bwd(q, k, v, o, g, lse, **bad)
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    else:
        fa.fa_bwd(q, k, v, o, g, lse, **bad)
    assert _right(call(), want)
    assert fa.device_status() == fa.FA_ERR_INVALID_ARG
    assert fa.device_status() == fa.FA_OK
