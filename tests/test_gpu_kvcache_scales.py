"""Appending to pages that were filled elsewhere, with scales that are no powers of
two: every byte is x / scale rounded once, to nearest even."""
import math

import pytest
import torch

from test_gpu_kvcache import block_table, f64, make_cache, plain_append

F16, BF = torch.float16, torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("page,D", [(16, 64), (64, 128), (48, 64)])
@pytest.mark.parametrize("scale", [41.0 / 64, 61.0 / 512, 0.75, 1.7, 1.0 / 3.0, 0.001])
def test_append_behind_other_scales(fa, cuda_device, scale, page, D, dt):
    """Held tokens whose scale stays (new values fit it), new values on or next to the
    ties of e4m3: t scale for the halfway points t, rounded to 16 bits, and its two
    neighbours.  And held tokens whose scale grows to a power of two."""
    H, lens, news = 2, [5, page - 3, page + 1, 3], [page + 4, 7, 20, page]
    table, pages = block_table([a + n for a, n in zip(lens, news)], page, extra=1, seed=3)
    k, v, ks, vs = make_cache(pages, H, page, D, 17)
    scale = float(torch.tensor(scale, dtype=torch.float32))   # as the cache holds it
    ks[:], vs[:] = scale, scale
    g = torch.Generator().manual_seed(18)
    # halfway between neighbouring e4m3 values: (m + 1/2) 2^(e - 3) for m in 8 .. 15, e in -6 .. 6;
    # at most 124, so that no scale has to grow for them
    m, e = torch.randint(8, 16, (sum(news), H, D), generator=g), torch.randint(-6, 7, (sum(news), H, D), generator=g)
    tie = (m.double() + 0.5) * torch.exp2(e.double() - 3)
    sign = torch.randint(0, 2, tie.shape, generator=g) * 2.0 - 1.0
    x = (tie * sign * scale).to(dt)
    step = torch.randint(-1, 2, x.shape, generator=g).to(torch.int16)   # the 16-bit neighbours
    x = (x.view(torch.int16) + step).view(dt)
    values = [x, x.flip(0)]
    big = sum(news[:3])   # the last sequence: values past the held scale, which grows to a power of two
    for t in values:
        t[big:] = (t[big:].double() * 5.0).to(dt)
    per = [tuple(t[sum(news[:b]):sum(news[:b + 1])] for t in values) for b in range(4)]
    dev = [t.cuda() for t in (k, v, ks, vs)]
    cache = fa.KvCache(*dev, table.cuda())
    cu = torch.tensor([sum(news[:i]) for i in range(5)], dtype=torch.int32).cuda()
    fa.kvcache_append(cache, torch.tensor(lens, dtype=torch.int32).cuda(), *(t.cuda() for t in values), cu_new=cu,
                      max_new=max(news))
    torch.cuda.synchronize()
    assert fa.device_status() == fa.FA_OK
    want = [f64(k), f64(v).transpose(2, 3).contiguous(), ks.double(), vs.double()]
    plain_append(*want, table, lens, per, page)
    kept = want[2][table[0, 0]]
    assert (kept == scale).all()                                                 # the first: as it was
    assert math.log2(float(want[2][table[3, 0], 0])).is_integer() and float(want[2][table[3, 0], 0]) > scale
    for got, w, name in zip(dev, (want[0], want[1].transpose(2, 3), want[2], want[3]), ("k", "v", "k_scale", "v_scale")):
        off = f64(got.cpu()) != w
        assert not off.any(), (name, int(off.sum()), f64(got.cpu())[off][:5], w[off][:5])
