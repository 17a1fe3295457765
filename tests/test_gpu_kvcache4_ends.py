"""Ends of the 4-bit cache's range: scales of zero under the sharpest scores, NaN and infinities that
some rows do not see, queries and softmax scales of any size, values next to the type's largest, calls
from several threads.  Plain forms and bounds are test_gpu_kvcache4's."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

from score_ref import check
from test_gpu_kvcache4 import (BF, F16, _attend, _keys_like, block_table, check_lse, ints, make_cache, plain_attention,
                               quantise, sums, unpack)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _two_keys(D, lens, high, dt, gap):
    """One query of two heads over caches of one sequence; its keys are multiples of the query, so that token
    `high` scores `gap` nats (before a cap) above every other one.  V scales: 0 for that token."""
    table, pages = block_table(lens, 16)
    host = make_cache(pages, 1, 16, D, 3)
    g = torch.Generator().manual_seed(4)
    q = torch.randn((1, 1, 2, D), generator=g)
    q[0, 0, 1] = q[0, 0, 0]
    x = q[0, 0, 0] * (gap / 2 / float((q[0, 0, 0] ** 2).sum()) / D ** -0.5)
    for t in range(lens[0]):
        at, slot = int(table[0, t // 16]), t % 16
        code, s = _keys_like(x if t == high else -x)
        host[0][at, 0, slot], host[2][at, 0, slot] = code, s
        if t == high:
            host[3][at, 0, slot, :, 0] = 0.0
    return q.to(dt), host, table


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.0, 60.0])
@pytest.mark.parametrize("lens,high", [([2], 0), ([2], 1), ([100], 3), ([100], 99), ([3000], 70), ([3000], 2999)])
@pytest.mark.parametrize("D", [64, 128])
def test_no_scale_under_the_top_score(fa, cuda_device, D, lens, high, cap):
    """The key with nearly all the weight has V scales of 0, and those with scales lie 100 to 400 nats below:
    the answer is the top key's middles."""
    for gap in (100.0, 140.0, 400.0):
        q, host, table = _two_keys(D, lens, high, BF, 1000.0 if cap else gap)   # (capped: up to 120 apart)
        cache = fa.KvCache4(*(t.cuda() for t in host), table.cuda())
        o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, ints(lens), softcap=cap)
        ro, rl, off, lse_off = plain_attention(q, *host, table, lens, 16, D ** -0.5, cap, -1)
        check(o, ro, off, "o")
        check_lse(lse, rl, lse_off)


class _Call(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("cache", ctypes.c_void_p), ("len", ctypes.c_void_p), ("o", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)]


@pytest.mark.gpu
def test_two_threads(fa, cuda_device, tmp_path):
    """Calls of one and of 4000 sequences from two threads at a time, each on its stream with its workspace:
    none is refused for what the other one needs."""
    cxx, cuda = shutil.which("g++") or shutil.which("c++"), os.environ.get("CUDA_HOME", "/usr/local/cuda")
    if cxx is None:
        pytest.skip("no C++ compiler")
    so = str(tmp_path / "two_callers.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(cuda, "include"), os.path.join(ROOT, "tests", "two_callers.cpp"), "-o", so,
                    "-L", os.path.join(cuda, "lib64"), "-lcudart"], check=True)
    held, calls = [], (_Call * 2)()
    for i, B in enumerate((1, 4000)):
        lens = [20] + [0] * (B - 1)
        table, pages = block_table(lens, 16)
        cache = fa.KvCache4(*(t.cuda() for t in make_cache(pages, 1, 16, 64, 1)), table.cuda())
        q = torch.ones((B, 1, 1, 64), dtype=BF, device="cuda")
        n, stream = ints(lens), torch.cuda.Stream()
        ws = torch.empty(fa.fa_fwd_kvcache4_workspace_bytes(64), dtype=torch.uint8, device="cuda")
        o, lse = torch.empty_like(q), torch.empty((B, 1, 1), device="cuda")
        held.append((cache, q, n, stream, ws, o, lse))
        calls[i] = _Call(q.data_ptr(), ctypes.addressof(cache._c), n.data_ptr(), o.data_ptr(), lse.data_ptr(), B, 1,
                         ws.data_ptr(), ws.numel(), stream.cuda_stream)
    torch.cuda.synchronize()
    entry = ctypes.cast(fa.lib().fa_fwd_kvcache4, ctypes.c_void_p)
    failed = ctypes.CDLL(so).two_callers(entry, calls, torch.cuda.current_device(), 5000)
    torch.cuda.synchronize()
    assert failed == 0 and fa.device_status() == fa.FA_OK
    assert torch.equal(held[0][5][0], held[1][5][0]) and not held[1][5][1:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("Hq,D", [(2, 64), (8, 128), (16, 64)])
def test_small_queries_and_softmax_scales(fa, cuda_device, Hq, D, cap):
    """Rows of zeros and of next to nothing under softmax scales down to the least: the mean of the values
    they see.  And large queries under scales that make up for them."""
    c = ([100, 7, 16], 2, Hq, 1, D, 16, BF, cap, 40)
    q, cache, n, plain = _attend(fa, c, 17)
    q[:, :, 0] = 0.0
    q[:, 1, 1] = (q[:, 1, 1].float() * 1e-37).to(BF)
    for scale in (1e-20, 1e-38):
        o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softmax_scale=scale, softcap=cap, window_left=40)
        ro, rl, off, lse_off = plain_attention(q, *plain, scale, cap, 40)
        check(o, ro, off, "o")
        check_lse(lse, rl, lse_off)
    big = (q.float() * 2.0 ** 100).to(BF)
    o, lse = fa.fa_fwd_kvcache4(big.cuda(), cache, n, softmax_scale=2.0 ** -103, softcap=cap, window_left=40)
    ro, rl, off, lse_off = plain_attention(big, *plain, 2.0 ** -103, cap, 40)
    check(o, ro, off, "o")
    check_lse(lse, rl, lse_off)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("Hq,Sq,D", [(4, 1, 128), (2, 1, 64), (8, 1, 128), (8, 3, 64)])
def test_a_nan_query_stays_in_its_row(fa, cuda_device, Hq, Sq, D, cap):
    c = ([300, 40], Sq, Hq, 1, D, 16, BF, cap, -1)
    q, cache, n, _ = _attend(fa, c, 18)
    want, want_lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=cap)
    for bad in (math.nan, math.inf):
        for i, h in ((0, 0), (Sq - 1, 1), (0, Hq - 1)):
            y = q.clone()
            y[0, i, h, 5] = bad
            o, lse = fa.fa_fwd_kvcache4(y.cuda(), cache, n, softcap=cap)
            assert torch.isnan(o[0, i, h]).all() and torch.isnan(lse[0, h, i])
            o[0, i, h], lse[0, h, i] = want[0, i, h], want_lse[0, h, i]
            assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_a_nan_query_that_sees_nothing(fa, cuda_device, cap):
    """More queries than tokens: the first ones see no key, whatever they are."""
    c = ([2, 100], 4, 2, 1, 64, 16, BF, cap, -1)
    q, cache, n, _ = _attend(fa, c, 20)
    want, want_lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=cap)
    q[0, 1, 0, 7] = math.nan
    o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=cap)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert not o[0, :2].any() and torch.isneginf(lse[0, :, :2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("Sq,Hq,D", [(2, 2, 64), (3, 1, 128), (4, 2, 128), (5, 4, 128), (5, 4, 64)])
def test_values_that_some_rows_do_not_see(fa, cuda_device, Sq, Hq, D, cap, bad):
    """A V middle of NaN or infinity reaches the rows that see its token, in its 64 dims, and no other row: of the
    last token (seen by the last query alone) and of the first in the first query's window."""
    for lens in ([150, 41], [5000, 41]):
        c = (lens, Sq, Hq, 1, D, 16, BF, cap, 30)
        q, cache, n, plain = _attend(fa, c, 19)
        want, want_lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=cap, window_left=30)
        vs = cache.v_scale.clone()
        for token, sees in ((lens[0] - 1, [Sq - 1]), (lens[0] - Sq - 30, [0])):
            group = (D // 64 - 1)
            cache.v_scale[int(plain[4][0, token // 16]), 0, token % 16, group, 1] = bad
            o, lse = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=cap, window_left=30)
            cache.v_scale.copy_(vs)
            dims = slice(64 * group, 64 * group + 64)
            for i in sees:
                assert not torch.isfinite(o[0, i, :, dims]).any()
                o[0, i, :, dims] = want[0, i, :, dims]
            assert torch.equal(o, want) and torch.equal(lse, want_lse)


def _near_the_largest(dt, D):
    """Rows whose groups reach down to the type's largest value and end at steps that make the least value a tie."""
    top, unit = (65280.0, 2.0 ** 7) if dt == F16 else (255 * 2.0 ** 120, 2.0 ** 120 / 2)
    ends = [3840.0] if dt == F16 else [15 * 2.0 ** 120]
    g = torch.Generator().manual_seed(5)
    rows = []
    for i in range(40):
        hi = ends[0] if i < 2 else float(torch.randint(1, 400, (), generator=g)) * unit
        lo = top if i < 2 else top - float(torch.randint(0, 40, (), generator=g)) * unit
        x = -(torch.rand((D,), generator=g, dtype=torch.float64) * (lo - hi) + hi)
        x[0::64], x[1::64] = -lo, -hi
        rows.append((x if i != 1 else -x).to(dt))
    return torch.stack(rows)[:, None]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_values_next_to_the_largest_stay_finite(fa, cuda_device, D, dt):
    """A group's least value is half a scale from codes 0 and 1 where rounding leaves it there; code 0 lies below it,
    and must not be taken where the type has no such value."""
    x = _near_the_largest(dt, D)
    n, largest = x.shape[0], torch.finfo(dt).max
    assert torch.isfinite(x).all()
    table, pages = block_table([n], 16)
    cache = fa.KvCache4(*(t.cuda() for t in make_cache(pages, 1, 16, D, 1)), table.cuda())
    fa.kvcache4_append(cache, ints([0]), x.cuda(), x.cuda(), cu_new=sums([n]), max_new=n)
    codes, scales = quantise(x)
    c, s, m = unpack(codes, scales)
    beyond = m - 8 * s < -largest
    assert beyond[0].all() and int((beyond & (c == -8)).sum()) > 0
    want = m + s * torch.where(beyond, c.clamp_min(-7), c)
    assert ((want - x.double()).abs() <= s * (0.5 + 2.0 ** -19)).all()
    for got in fa.kvcache4_read(cache, ints([n]), sums([n]), n, dt):
        assert torch.isfinite(got).all()
        assert torch.equal(got.cpu(), want.to(dt))   # (from 64 bits at once: the sums are exact in 32)
    for i in (0, 1):   # a token by itself: its own values
        one = fa.KvCache4(cache.k, cache.v, cache.k_scale, cache.v_scale, ints([[int(table[0, 0])]]))
        o, _ = fa.fa_fwd_kvcache4(torch.zeros((1, 1, 1, D), dtype=dt, device="cuda"), one, ints([i + 1]),
                                  window_left=0)
        assert torch.isfinite(o).all()
