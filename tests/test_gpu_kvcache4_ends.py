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
