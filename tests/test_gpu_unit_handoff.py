"""Backward problems in which every CTA runs several units, so that a unit's dK and
dV stores meet the next unit's dS^T: against 64 bits, and dK / dV bit for bit over
many calls.  Each is summed in a fixed order inside one unit, so they repeat in the
ordinary mode too (dQ, added up across units, does not)."""
import pytest
import torch

from test_gpu_score import _build, _check_all, _inputs, _mask
from score_ref import band

F16, BF = torch.float16, torch.bfloat16

# B, S, Hq, Hkv, D, dtype, mask keywords (None: causal), cap.  A tile of 128 columns in all
# but the 64-wide ones, which below 4096 keys run in a tile of their own
UNITS = [
    (4, 512, 30, 30, 128, BF, None, 50.0),
    (4, 512, 30, 30, 128, F16, dict(doc="mixed"), 0.0),
    (4, 512, 60, 30, 128, BF, dict(doc="pad", prefix="doc"), 30.0),
    (4, 512, 30, 30, 128, BF, None, 0.0),
    (4, 500, 30, 30, 120, BF, dict(doc="again", causal=False), 20.0),   # last blocks leave without the tiles
    (4, 512, 30, 30, 64, BF, dict(doc="mixed"), 30.0),
    (1, 4096, 16, 16, 64, BF, None, 0.0),
    (1, 4096, 16, 16, 64, F16, dict(doc="mixed"), 0.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("c", UNITS, ids=lambda c: "b%d_s%d_h%d_%d_d%d_%s_%s_cap%g" % (
    *c[:5], str(c[5])[6:], "_".join("%s%s" % kv for kv in (c[6] or {"causal": ""}).items()), c[7]))
def test_several_units_per_cta(fa, cuda_device, c):
    B, S, Hq, Hkv, D, dt, mask, cap = c
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert B * Hkv * ((S + 127) // 128) > 3 * sms
    x = _inputs(B, S, S, Hq, Hkv, D, dt, S + D, a=1.5 if cap else 1.0)
    if mask is None:
        kw, oks = dict(causal=True), [band(S, S, True)] * B
    else:
        m, oks = _mask(dict(B=B, S=S, **mask))
        kw = dict(mask_ranges=_build(fa, B, S, m))
    q, k, v, g = (t.cuda() for t in x)
    if S < 4096:   # (64-bit scores of every head at once)
        o, lse, first = _check_all(fa, x, oks, D ** -0.5, cap, kw)
    else:
        o, lse = fa.fa_fwd(q, k, v, softmax_scale=D ** -0.5, softcap=cap, **kw)
        first = fa.fa_bwd(q, k, v, o, g, lse, softmax_scale=D ** -0.5, softcap=cap, **kw)
    off = torch.zeros(2, dtype=torch.int64, device="cuda")
    for _ in range(49):
        again = fa.fa_bwd(q, k, v, o, g, lse, softmax_scale=D ** -0.5, softcap=cap, **kw)
        for i in (1, 2):
            off[i - 1] += (again[i].view(torch.int16) != first[i].view(torch.int16)).sum()
    assert off.tolist() == [0, 0], "elements of dK, dV that differ from the first call's"
    assert fa.device_status() == fa.FA_OK
