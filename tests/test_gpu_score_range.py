"""Capped scores whose uncapped ones leave 32 bits: a cap maps them to +-softcap, and a
visible key at -softcap is not a hidden one."""
import pytest
import torch

from test_gpu_score import _build, _check_all, _inputs, _mask
from score_ref import band

BF = torch.bfloat16

# B, S, Hq, Hkv, D, mask keywords (None: causal); few tiles, and more than the GPU has SMs
SHAPES = [
    (1, 200, 2, 1, 64, None), (1, 200, 2, 2, 128, None), (2, 150, 2, 1, 128, dict(doc="mixed")),
    (1, 300, 60, 20, 128, None), (1, 300, 60, 60, 64, None), (1, 300, 60, 20, 128, dict(doc="pad", prefix="doc")),
]


@pytest.mark.gpu
@pytest.mark.parametrize("signs", ["all below", "mixed"])
@pytest.mark.parametrize("c", SHAPES, ids=lambda c: "b%d_s%d_h%d_%d_d%d_%s" % (*c[:5], "band" if c[5] is None else "docs"))
def test_scores_beyond_32_bits(fa, cuda_device, c, signs):
    """q = 1e20 and k = -1e20, 0 or 1e20 in every dim: products of -inf, 0 and inf in 32
    bits, capped -1.5, 0 and 1.5, all of which weigh in the softmax."""
    B, S, Hq, Hkv, D, mask = c
    _, _, v, g = _inputs(B, S, S, Hq, Hkv, D, BF, S + D)
    gen = torch.Generator().manual_seed(S)
    s = torch.randint(-1, 2, (B, S, Hkv, 1), generator=gen).float() if signs == "mixed" else -torch.ones((B, S, Hkv, 1))
    q = torch.full((B, S, Hq, D), 1e20).to(BF)
    k = (s * 1e20).expand(B, S, Hkv, D).contiguous().to(BF)
    if mask is None:
        kw, oks = dict(causal=True), [band(S, S, True)] * B
    else:
        m, oks = _mask(dict(B=B, S=S, **mask))
        kw = dict(mask_ranges=_build(fa, B, S, m))
    _check_all(fa, (q, k, v, g), oks, D ** -0.5, 1.5, kw)
