"""Tensors of one call that lie over each other: refused by rope and by the 4-bit cache's read (no GPU)."""
import pytest
import torch

from test_gpu_kvcache4 import _read4, _struct
from test_gpu_rope import _call

@pytest.mark.parametrize("q,k", [
    (dict(in_=0x2000, out=0x3000), dict(in_=0x4000, out=0x3000)),      # one output for both
    (dict(in_=0x2000, out=0x2000), dict(in_=0x2000, out=0x2000)),      # one tensor as both, in place
    (dict(in_=0x2000, out=0x4000), dict(in_=0x4000, out=0x5000)),      # q's output is k's input
    (dict(in_=0x2000, out=0x3000), dict(in_=0x4000, out=0x2000)),
    (dict(in_=0x2000, out=0x3000), dict(in_=0x4000, out=0x3100)),      # outputs a row apart
    (dict(in_=0x2000, out=0x2100), None),                              # a row further, not in place
    (dict(in_=0x2100, out=0x2000), None),
    (dict(in_=0x2000, out=0x3000), dict(in_=0x3500, out=0x5000)),      # the last row of 1536 bytes
    (dict(in_=0x2000, out=0x2000, in_stride=(1152, 384, 64), out_stride=(1152, 384, 64)),
     dict(in_=0x4000, out=0x2000, out_stride=(1152, 384, 64)))])       # strides: the same start
def test_rope_over_itself(fa, q, k):
    assert _call(fa, q, k) == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="such calls would run, and these addresses are nobody's")
def test_rope_beside_itself(fa):
    """Neighbours, slices of a joint projection in place, and one input with two outputs are no overlap: such
    calls get as far as asking for a GPU."""
    joint = dict(in_stride=(1152, 384, 64), out_stride=(1152, 384, 64))
    no_gpu = _call(fa, dict(in_=0x2000, out=0x2000))
    assert no_gpu not in (0, 1)
    for q, k in ((dict(in_=0x2000, out=0x2600), dict(in_=0x2c00, out=0x3200)),
                 (dict(in_=0x2000, out=0x2000, **joint), dict(in_=0x2100, out=0x2100, **joint)),
                 (dict(in_=0x2000, out=0x3000), dict(in_=0x2000, out=0x4000))):
        assert _call(fa, q, k) == no_gpu


@pytest.mark.parametrize("v", [0x7000, 0x7010, 0x7000 + 15 * 2 * 128 * 2 - 16])
def test_read_over_itself(fa, v):
    assert _read4(fa, _struct(fa), cu=0x9000, k=0x7000, v=v) == 1
    assert _read4(fa, _struct(fa), cu=0x9000, k=v, v=0x7000) == 1
