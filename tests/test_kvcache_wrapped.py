"""The 8-bit cache calls take what stands in for a KvCache (a wrapper that hands its fields on); no call takes the
other kind of cache."""
import pytest
import torch

import attention_backward_preprocess_gb300 as mod

BF = torch.bfloat16


class Wrapped:
    """A cache with a note of its user's, handing everything else on."""

    def __init__(self, cache, note):
        self._inner, self.note = cache, note

    def __getattr__(self, name):
        return getattr(self._inner, name)


def _cache(cls, dtype):
    cache = cls.__new__(cls)
    cache._tensors = tuple(torch.zeros(1, dtype=dtype) for _ in range(5))
    return cache


def test_which_kind():
    eight, four = _cache(mod.KvCache, torch.float8_e4m3fn), _cache(mod.KvCache4, torch.uint8)
    mod._kind(eight, mod.KvCache)
    mod._kind(Wrapped(eight, 1), mod.KvCache)
    mod._kind(four, mod.KvCache4)
    for cache, cls in ((four, mod.KvCache), (Wrapped(four, 1), mod.KvCache), (eight, mod.KvCache4), (None, mod.KvCache),
                       (Wrapped(eight, 1), mod.KvCache4), (eight._tensors[0], mod.KvCache), (None, mod.KvCache4)):
        with pytest.raises(ValueError, match="cache: a KvCache"):
            mod._kind(cache, cls)


@pytest.mark.gpu
def test_wrapped(fa, cuda_device):
    f8 = torch.float8_e4m3fn
    cache = fa.KvCache(torch.zeros((4, 2, 16, 64), dtype=f8, device="cuda"), torch.zeros((4, 2, 64, 16), dtype=f8, device="cuda"),
                       torch.zeros((4, 2), device="cuda"), torch.zeros((4, 2), device="cuda"),
                       torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2))
    x = torch.randn((2, 20, 2, 64), device="cuda").to(BF)
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    fa.kvcache_append(Wrapped(cache, "a"), n, x, x)
    q = x[:, :1].contiguous()
    want = fa.fa_fwd_kvcache(q, cache, n + 20)
    for stream in (None, torch.cuda.current_stream()):
        got = fa.fa_fwd_kvcache(q, Wrapped(cache, "a"), n + 20, stream=stream)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and want[0].any()
