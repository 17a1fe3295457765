"""The 4-bit cache's and the rotary calls give the same through the compiled short way in and through Python, and
refuse the same."""
import pytest
import torch

import attention_backward_preprocess_gb300 as mod

BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(params=["short", "python"])
def way(request, fa, monkeypatch, tmp_path):
    if request.param == "python":
        monkeypatch.setattr(mod, "SHORT_PATH", str(tmp_path / "missing.so"))
        monkeypatch.setattr(mod, "_short", None)
        with pytest.warns(RuntimeWarning):
            mod._binding()
        assert isinstance(mod._binding(), mod._NoShortWay)
    return request.param


def _tensors(D=64, H=2, P=6, page=32):
    codes = [torch.zeros((P, H, page, D // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((P, H, page, D // 64, 2), dtype=BF, device="cuda") for _ in range(2)]
    return codes + scales + [torch.arange(P, dtype=torch.int32, device="cuda").view(2, P // 2)]


def _run(D, dt):
    g = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)   # noqa: E731
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    at = torch.randint(-9, 9000, (2, 70), generator=g, device="cuda").int()
    table = mod.rope_table(D // 2, scaling=("ntk", 2.0))
    qkv = r(2, 70, 8, D)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:].contiguous()   # q, k: slices of a joint projection
    out = list(mod.rope(q, k, table, positions=at))
    out += mod.rope(q, k, table, offsets=at[:, 0].contiguous(), interleaved=True)
    out += mod.rope_bwd(out[0], out[1], table)
    out += mod.rope(q.reshape(140, 4, D), None, table, positions=at.view(140))[:1]
    assert mod.rope(q, None, table)[1] is None
    tensors = _tensors(D)
    cache = mod.KvCache4(*tensors)
    for held, n in ((0, 41), (41, 29)):
        mod.kvcache4_append(cache, none + held, out[1][:, held:held + n].contiguous(), v[:, held:held + n].contiguous())
    cu = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    mod.kvcache4_append(cache, none + 70, r(8, 2, D), r(8, 2, D), cu_new=cu, max_new=5)
    lens = torch.tensor([73, 75], dtype=torch.int32, device="cuda")
    last = out[0][:, -3:].contiguous()
    for kw in ({}, dict(softmax_scale=0.3, softcap=20.0, window_left=33)):
        out += mod.fa_fwd_kvcache4(last, cache, lens, **kw)
    out += mod.kvcache4_read(cache, lens, torch.tensor([0, 73, 148], dtype=torch.int32, device="cuda"), 148, dt)
    out += mod.kvcache4_read(cache, lens, cu, 8, F16, first=none + 60)
    assert mod.device_status() == mod.FA_OK
    return out + [t.view(torch.uint8).clone() for t in tensors[:4]]


_first = {}


@pytest.mark.gpu
@pytest.mark.parametrize("D,dt", [(64, BF), (128, F16)])
def test_same_results(cuda_device, way, D, dt):
    got = _run(D, dt)
    want = _first.setdefault((D, dt), got)   # (of whichever way came first)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.gpu
def test_caches_refused(cuda_device, way):
    k, v, ks, vs, t = _tensors()
    mod.KvCache4(k, v, ks, vs, t)
    for bad in ((k.view(torch.int8), v, ks, vs, t), (k, v[:3], ks, vs, t), (k, v, ks.half(), vs, t), (k, v, ks, vs[..., :1], t),
                (k, v, ks, vs, t.long()), (k, v, ks, vs, t.cpu()), (k, v.cpu(), ks, vs, t), (k, v, ks, vs, t[:, ::2]),
                (k[0], v, ks, vs, t), (k, v, ks, vs, t.view(-1)), (k[..., ::2], v[..., ::2], ks, vs, t)):
        with pytest.raises(ValueError):
            mod.KvCache4(*bad)
    cache = mod.KvCache4(k, v, ks, vs, t)
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros((2, 1, 2, 64), dtype=BF, device="cuda")
    for call in (lambda: mod.kvcache4_append(cache, n.long(), x, x), lambda: mod.kvcache4_append(cache, n, x, x[:, :, :1]),
                 lambda: mod.fa_fwd_kvcache4(x[:1], cache, n), lambda: mod.fa_fwd_kvcache4(x, cache, n[:1]),
                 lambda: mod.kvcache4_read(cache, n, n, 4), lambda: mod.kvcache4_read(cache, n, torch.zeros_like(t).view(-1)[:3], 0),
                 lambda: mod.rope(x, x.half(), mod.rope_table(64)), lambda: mod.rope(x, x, mod.rope_table(64), positions=n)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mod.rope(x, x, mod.rope_table(66)), lambda: mod.fa_fwd_kvcache4(x, cache, n, softcap=-1.0)):
        with pytest.raises(mod.FaError):
            call()
    assert mod.device_status() == mod.FA_OK
