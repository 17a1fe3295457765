"""Without the compiled short way in (not built, or built against another torch) every
call still goes through, with the same results."""
import pytest
import torch

import attention_backward_preprocess_gb300 as mod

BF = torch.bfloat16


@pytest.fixture(params=["missing", "another", "no library"])
def without(request, fa, tmp_path, monkeypatch):
    """The binding with no file, a library that is no such module, one that does not load."""
    path = tmp_path / "_fa_torch.so"
    if request.param == "another":
        path = mod.LIB_PATH
    elif request.param == "no library":
        path.write_bytes(b"not for this machine")
    monkeypatch.setattr(mod, "SHORT_PATH", str(path))
    monkeypatch.setattr(mod, "_short", None)
    return mod


def test_calls_take_the_python_way(without):
    with pytest.warns(RuntimeWarning, match="us more on the host"):
        b = without._binding()
    assert b is without._binding()
    for name in ("agree", "fwd", "bwd", "mask_ranges", "cache", "append", "attend"):
        assert getattr(b, name)(1, 2, 3) is None
    q = torch.zeros((1, 64, 2, 64), dtype=BF)
    with pytest.raises(ValueError, match="q: not on a GPU"):   # the checks of the Python way
        without.fa_fwd(q, q, q)


def test_the_library_itself_stays_required(without, tmp_path, monkeypatch):
    monkeypatch.setattr(without, "_lib", None)
    monkeypatch.setattr(without, "LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(RuntimeError, match="no fallback"):
        without._binding()


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore::RuntimeWarning")
def test_same_results(fa, cuda_device, tmp_path, monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)   # noqa: E731
    q, k, v, do = r(2, 200, 4, 64), r(2, 200, 2, 64), r(2, 200, 2, 64), r(2, 200, 4, 64)
    ids = torch.randint(0, 3, (2, 200), generator=g, device="cuda").int()
    pages = [torch.zeros(s, dtype=torch.float8_e4m3fn, device="cuda") for s in ((6, 2, 32, 64), (6, 2, 64, 32))]
    scales = [torch.zeros((6, 2), device="cuda") for _ in range(2)]
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    none = torch.zeros(2, dtype=torch.int32, device="cuda")

    def run():
        out = list(mod.fa_fwd(q, k, v, causal=True))
        out += mod.fa_bwd(q, k, v, out[0], do, out[1], causal=True)[1:]
        m = mod.mask_ranges(2, 200, doc_ids=ids)
        out += mod.fa_fwd(q, k, v, softcap=20.0, mask_ranges=m)
        out += mod.fa_bwd(q, k, v, out[-2], do, out[-1], softcap=20.0, mask_ranges=m)[1:]
        cache = mod.KvCache(*pages, *scales, table)
        mod.kvcache_append(cache, none, k[:, :70].contiguous(), v[:, :70].contiguous())
        out += mod.fa_fwd_kvcache(q[:, :2].contiguous(), cache, none + 70)
        return out + [t.clone().view(torch.uint8) for t in pages] + [t.clone() for t in scales]
    want = run()
    monkeypatch.setattr(mod, "SHORT_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(mod, "_short", None)
    assert isinstance(mod._binding(), mod._NoShortWay)
    for a, b in zip(want, run()):
        assert torch.equal(a, b)
