"""Tensors of a call that do not belong together are refused by the binding: the
kernels would read or write past the smaller ones (no GPU needed)."""
import pytest
import torch

BF = torch.bfloat16
B, Sq, Sk, Hq, Hkv, D = 2, 16, 24, 4, 2, 64


def _dense():
    x = dict(q=(B, Sq, Hq, D), k=(B, Sk, Hkv, D), v=(B, Sk, Hkv, D), o=(B, Sq, Hq, D), dout=(B, Sq, Hq, D))
    x = {n: torch.zeros(s, dtype=BF) for n, s in x.items()}
    x["lse"] = torch.zeros((B, Hq, Sq))
    return x


def _packed():
    x = {n: t.flatten(0, 1) for n, t in _dense().items() if n != "lse"}
    x["lse"] = torch.zeros((Hq, B * Sq))
    return x


def _half(t, dim):
    return t.narrow(dim, 0, t.shape[dim] // 2).contiguous()


WRONG = [("k", 0), ("k", 3), ("v", 0), ("v", 1), ("v", 2), ("o", 0), ("o", 1), ("o", 2), ("o", 3), ("dout", 0),
         ("dout", 1), ("dout", 3), ("lse", 0), ("dq", 0), ("dq", 1), ("dk", 1), ("dk", 2), ("dv", 0), ("dv", 3),
         ("k", "type"), ("v", "type"), ("o", "type"), ("dout", "type"), ("lse", "type"), ("dq", "type"), ("dv", "type")]
OF = dict(dq="q", dk="k", dv="v")


def _spoil(x, name, how):
    t = x[OF.get(name, name)]
    return dict(x, **{name: t.to(torch.float16 if name != "lse" else BF) if how == "type" else _half(t, how)})


@pytest.mark.parametrize("name,how", WRONG)
def test_dense(fa, name, how):
    x = _spoil(_dense(), name, how)
    with pytest.raises(ValueError, match="^%s:" % name):
        fa.fa_bwd(**x)
    if name in ("k", "v"):
        with pytest.raises(ValueError, match="^%s:" % name):
            fa.fa_fwd(x["q"], x["k"], x["v"])
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="^%s:" % name):
        fa.fa_bwd_stages(workspace=ws, **x)
    outs = {n: torch.zeros_like(_dense()[m]) for n, m in OF.items()}
    with pytest.raises(ValueError, match="^%s:" % name):
        fa.fa_bwd_noalloc(**dict(outs, **x))


@pytest.mark.parametrize("name,how", [("k", 2), ("v", 0), ("v", 1), ("o", 0), ("dout", 1), ("dq", 0), ("dk", 1), ("dv", 2),
                                      ("lse", "rows"), ("cu_seqlens_k", 0), ("cu_seqlens_q", "long"),
                                      ("cu_seqlens_k", "long"), ("cu_seqlens_k", "none")])
def test_packed(fa, name, how):
    cu = torch.tensor([0, 16, 32], dtype=torch.int32)
    x = dict(_packed(), cu_seqlens_q=cu, cu_seqlens_k=cu.clone(), max_seqlen_q=Sq, max_seqlen_k=Sk)
    if how == "long":
        x[name] = x[name].long()
    elif how == "none":
        x[name] = None
    elif how == "rows":
        x[name] = torch.zeros((Hq, 2 * B * Sq))
    else:
        x = _spoil(x, name, how)
    with pytest.raises(ValueError, match=name):
        fa.fa_bwd(**x)
    if name in ("k", "v", "cu_seqlens_q", "cu_seqlens_k"):
        with pytest.raises(ValueError, match=name):
            fa.fa_fwd(**{n: t for n, t in x.items() if n not in ("o", "dout", "lse", "dq", "dk", "dv")})


def test_what_belongs_together_but_is_no_gpus(fa):
    with pytest.raises(ValueError, match="q: not on a GPU"):
        fa.fa_bwd(**_dense())
    cu = torch.tensor([0, 16, 32], dtype=torch.int32)
    with pytest.raises(ValueError, match="q: not on a GPU"):
        fa.fa_bwd(cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=Sq, max_seqlen_k=Sk, **_packed())


def test_value_head_dim_of_the_staged_calls(fa):
    x = _dense()
    for n in ("v", "o", "dout"):
        x[n] = torch.cat([x[n], x[n]], dim=3)
    with pytest.raises(ValueError, match="^v:"):
        fa.fa_bwd_stages(workspace=torch.zeros(1 << 20, dtype=torch.uint8), **x)


# ------------------------------------------- the tensors of the extensions
def _more(**kw):
    """_ext for q [2, 16, 4, D] and 24 keys, whose tensors lie on ``at`` (-1: these)."""
    import attention_backward_preprocess_gb300 as mod
    at = kw.pop("at", -1)
    return mod._ext(Hq, sizes=(B, Sq, Sk, at), rows=B * Sq, dtype=BF, **kw)


GOOD = dict(alibi_slopes=torch.zeros(Hq), seqused_q=torch.zeros(B, dtype=torch.int32),
            seqused_k=torch.zeros(B, dtype=torch.int32), bias=torch.zeros((1, Hq, Sq, Sk), dtype=BF),
            dbias=torch.zeros((B, Hq, Sq, Sk), dtype=BF),
            dropout=(0.1, 1, 0, torch.zeros((B, Hq, Sq, 1), dtype=torch.int32)))
SHORT = [("alibi_slopes", torch.zeros(Hq - 1)), ("alibi_slopes", torch.zeros((B - 1, Hq))),
         ("seqused_q", torch.zeros(B - 1, dtype=torch.int32)), ("seqused_k", torch.zeros(0, dtype=torch.int32)),
         ("bias", torch.zeros((B, Hq, Sq, Sk))), ("bias", torch.zeros((B, Hq - 2, Sq, Sk), dtype=BF)),
         ("bias", torch.zeros((B, Hq, Sq - 1, Sk), dtype=BF)), ("bias", torch.zeros((1, 1, Sq, Sk - 8), dtype=BF)),
         ("dbias", torch.zeros((B, Hq, Sq, Sk - 8), dtype=BF)), ("dbias", torch.zeros((B, Hq, Sq, Sk))),
         ("dropout", (0.1, 1, 0, torch.zeros((B, Hq, Sq - 1, 1), dtype=torch.int32)))]


@pytest.mark.parametrize("name", GOOD)
def test_extension_tensors_that_reach(name):
    assert _more(**{name: GOOD[name]}) is not None
    with pytest.raises(ValueError, match="on q's GPU"):
        _more(at=0, **{name: GOOD[name]})   # they lie elsewhere


@pytest.mark.parametrize("name,t", SHORT, ids=["%s%d" % (n, i) for i, (n, _) in enumerate(SHORT)])
def test_extension_tensors_too_short(name, t):
    with pytest.raises(ValueError, match=name):
        _more(**{name: t})


def test_a_workspace_elsewhere():
    import attention_backward_preprocess_gb300 as mod
    ws = torch.zeros(256, dtype=torch.uint8)
    mod._scratch(ws, -1)
    mod._scratch(None, 0)
    for bad, at in ((ws, 0), (ws.view(torch.float32), -1), (ws[::2], -1)):
        with pytest.raises(ValueError, match="workspace"):
            mod._scratch(bad, at)
