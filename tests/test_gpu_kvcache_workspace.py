"""fa_fwd_kvcache keeps to the workspace it asks for."""
import pytest
import torch

from test_gpu_kvcache import BF, F16, _attend


@pytest.mark.gpu
@pytest.mark.parametrize("D,Sq,Hq,Hkv,dt", [(64, 1, 8, 8, BF), (128, 1, 8, 8, F16), (64, 4, 16, 4, F16), (128, 4, 16, 4, BF)])
def test_nothing_behind_the_workspace(fa, cuda_device, D, Sq, Hq, Hkv, dt):
    """Long sequences cut between all workers, 8 and 16 rows a worker; the bytes behind
    the workspace stay as they were, and the results are those of a call without one."""
    c = ([9000, 4100, 30000], Sq, Hq, Hkv, D, 64, dt, 0.0, -1)
    q, cache, n, _ = _attend(fa, c, 31)
    q = q.cuda()
    want = fa.fa_fwd_kvcache(q, cache, n)
    need = fa.fa_fwd_kvcache_workspace_bytes(D)
    room = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = fa.fa_fwd_kvcache(q, cache, n, workspace=room[:need])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((room[need:] == 0xA5).all()) and bool((room[:need] != 0xA5).any())
