"""Wait budgets of any size: the second bound of the 4-bit cache attention's loading warps, on the CPU through
the kernel's own comparison."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bound(tmp_path_factory):
    cxx, cuda = shutil.which("g++") or shutil.which("c++"), os.environ.get("CUDA_HOME", "/usr/local/cuda")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path_factory.mktemp("budget") / "wait_budget"
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(cuda, "include"), "-I",
                    os.path.join(ROOT, "attention_backward_preprocess_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "wait_budget.cpp"), "-o", str(exe)], check=True)
    return lambda *a: subprocess.run([str(exe)] + [str(x) for x in a], check=True, capture_output=True, text=True).stdout.strip()


@pytest.mark.parametrize("budget", [1, 2 * 10 ** 9, 2 ** 62 - 1, 2 ** 62, 2 ** 63 - 1])
def test_twice_the_budget(bound, budget):
    """(2^62 and above: twice that has no place in 64 bits with a sign)"""
    for waited in (0, 1, budget, 2 * budget):
        assert bound(waited, budget) == "within"
    if 2 * budget + 2 < 2 ** 64:
        assert bound(2 * budget + 2, budget) == "over"


@pytest.mark.gpu
def test_no_limit_worth_the_name(fa, cuda_device):
    """Calls under the largest budget there is end without an error, with the results of every other call."""
    from test_gpu_kvcache4 import BF, _attend
    q, cache, n, _ = _attend(fa, ([20000, 300], 3, 16, 2, 128, 64, BF, 20.0, -1))
    want = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=20.0)
    assert fa.device_status() == fa.FA_OK
    before = fa.lib().fa_set_wait_timeout_ns(2 ** 63 - 1)
    try:
        got = fa.fa_fwd_kvcache4(q.cuda(), cache, n, softcap=20.0)
        assert fa.device_status() == fa.FA_OK
    finally:
        fa.lib().fa_set_wait_timeout_ns(before)
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()
