"""The hand-off of the main backward kernel's dS^T tiles between units: every
interleaving of its warps on the CPU, through the kernel's own phase arithmetic."""
import itertools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path_factory.mktemp("epi") / "epi_handoff"
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "attention_backward_preprocess_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "epi_handoff.cpp"), "-o", str(exe)], check=True)
    return lambda *a: subprocess.run([str(exe)] + [str(x) for x in a], check=True, capture_output=True,
                                     text=True).stdout.strip()


@pytest.mark.parametrize("stores", list(itertools.product((0, 1), repeat=3)))
@pytest.mark.parametrize("slices", [1, 2])
def test_no_interleaving_overwrites_a_tile(walk, slices, stores):
    """One slice per unit (64-wide tiles) and two (128-wide), units whose results
    leave by tensor stores and units whose results do not, in any order."""
    got = walk(slices, *stores, 0)
    assert got.startswith("ok "), got
    assert int(got.split()[1]) > 100


def test_the_walk_finds_a_wait_that_does_not_hold(walk):
    """A wait for the other group's slice barrier looks at the same parity in every
    unit of two slices and lets a group through while the other has stored none;
    with one slice the parity alternates and it holds.  Without a wait neither does."""
    assert "under a store" in walk(2, 1, 1, 1, 1)
    assert walk(1, 1, 1, 1, 1).startswith("ok ")
    assert "under a store" in walk(1, 1, 1, 1, 2) and "under a store" in walk(2, 1, 1, 1, 2)
