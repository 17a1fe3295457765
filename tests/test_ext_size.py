"""fa_ext carries no size: who passes one can ask the library for its own (no GPU)."""
import ctypes
import os
import shutil
import subprocess

import pytest

import attention_backward_preprocess_gb300 as mod

C = """#include <stdio.h>
#include <stddef.h>
size_t fa_ext_bytes(void);
int main(void) { printf("%zu\\n", fa_ext_bytes()); return 0; }
"""


def test_the_library_says_its_size(fa):
    assert fa.lib().fa_ext_bytes() == ctypes.sizeof(fa.FaExt)


def test_from_c(fa, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "size.c").write_text(C)
    where = os.path.dirname(mod.LIB_PATH)
    subprocess.run([cc, str(tmp_path / "size.c"), "-o", str(tmp_path / "size"), "-L" + where, "-l:libfa_gb300.so",
                    "-Wl,-rpath," + where], check=True)
    out = subprocess.run([str(tmp_path / "size")], check=True, capture_output=True, text=True).stdout
    assert int(out) == ctypes.sizeof(fa.FaExt)


@pytest.mark.parametrize("size", [None, 136])
def test_a_library_of_another_header_is_refused(tmp_path, monkeypatch, size):
    """One whose struct is shorter, and one from before it could say so."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "old.c").write_text("#include <stddef.h>\n" + (
        "int other;\n" if size is None else "size_t fa_ext_bytes(void) { return %d; }\n" % size))
    subprocess.run([cc, "-shared", "-fPIC", str(tmp_path / "old.c"), "-o", str(tmp_path / "old.so")], check=True)
    monkeypatch.setattr(mod, "_lib", None)
    monkeypatch.setattr(mod, "LIB_PATH", str(tmp_path / "old.so"))
    with pytest.raises(RuntimeError, match="another include/fa.h"):
        mod.lib()
