"""When build() compiles again: after a change of any file that the library is made of."""
import os

import pytest

from sparse_verification_attention_gb300 import build_lib


@pytest.mark.parametrize("name", ["csrc/kernel.cu", "csrc/types.h", "csrc/plan.cuh", "include/sva.h"])
def test_library_is_stale_after_a_source_changed(tmp_path, monkeypatch, name):
    files = ["csrc/kernel.cu", "csrc/types.h", "csrc/plan.cuh", "include/sva.h", "libsva.so"]
    for f in files:
        (tmp_path / f).parent.mkdir(exist_ok=True)
        (tmp_path / f).write_text("")
    built = os.path.getmtime(build_lib.__file__) + 1000
    for f in files:
        os.utime(tmp_path / f, (built, built))
    monkeypatch.setattr(build_lib, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(build_lib, "INCLUDE", str(tmp_path / "include"))
    monkeypatch.setattr(build_lib, "LIB", str(tmp_path / "libsva.so"))
    assert not build_lib._stale([])
    os.utime(tmp_path / name, (built + 1, built + 1))
    assert build_lib._stale([])
