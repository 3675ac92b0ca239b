"""Building the native parts: what depends on what, and when a part is built again."""
import os

import pytest

from sparse_mla_decode_front_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build working in an empty folder, with one small source."""
    os.makedirs(tmp_path / "csrc")
    (tmp_path / "csrc" / "small.cu").write_text('extern "C" int small(void) { return 7; }\n')
    (tmp_path / "csrc" / "bind.cpp").write_text("")
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / "_bind.so"))
    return tmp_path


def test_library_is_built_where_the_binding_cannot_be(tree, monkeypatch):
    # the C library needs nvcc alone; the binding needs torch's headers, Python's and a host compiler
    monkeypatch.setenv("CXX", "false")
    for _ in range(2):   # the second time the library is up to date, and the binding still is not
        with pytest.raises(Exception):
            build.build()
        assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)
