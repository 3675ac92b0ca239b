"""Building the native parts: what depends on what, and when a part is built again."""
import os

import pytest

from sparse_mla_decode_front_b200 import _lib, build, experts


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


def test_binding_is_built_again_for_another_torch(tree, monkeypatch):
    built = []

    def compiler(cmd, check):
        built.append(cmd)
        (tree / "_bind.so.tmp").write_text("")
    monkeypatch.setattr(build.subprocess, "run", compiler)
    tag = [_lib.bind_tag()]
    monkeypatch.setattr(_lib, "bind_tag", lambda: tag[0])
    build.build_bind()
    build.build_bind()
    assert len(built) == 1                       # nothing changed
    tag[0] = "torch 0.1, cpython-399"
    build.build_bind()
    build.build_bind()
    assert len(built) == 2 and any(tag[0] in a for a in built[1])
    (tree / "_build" / "bind.tag").unlink()      # built for what is not known
    build.build_bind()
    assert len(built) == 3


def test_binding_of_another_torch_is_refused(monkeypatch):
    monkeypatch.setattr(experts, "_bound", None)
    experts._native()                            # the one that the tests run with fits
    monkeypatch.setattr(experts, "_bound", None)
    monkeypatch.setattr(_lib, "bind_tag", lambda: "torch 0.1, cpython-399")
    with pytest.raises(ImportError, match="built for torch .* this is torch 0.1"):
        experts._native()
