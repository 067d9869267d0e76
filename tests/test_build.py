"""The build's two parts: the library, which C hosts use without PyTorch, and the
CPython binding, which belongs to one PyTorch. On sources of a few lines."""
import ctypes
import os

import pytest

from chunked_prefill_gqa_gb300 import build as B

KERNEL = 'extern "C" int answer() { return 42; }\n__global__ void k(int* p) { *p = 1; }\n'


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source folder with one small kernel, and a folder for what is built from it."""
    src, inc, out = tmp_path / "csrc", tmp_path / "include", tmp_path / "out"
    src.mkdir()
    inc.mkdir()
    (src / "small.cu").write_text(KERNEL)
    (src / "binding.cpp").write_text('extern "C" int answer();\nextern "C" int twice() { return 2 * answer(); }\n')
    (inc / "attn_prefill.h").write_text("")
    monkeypatch.setattr(B, "CSRC", str(src))
    monkeypatch.setattr(B, "INCLUDE", str(inc))
    monkeypatch.setattr(B, "OUT", str(out))
    monkeypatch.setattr(B, "LIB", str(out / "libattnprefill.so"))
    if hasattr(B, "BINDING"):
        monkeypatch.setattr(B, "BINDING", str(out / "_binding.so"))
    return tmp_path


def answer():
    return ctypes.CDLL(B.LIB).answer()


def test_the_library_without_pytorch(tree, monkeypatch, capfd):
    find = B.importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert B.build() == B.LIB and answer() == 42
    assert "PyTorch is not installed" in capfd.readouterr().err
    assert [f for f in os.listdir(B.OUT) if "binding" in f] == []
    assert B.up_to_date()
    before = os.path.getmtime(B.LIB)
    B.build()  # nothing to do
    assert os.path.getmtime(B.LIB) == before


def test_a_binding_that_does_not_compile_leaves_the_library(tree):
    pytest.importorskip("torch")
    (tree / "csrc" / "binding.cpp").write_text("this is not C++\n")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        B.build()
    assert answer() == 42
    assert not B.up_to_date()
