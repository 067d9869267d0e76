"""The build's two parts: the library, which C hosts use without PyTorch, and the
CPython binding, which belongs to one PyTorch. On sources of a few lines."""
import ctypes
import os

import pytest

from chunked_prefill_gqa_gb300 import build as B

KERNEL = 'extern "C" int answer() { return 42; }\n__global__ void k(int* p) { *p = 1; }\n'


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


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


@pytest.mark.parametrize("what", ["version", "git_version", "python"])
def test_a_binding_of_another_pytorch_or_python_does_not_count(tree, monkeypatch, what):
    """After an upgrade the old binding is neither current nor the one that is loaded."""
    pytest.importorskip("torch")
    B.build()
    old = B.binding_path()
    assert B.up_to_date() and os.path.exists(old)
    if what == "python":
        config = B.sysconfig.get_config_var
        monkeypatch.setattr(B.sysconfig, "get_config_var", lambda k: "cpython-399" if k == "SOABI" else config(k))
    else:
        other = tree / "torch"
        other.mkdir()
        with open(os.path.join(B._torch(), "version.py")) as f:
            lines = f.read().splitlines()
        key = {"version": "__version__", "git_version": "git_version"}[what]
        (other / "version.py").write_text("\n".join(f"{key} = '99.0'" if x.startswith(key) else x for x in lines))
        monkeypatch.setattr(B, "_torch", lambda: str(other))
    assert not B.up_to_date()
    assert B.binding_path() != old and not os.path.exists(B.binding_path())


def test_a_missing_binding_is_named(tree, monkeypatch):
    pytest.importorskip("torch")
    import chunked_prefill_gqa_gb300 as cp
    cp.load()
    monkeypatch.setattr(cp, "_binding", None)
    with pytest.raises(RuntimeError, match="no binding for this Python and PyTorch"):
        cp._native()
