"""What the build makes without torch, and what the binding does without the native marshalling (no GPU)."""

import os

import pytest
import torch

import mla_decode_attention_02_gb300 as mla
import mla_decode_attention_02_gb300._binding as binding
from mla_decode_attention_02_gb300 import build as B


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one small translation unit, built in a directory of its own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int mla_one() { return 1; }\n')
    monkeypatch.setattr(B, "sources", lambda: [str(src)])
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libone.so"))
    return tmp_path


def test_the_library_is_built_where_the_host_module_cannot_be(small, monkeypatch):
    def fails():
        raise RuntimeError("no Python.h")
    monkeypatch.setattr(B, "_build_host", fails)
    with pytest.warns(UserWarning, match="no Python.h"):
        assert B.build(force=True) == B.LIB_PATH
    assert os.path.getsize(B.LIB_PATH) > 0


def test_the_library_is_built_without_torch(small, monkeypatch):
    real = B.importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else real(n, *a))
    monkeypatch.setattr(B, "_build_host", lambda: pytest.fail("needs torch"))
    B.build(force=True)
    assert os.path.getsize(B.LIB_PATH) > 0 and B.up_to_date()
    os.utime(B.sources()[0], (4e9, 4e9))
    assert not B.up_to_date()


def test_the_library_is_built_beside_a_torch_that_does_not_import(small, monkeypatch):
    def broken():
        raise ImportError("libtorch is broken")
    monkeypatch.setattr(B, "host_path", broken)
    assert not B.up_to_date()
    with pytest.warns(UserWarning, match="libtorch is broken"):
        B.build()
    assert os.path.getsize(B.LIB_PATH) > 0


def test_a_source_that_does_not_compile_is_an_error(small):
    (small / "one.cu").write_text("int x = ;\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build(force=True)


def test_calls_without_the_native_marshalling(monkeypatch):
    """The Python checks take every call (here: refuse it), after one warning."""
    monkeypatch.setattr(binding, "_host", None)
    monkeypatch.setattr(binding, "_load_host", lambda: exec("raise ImportError('none here')"))
    cpu = torch.zeros(4, 128, 192, dtype=torch.bfloat16)
    with pytest.warns(UserWarning, match="marshalled in Python"):
        with pytest.raises(ValueError, match="CUDA"):
            mla.query(cpu[..., :128], cpu[..., 128:], None, None)
    for call in (lambda: mla.cache_append(cpu[0], cpu[0], None, None, None, None, None),
                 lambda: mla.tree_plan(torch.zeros(2, dtype=torch.int32), None, None, max_pages_per_seq=1),
                 lambda: mla.cache_commit(None, torch.zeros(1, 1, dtype=torch.int32), None, None, None, None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_a_host_module_of_another_torch_is_not_used(monkeypatch):
    """Its name carries the torch and the Python ABI that it was built for: another's is neither up to date nor loaded."""
    assert B.up_to_date() and binding._load_host() is not None
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert not B.up_to_date()
    with pytest.raises(ImportError, match="1.0.0"):
        binding._load_host()
    monkeypatch.setattr(binding, "_host", None)
    with pytest.warns(UserWarning, match="1.0.0"):
        assert binding._native() is binding._PythonOnly
