"""The compiled part of the Python binding, what needs no GPU: its file's name, and that it is used."""
import os
import sysconfig

import pytest
import torch

import deterministic_attention_backward_fa_gb300 as dash
from deterministic_attention_backward_fa_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_the_file_is_named_by_all_that_it_is_compiled_against():
    # it is C++ against torch and C against the interpreter: another of either must not find it
    name = os.path.basename(_build.binding_path())
    assert torch.__version__.replace("+", "_") in name
    assert name.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and sysconfig.get_config_var("SOABI") in name
    assert os.path.exists(_build.binding_path())


def test_the_compiled_form_is_the_one_that_is_asked():
    fast = dash._fast()
    for name in ("qk_norm_rope", "qk_norm_rope_bwd", "cache_write_fp8", "cache_read_fp8", "attn_decode_fp8",
                 "attn_decode_shared"):
        f = getattr(fast, name)
        assert type(f).__name__ == "builtin_function_or_method"
        assert f() is None  # a wrong number of arguments: the Python form's to answer


def test_the_library_is_built_without_what_the_binding_needs(tmp_path, monkeypatch):
    # a stand-in for nvcc that makes empty files: only the order and the needs are looked at
    cc = tmp_path / "nvcc"
    cc.write_text("#!/bin/sh\nwhile [ $# -gt 1 ]; do if [ $1 = -o ]; then : > $2; fi; shift; done\n")
    cc.chmod(0o755)
    lib, so = tmp_path / "lib.so", tmp_path / "binding.so"
    for name, value in (("nvcc", lambda: str(cc)), ("BUILD", str(tmp_path / "objects")), ("LIB", str(lib)),
                        ("binding_path", lambda: str(so))):
        monkeypatch.setattr(_build, name, value)
    # without Python's headers
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    with pytest.warns(UserWarning, match="Python.h"):
        assert _build.build(force=True) == str(lib)
    assert lib.exists() and not so.exists() and _build.up_to_date()
    monkeypatch.undo()
    # with all of them, where it does not compile: the library stands, and the error is told
    for name, value in (("nvcc", lambda: str(cc)), ("BUILD", str(tmp_path / "objects")), ("LIB", str(lib)),
                        ("binding_path", lambda: str(so)), ("_torch_flags", lambda: (["-DDASH_H", "-include", "/none"], []))):
        monkeypatch.setattr(_build, name, value)
    lib.unlink()
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        _build.build(force=True)
    assert lib.exists() and not so.exists()
