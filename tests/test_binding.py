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


def test_without_the_file_the_python_form_makes_the_calls(tmp_path, monkeypatch):
    monkeypatch.setattr(dash, "_FAST", None)
    monkeypatch.setattr(_build, "binding_path", lambda: str(tmp_path / "none.so"))
    pages, scales = torch.zeros(2, 3, 4, 64, dtype=torch.float8_e4m3fn), torch.zeros(2, 3, 4)
    q, i = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.warns(UserWarning, match="is missing"):
        with pytest.raises(ValueError, match="q must be a CUDA"):
            dash.attn_decode_fp8(q, pages, pages, scales, scales, i[None], i[:1])
    for call in (lambda: dash.qk_norm_rope(q, q, q[0, 0], q[0, 0], scales[0], i[:1]),
                 lambda: dash.cache_write_fp8(q, q, pages, pages, scales, scales, i[None], i[:1], i),
                 lambda: dash.attn_decode_shared(q, q[None], q[None], i[None], i[:1], 3)):
        with pytest.raises(ValueError, match="must be a CUDA"):
            call()


@pytest.mark.gpu
def test_both_forms_give_the_same(monkeypatch):
    g = torch.Generator("cuda").manual_seed(1)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda").bfloat16()
    hq, hkv, D, page, n = 4, 2, 128, 16, 50
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q, k, dq, dk = normal(n, hq, D), normal(n, hkv, D), normal(n, hq, D), normal(n, hkv, D)
    w = [torch.ones(D, device="cuda")] * 2
    rope, pos = dash.rope_table(n, D), torch.arange(n, dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]

    def all_calls():
        kp, vp = (torch.zeros(4, page, hkv, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv")
        ks, vs = (torch.zeros(4, page, hkv, device="cuda") for _ in "kv")
        out = [*dash.qk_norm_rope(q, k, *w, rope, pos), *dash.qk_norm_rope_bwd(q, k, dq, dk, *w, rope, pos)]
        dash.cache_write_fp8(k, dk, kp, vp, ks, vs, table, i32(0), i32(0, n))
        out += [kp.view(torch.uint8), vp.view(torch.uint8), ks, vs]
        out += dash.cache_read_fp8(kp, vp, ks, vs, table, i32(0), i32(0, n), n)
        out += dash.attn_decode_fp8(q[:1], kp, vp, ks, vs, table, i32(n))
        out += dash.attn_decode_shared(q[:1], *(torch.nn.functional.pad(t, (0, 0, 0, 0, 0, 14)).reshape(
            4, page, hkv, D) for t in (k, dk)), table, i32(n), 20)
        dash.dash_sync_status()
        return out

    compiled = all_calls()
    monkeypatch.setattr(dash, "_FAST", dash._NoFast())
    assert all(torch.equal(a, b) for a, b in zip(compiled, all_calls(), strict=True))
