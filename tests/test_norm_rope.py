"""Norms of queries and keys with their rotation, what needs no GPU: the
refusals, the table of angles, and the 64-bit backward that the GPU tests compare
with, against differences of the forward."""
import ctypes

import pytest
import torch

import deterministic_attention_backward_fa_gb300 as dash

import _norm_rope as R


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [8, 16])
def test_plain_backward_against_differences(pairs, rot):
    g = torch.Generator().manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=g, dtype=R.F64)
    x, dz, w, h, eps = normal(5, 3, 16), normal(5, 3, 16), 1 + 0.3 * normal(16), 1e-6, 1e-5
    rope, pos = R.table(40, rot), torch.tensor([0, 1, 2, 39, 7])
    loss = lambda a, b: (R.forward(a, b, rope, pos, eps, pairs)[0] * dz).sum()
    (dx, dw), _ = R.backward(x, dz, w, rope, pos, eps, pairs)
    for grad, args in ((dx, lambda d: (x + d, w)), (dw, lambda d: (x, w + d))):
        d = normal(*grad.shape)
        diff = (loss(*args(h * d)) - loss(*args(-h * d))) / (2 * h)
        assert abs(diff - (grad * d).sum()) <= 1e-7 * (1 + abs(diff))


def test_rope_table():
    # in 64 bits, so that far positions keep their digits; fp32 holds a value to 2^-24 of it
    t = dash.rope_table(200000, 32, base=500000.0, device="cpu")
    want = R.table(200000, 32, 500000.0)
    assert t.shape == (200000, 32) and t.dtype == torch.float32
    assert (t.double() - want).abs().max() <= 2.0 ** -24


def test_refusals_before_any_device_call():
    L, nul, fake = dash.lib(), ctypes.c_void_p(0), ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
    odd = ctypes.c_void_p((1 << 20) + 2)

    def norm(bwd, ptr=fake, weight=fake, rope=fake, positions=fake, rows=4, hq=4, hkv=2, D=64, rot=64, most=9,
             eps=1e-6, strides=None, ws=fake, size=1 << 30, dw=fake):
        n = 12 if bwd else 8
        strides = None if strides is None else (ctypes.c_int64 * n)(*(strides * n)[:n])
        head = [ptr] * (6 if bwd else 4) + [weight] * 2 + [0] + ([dw] * 2 if bwd else [])
        tail = [ws, size, nul] if bwd else [nul]
        f = L.dash_qk_norm_rope_bwd if bwd else L.dash_qk_norm_rope
        return f(*head, rope, positions, rows, hq, hkv, D, rot, most, 0, eps, strides, *tail)

    for bwd in (False, True):
        for code, word, kw in ((2, "head dim", {"D": 96}), (1, "heads", {"hkv": 0}), (1, "heads", {"hq": -1}),
                               (2, "65535", {"hq": 70000}), (1, "multiple of 8", {"rot": 12}),
                               (1, "multiple of 8", {"rot": 72}), (1, "multiple of 8", {"rot": 0}),
                               (1, "positions", {"most": 0}), (1, "rows", {"rows": -1}), (2, "rows", {"rows": 2**31}),
                               (1, "eps", {"eps": -1.0}), (1, "eps", {"eps": float("nan")}),
                               (1, "eps", {"eps": float("inf")}), (1, "null", {"ptr": nul}), (1, "null", {"weight": nul}),
                               (1, "aligned", {"weight": odd}), (1, "null", {"rope": nul}), (1, "aligned", {"ptr": odd}),
                               (1, "null", {"positions": nul}), (1, "aligned", {"positions": odd}),
                               (1, "strides", {"strides": [256, 60]}), (1, "overlap", {"strides": [64, 64]}),
                               (2, "2^38", {"strides": [1 << 60, 64]})):
            assert norm(bwd, **kw) == code, (bwd, kw)
            assert word in dash.dash_last_error(), (bwd, kw, dash.dash_last_error())
        if not bwd:
            assert norm(bwd, rows=0, ptr=nul, positions=nul) == 0
    for kw in ({"ws": nul}, {"ws": odd}, {"size": 100}):
        assert norm(True, rows=100, **kw) == 1 and "workspace" in dash.dash_last_error()
    assert norm(True, dw=nul) == 1 and "dq_weight" in dash.dash_last_error()
    need = dash.dash_norm_rope_workspace
    assert {need(-1, 4, 2, 64), need(2**31, 4, 2, 64), need(5, 4, 2, 80), need(5, 0, 2, 64), need(5, 4, 70000, 64)} == {-1}
    # a few rows need few parts, many rows a bounded number
    assert 0 == need(0, 4, 2, 64) < need(1, 4, 2, 64) < need(100, 4, 2, 64) < need(100, 400, 2, 64)
    assert need(10**6, 8, 2, 128) == need(10**9, 8, 2, 128) < 1 << 20


def test_binding_refuses_wrong_tensors():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dash.qk_norm_rope(q, q, q[0, 0], q[0, 0], torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32))
