"""Decode of a batch that shares a prefix, what needs no GPU: refusals and sizes."""
import ctypes

import pytest

import deterministic_attention_backward_fa_gb300 as dash


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_refusals_before_any_device_call():
    L, nul, fake = dash.lib(), ctypes.c_void_p(0), ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
    odd = ctypes.c_void_p((1 << 20) + 2)

    def call(ptr=fake, table=fake, lengths=fake, prefix=20, B=2, hq=4, hkv=2, D=64, n=8, page=16, width=4, strides=None,
             scale=0.1, ws=fake, size=1 << 30):
        return L.dash_attn_decode_shared(ptr, ptr, ptr, table, lengths, prefix, ptr, nul, B, hq, hkv, D, n, page, width,
                                         strides, scale, ws, size, nul)

    put = lambda i, v: (ctypes.c_int64 * 11)(*[v if j == i else x for j, x in
                                              enumerate([256, 64, 256, 64] + [2048, 128, 64] * 2 + [4])])
    for prefix in (20, 0):
        for code, word, kw in ((2, "head dim", {"D": 96}), (1, "multiple", {"hq": 5}), (1, "scale", {"scale": -1.0}),
                               (1, "null", {"ptr": nul}), (1, "aligned", {"ptr": odd}), (1, "pages", {"n": 0}),
                               (1, "aligned", {"table": odd}), (1, "null", {"lengths": nul}),
                               (2, "2^31", {"width": 1 << 28}), (2, "65535", {"B": 70000}),
                               (1, "strides", {"strides": put(0, 252)}), (1, "overlap", {"strides": put(5, 64)}),
                               (1, "table rows", {"strides": put(10, 3)}), (1, ">= 0", {"B": -1})):
            assert call(prefix=prefix, **kw) == code, kw
            assert word in dash.dash_last_error(), (kw, dash.dash_last_error())
        assert call(prefix=prefix, B=0, ptr=nul) == 0
    for prefix in (-1, 65, 2**31 - 1):
        assert call(prefix=prefix) == 1 and "does not fit" in dash.dash_last_error()
    for kw in ({"ws": nul}, {"ws": odd}, {"size": 64}):
        assert call(width=300, **kw) == 1 and "workspace" in dash.dash_last_error()
    assert call(B=65000, hq=65000, hkv=1) == 2 and "rows on one" in dash.dash_last_error()
    for bad in ((2, 5, 2, 64, 16, 4, 20), (2, 4, 0, 64, 16, 4, 20), (2, 4, 2, 80, 16, 4, 20), (2, 4, 2, 64, 16, 4, 65),
                (2, 4, 2, 64, 16, 4, -1), (-1, 4, 2, 64, 16, 4, 20), (2, 4, 2, 64, 16, 1 << 28, 20)):
        assert dash.dash_decode_shared_workspace(*bad) == -1


def test_workspace_holds_the_parts_of_any_size():
    # a part is D sums, a maximum and a sum, in 32 bits; at most 64 of the prefix and 64 of a tail
    for B in (1, 7, 64, 1000):
        for hq, hkv in ((1, 1), (32, 8), (16, 1)):
            for prefix in (1, 127, 128, 129, 5000, 100000):
                need = dash.dash_decode_shared_workspace(B, hq, hkv, 128, 16, 7000, prefix)
                part = B * hq * (128 * 4 + 8)
                assert 2 * part <= need <= 128 * part + 256
    assert dash.dash_decode_shared_workspace(3, 8, 2, 64, 16, 7000, 0) == dash.dash_decode_workspace(3, 8, 64, 16, 7000)
