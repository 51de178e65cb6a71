"""The 8-bit paged cache, what needs no GPU: refusals and the plain form's own quantisation."""
import ctypes
import os
import subprocess

import pytest
import torch

import deterministic_attention_backward_fa_gb300 as dash

import _cache8 as R


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_plain_quantisation():
    x = torch.zeros(8, 64, dtype=torch.float64)
    x[1, 0], x[2, 0], x[3, 3], x[4, 0], x[4, 1] = 448.0, 450.0, -1e-40, 1.0, 17.0 / 16
    x[5, 0], x[6, 0], x[7] = float("nan"), float("inf"), torch.linspace(-3, 3, 64)
    codes, scale = R.quantise(x)
    # 448 fits, what is above it needs the next power of two; subnormal and zero rows have the smallest scale
    assert scale.tolist()[:5] == [2.0 ** -126, 1.0, 2.0, 2.0 ** -126, 2.0 ** -8]
    assert scale[5:7].isnan().all() and not codes[5:7].any()
    # the step from 256 to 512 is 32: 17/16 x 256 = 272 stands between 256 and 288, and 256 is the even one
    assert codes[1, 0] == 448 and codes[2, 0] == 224 and codes[4, 0] == 256 and codes[4, 1] == 256
    # (448 stays, 450 / 2 = 225 is nearest to 224, the step from 128 to 256 being 16)
    # every code is one that the type holds, and no other is nearer
    held = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    held = held[held.isfinite()]
    y = x[7] / scale[7]
    assert ((y[:, None] - held).abs().min(1).values == (y - codes[7]).abs()).all()
    assert torch.isin(codes, held).all()


def test_refusals_before_any_device_call():
    L, nul, fake, odd = dash.lib(), ctypes.c_void_p(0), ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)
    seventeen = lambda *v: (ctypes.c_int64 * 17)(*v)
    good = [256, 64, 256, 64] + [2048, 128, 64] * 2 + [32, 2, 1] * 2 + [4]

    def decode(q=fake, pages=fake, scales=fake, table=fake, lengths=fake, B=2, hq=4, hkv=2, D=64, n=8, page=16, width=4,
               strides=None, scale=0.1, ws=nul, size=0):
        return L.dash_attn_decode_fp8(q, pages, pages, scales, scales, table, lengths, fake, nul, B, hq, hkv, D, n, page,
                                      width, strides, scale, ws, size, nul)

    def rows(f, k=fake, pages=fake, scales=fake, table=fake, starts=fake, cu=fake, n=4, B=2, hkv=2, D=64, pages_n=8,
             page=16, width=4, strides=None):
        return f(k, k, pages, pages, scales, scales, table, starts, cu, n, B, hkv, D, pages_n, page, width, strides, nul)

    def put(i, v):
        out = list(good)
        out[i] = v
        return seventeen(*out)

    strided = ((1, "multiples of 16", put(4, 2056)), (1, "overlap", put(5, 64)), (1, "overlap", put(11, 1)),
               (1, "at least 1", put(12, 0)), (1, "v_scales", put(14, -2)), (1, "table rows", put(16, 3)))
    for code, word, kw in ((2, "head dim", {"D": 96}), (1, "multiple", {"hq": 5}), (1, "scale", {"scale": 0.0}),
                           (1, "null", {"q": nul}), (1, "null", {"pages": nul}), (1, "aligned", {"pages": odd}),
                           (1, "null", {"scales": nul}), (1, "aligned", {"scales": odd}), (1, "pages", {"n": 0}),
                           (1, "aligned", {"table": odd}), (1, "null", {"lengths": nul}), (2, "2^31", {"width": 1 << 28}),
                           (2, "65535", {"B": 70000}), (1, "workspace", {"width": 1024}), (1, ">= 0", {"B": -1}),
                           *((c, w, {"strides": s}) for c, w, s in strided)):
        assert decode(**kw) == code, kw
        assert word in dash.dash_last_error(), (kw, dash.dash_last_error())
    assert decode(B=0, q=nul) == 0
    for f in (L.dash_cache_write_fp8, L.dash_cache_read_fp8):
        for code, word, kw in ((2, "head dim", {"D": 96}), (1, "null", {"k": nul}), (1, "aligned", {"pages": odd}),
                               (1, "aligned", {"scales": odd}), (1, "null", {"starts": nul}), (1, "null", {"cu": nul}),
                               (1, "null", {"table": nul}), (1, "2^31", {"n": -1}), (1, "2^31", {"n": 2**31 - 1}),
                               (1, "tokens in a page", {"page": 0}), (2, "pages", {"page": 1 << 26}),
                               *((c, w, {"strides": s}) for c, w, s in strided)):
            assert rows(f, **kw) == code, kw
            assert word in dash.dash_last_error(), (kw, dash.dash_last_error())
        assert rows(f, n=0) == 0
    assert rows(L.dash_cache_write_fp8, B=0) == 0
    copy = lambda s, d, pages=fake: L.dash_cache_copy_fp8(pages, fake, fake, fake, (ctypes.c_int32 * len(s))(*s),
                                                          (ctypes.c_int32 * len(d))(*d), len(s), 2, 64, 8, 16, None, nul)
    for s, d, word in (([0, 1], [2, 2], "twice"), ([0, 2], [2, 3], "source and a destination"), ([8], [1], "outside"),
                       ([1], [-2], "outside")):
        assert copy(s, d) == 1 and word in dash.dash_last_error()
    assert copy([0], [1], odd) == 1 and "aligned" in dash.dash_last_error()
    assert copy([], []) == 0


def test_binding_refuses_wrong_tensors():
    pages, scales = torch.zeros(2, 3, 4, 64, dtype=torch.float8_e4m3fn), torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="CUDA float8"):
        dash.cache_copy_fp8(pages, pages, scales, scales, [0], [1])


def test_the_waits_on_the_way_out_have_one_limit(tmp_path):
    # ten barriers, of which some never complete, with a clock that the host drives
    (tmp_path / "d.cpp").write_text("""
#include "drain.h"
#include <cstdio>
int main() {
  for (int never = 0; never < 1024; ++never) {  // a bit for each that never completes
    unsigned long long clock = 5000, asked = 0;
    dash::drain_all(
        10, [&](int i) { ++asked; clock += 7; return !(never >> i & 1) && clock > 5000u + 40 * i; }, [&] { return clock; },
        1000);
    if (clock > 5000 + 1000 + 2 * 7) return std::printf("%d: took %llu\\n", never, clock - 5000), 1;
    if (!never && clock <= 5000 + 360) return std::printf("left too early\\n"), 1;
    if (!asked) return 1;
  }
  return 0;
}
""")
    exe = str(tmp_path / "d")
    src = os.path.join(os.path.dirname(dash.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", src, "-o", exe, str(tmp_path / "d.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
