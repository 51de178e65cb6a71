"""Packed attention and paged cache, what needs no GPU: the task tables, the
refusals, and the plain 64-bit forms the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import deterministic_attention_backward_fa_gb300 as dash

import _packed as R


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


LENS = [[1], [128], [129, 1, 127], [4096], [0, 5, 0, 300, 0], [], [0], [1000, 3, 257], [4000], list(range(1, 40))]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (6, 2), (8, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_items_cover_every_tile_once(lens, hq, hkv, causal):
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    tiles = [(s, i) for s, n in enumerate(lens) for i in range(-(-n // 128))]
    first = {s: tiles.index((s, 0)) for s, n in enumerate(lens) if n}
    rows = lambda s, i: min(128, lens[s] - 128 * i)
    for P in (1, 7, 152):
        got = {}
        for kernel in range(3):
            items, off = dash.dash_build_packed_items(lens, hq, hkv, causal, kernel, P)
            assert off[0] == 0 and off[-1] == len(items) and (np.diff(off) >= 0).all() and len(off) - 1 <= P
            got[kernel] = items.tolist()
        n_of = {s: -(-lens[s] // 128) for s in range(len(lens))}
        q_tiles = sorted((starts[s] + 128 * i, rows(s, i), i + 1 if causal else n_of[s], h, 128 * i, starts[s], lens[s])
                         for s, i in tiles for h in range(hq))
        fwd = []
        for it in got[0]:
            halves = [h for h in range(2) if it[4 + h]]
            assert halves in ([0], [0, 1])
            for h in halves:
                assert it[6 + h] // (hq // hkv) == it[12]
                fwd.append((it[h], it[2 + h], it[4 + h], it[6 + h], it[8 + h], it[10], it[11]))
        assert sorted(fwd) == q_tiles
        assert sorted(tuple(it[:7]) for it in got[1]) == q_tiles
        assert all(it[7] == next(first[s] + i for s, i in tiles if starts[s] + 128 * i == it[0]) for it in got[1])
        # the parts of every KV tile cover its Q tiles once, and parts have places of their own
        parts, places = {}, []
        for it in got[2]:
            parts.setdefault(tuple(it[:8]), []).append((it[8], it[9], it[10]))
        assert set(parts) == {(starts[s] + 128 * i, rows(s, i), i, h, n_of[s], starts[s], lens[s], first[s])
                              for s, i in tiles for h in range(hkv)}
        for key, v in parts.items():
            v.sort()
            assert v[0][0] == 0 and v[-1][1] == (hq // hkv) * (key[4] - (key[2] if causal else 0))
            assert all(a[1] == b[0] for a, b in zip(v, v[1:])) and all(a < b for a, b, _ in v)
            if len(v) == 1:
                assert v[0][2] == -1
            else:  # in their order, side by side
                assert [x[2] for x in v] == list(range(v[0][2], v[0][2] + len(v)))
                places += [x[2] for x in v]
        assert sorted(places) == list(range(len(places)))


def test_item_refusals():
    for args, word in ((([-1], 4, 2, True, 0, 8), "negative"), (([5], 4, 3, True, 0, 8), "multiple"),
                       (([5], 4, 0, True, 1, 8), "multiple"), (([5], 4, 2, True, 2, 0), "out of range"),
                       (([5], 4, 2, True, 3, 8), "out of range"),
                       (([2**31 - 1, 2**31 - 1], 1, 1, True, 0, 8), "rows")):
        with pytest.raises(dash.DashError, match=word) as ei:
            dash.dash_build_packed_items(*args)
        assert ei.value.code == 1
    with pytest.raises(dash.DashError, match="32-bit") as ei:
        dash.dash_build_packed_items([1 << 24], 65024, 8, True, 1, 152)
    assert ei.value.code == 2


def _nul(n):
    return [ctypes.c_void_p(0)] * n


def test_refusals_before_any_device_call():
    L, nul = dash.lib(), ctypes.c_void_p(0)
    fake = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
    out = ctypes.c_void_p()
    lens = (ctypes.c_int32 * 2)(5, -7)
    assert L.dash_packed_plan_create(lens, 2, 4, 2, 64, 1, 0, ctypes.byref(out)) == 1
    assert "negative" in dash.dash_last_error()
    assert L.dash_packed_plan_create(lens, 1, 4, 2, 96, 1, 0, ctypes.byref(out)) == 2
    assert L.dash_packed_plan_create(lens, 1, 4, 3, 64, 1, 0, ctypes.byref(out)) == 1
    assert L.dash_packed_plan_create(None, 1, 4, 2, 64, 1, 0, ctypes.byref(out)) == 1
    assert L.dash_packed_plan_create(lens, 1, 4, 2, 64, 1, 0, None) == 1
    assert L.dash_attn_packed_fwd(nul, *_nul(5), 5, None, 0.1, nul) == 1 and "plan" in dash.dash_last_error()
    assert L.dash_attn_packed_fwd(nul, *_nul(5), 5, None, -1.0, nul) == 1 and "scale" in dash.dash_last_error()
    assert L.dash_packed_bwd_workspace(nul) == -1

    def decode(ptr=fake, B=2, hq=4, hkv=2, D=64, pages=8, page=16, width=4, strides=None, scale=0.1, ws=None, n=0):
        return L.dash_attn_decode(ptr, ptr, ptr, ptr, ptr, ptr, nul, B, hq, hkv, D, pages, page, width, strides,
                                  scale, ws, n, nul)

    bad = lambda *v: (ctypes.c_int64 * 11)(*v)
    good = (256, 64, 256, 64, 2048, 128, 64, 2048, 128, 64, 4)
    for code, word, kw in ((2, "head dim", {"D": 96}), (1, "multiple", {"hq": 5}), (1, "scale", {"scale": 0.0}),
                           (1, "null pointer", {"ptr": nul}), (1, "aligned", {"ptr": ctypes.c_void_p((1 << 20) + 8)}),
                           (1, "pages", {"pages": 0}), (2, "2^31", {"width": 1 << 28}), (2, "65535", {"B": 70000}),
                           (1, "workspace", {"width": 1024}), (1, ">= 0", {"B": -1}),
                           (1, "strides", {"strides": bad(255, *good[1:])}),
                           (1, "overlap", {"strides": bad(*good[:4], 2048, 128, 128, *good[7:])}),
                           (1, "overlap", {"strides": bad(64, 64, *good[2:])}),
                           (1, "table rows", {"strides": bad(*good[:10], 3)})):
        assert decode(**kw) == code, kw
        assert word in dash.dash_last_error(), (kw, dash.dash_last_error())
    assert decode(B=0) == 0
    copy = lambda s, d, pages=8: L.dash_cache_copy(fake, fake, (ctypes.c_int32 * len(s))(*s),
                                                   (ctypes.c_int32 * len(d))(*d), len(s), 2, 64, pages, 16, None, nul)
    for s, d, word in (([0, 1], [2, 2], "twice"), ([0, 2], [2, 3], "source and a destination"),
                       ([3], [3], "source and a destination"), ([8], [1], "outside"), ([-1], [1], "outside"),
                       ([1], [8], "outside"), ([1], [-2], "outside")):
        assert copy(s, d) == 1 and word in dash.dash_last_error()
    write = lambda n=4, B=2, D=64, page=16: L.dash_cache_write(*[fake] * 7, n, B, 2, D, 8, page, 4, None, nul)
    assert write(n=-1) == 1 and write(D=80) == 2 and write(page=0) == 1 and write(n=0) == 0 and write(B=0) == 0


def test_refusals_of_words_and_sizes_beyond_32_bits():
    L, nul, fake, odd = dash.lib(), ctypes.c_void_p(0), ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)

    def decode(table=fake, lengths=fake, lse=nul, hkv=2, page=16, width=4, strides=None):
        return L.dash_attn_decode(fake, fake, fake, table, lengths, fake, lse, 2, 4, hkv, 64, 8, page, width, strides,
                                  0.1, fake, 1 << 40, nul)

    def write(table=fake, starts=fake, cu=fake):
        return L.dash_cache_write(*[fake] * 4, table, starts, cu, 4, 2, 2, 64, 8, 16, 4, None, nul)

    for call, name in ((decode, "lengths"), (decode, "table"), (decode, "lse"), (write, "table"), (write, "starts"),
                       (write, "cu")):
        assert call(**{name: odd}) == 1 and "aligned" in dash.dash_last_error()
        if name != "lse":
            assert call(**{name: nul}) == 1 and "null" in dash.dash_last_error()
    big = 1 << 60
    wide = (ctypes.c_int64 * 11)(big, 64, 256, 64, 2048, 128, 64, 2048, 128, 64, 4)
    assert decode(strides=wide) == 2 and "2^38" in dash.dash_last_error()
    wide = (ctypes.c_int64 * 11)(256, 64, 64, big, 2048, 128, 64, 2048, 128, 64, 4)
    assert decode(strides=wide) == 2 and "2^38" in dash.dash_last_error()
    # pages of 2^30 vectors of 16 bytes, tables of nearly 2^31 tokens
    assert decode(page=1 << 26) == 2 and "pages" in dash.dash_last_error()
    top = (2**31 - 1 - 2**26) // 16
    assert decode(width=top + 1) == 2 and "tokens" in dash.dash_last_error()
    assert dash.dash_decode_workspace(2, 4, 64, 16, top) > 0 > dash.dash_decode_workspace(2, 4, 64, 16, top + 1)
    assert L.dash_cache_copy(fake, fake, (ctypes.c_int32 * 1)(0), (ctypes.c_int32 * 1)(1), 1, 2, 64, 8, 1 << 26, None,
                             nul) == 2


def test_decode_workspace_holds_every_length_a_table_has_room_for():
    # longer splits past a limit make fewer of them: a table just past it still has room for sequences at it
    for page in (1, 16):
        most = 0
        for pages in sorted({max(1, (1 << n) // page + d) for n in range(6, 20) for d in (-1, 0, 1, 2, 40)}):
            need = dash.dash_decode_workspace(2, 8, 64, page, pages)
            assert need >= most
            most = need


def test_binding_refuses_wrong_tensors():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dash._rows("q", q, 2, 64, None, None)
    with pytest.raises(ValueError, match="CUDA bfloat16"):
        dash.cache_copy(torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 4, 64), [0], [1])
    with pytest.raises(ValueError, match="32 bits"):
        dash.dash_packed_plan_create([2**40], 4, 2, 64, True, False)


@pytest.mark.parametrize("causal", [True, False])
def test_plain_backward_against_differences(causal):
    # the 64-bit backward that the GPU tests compare with, against central differences of the 64-bit forward
    lens, hq, hkv, D, scale, h = [5, 1, 9], 4, 2, 8, 0.3, 1e-5
    g = torch.Generator().manual_seed(3)
    q, do = (torch.randn(15, hq, D, generator=g, dtype=R.F64) for _ in range(2))
    k, v = (torch.randn(15, hkv, D, generator=g, dtype=R.F64) for _ in range(2))
    loss = lambda a, b, c: (R.forward(lens, a, b, c, causal, scale)[0] * do).sum()
    o, lse, _ = R.forward(lens, q, k, v, causal, scale)
    grads, _ = R.backward(lens, q, k, v, o, do, lse, causal, scale)
    for i in range(3):
        d = torch.randn([q, k, v][i].shape, generator=g, dtype=R.F64)
        args = lambda s: [t + s * h * d if j == i else t for j, t in enumerate((q, k, v))]
        diff = (loss(*args(1)) - loss(*args(-1))) / (2 * h)
        assert abs(diff - (grads[i] * d).sum()) <= 1e-7 * (1 + abs(diff))


def test_refusals_of_a_spin_limit():
    L, nul = dash.lib(), ctypes.c_void_p(0)
    assert L.dash_packed_plan_spin_limit(nul, 0) == 1 and "null plan" in dash.dash_last_error()


def test_no_exception_leaves_a_c_entry(tmp_path):
    # every allocation of the library fails while a flag is set: calls return a code and a message
    import subprocess
    import sys
    (tmp_path / "f.cpp").write_text("""
#include <cstdlib>
#include <new>
extern "C" { int fail_new = 0; }
void *operator new(std::size_t n) {
  void *p = fail_new ? nullptr : std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }
""")
    so = str(tmp_path / "f.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-o", so, str(tmp_path / "f.cpp")], check=True)
    code = """
import ctypes, sys
new, L = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
flag = ctypes.c_int.in_dll(new, "fail_new")
L.dash_last_error.restype = ctypes.c_char_p
nul, n, F, I64 = ctypes.c_void_p(0), ctypes.c_longlong(), ctypes.c_float, ctypes.c_longlong
lens, out = (ctypes.c_int32 * 2)(300, 40), ctypes.c_void_p()
flag.value = 1
calls = [(1, lambda: L.dash_attn_decode(*[nul] * 7, 1, 4, 2, 64, 8, 16, 4, nul, F(-1.0), nul, I64(0), nul)),
         (1, lambda: L.dash_cache_write(*[nul] * 7, I64(4), 1, 2, 64, 8, 0, 4, nul, nul)),
         (1, lambda: L.dash_cache_copy(*[nul] * 4, -1, 2, 64, 8, 16, nul, nul)),
         (5, lambda: L.dash_cache_copy(*[ctypes.c_void_p(1 << 20)] * 2, lens, lens, 1, 2, 64, 400, 16, nul, nul)),
         (1, lambda: L.dash_attn_packed_fwd(*[nul] * 6, I64(5), nul, F(-1.0), nul)),
         (1, lambda: L.dash_attn_packed_bwd(*[nul] * 10, I64(5), nul, F(-1.0), nul, I64(0), nul)),
         (5, lambda: L.dash_packed_plan_create(lens, 2, 4, 2, 64, 1, 1, ctypes.byref(out))),
         (5, lambda: L.dash_build_packed_items(lens, 2, 4, 2, 1, 0, 8, nul, nul, nul, ctypes.byref(n))),
         (1, lambda: L.dash_attn_fwd(*[nul] * 5, 1, 1, 128, 64, 1, F(-1.0), nul))]
for want, call in calls:
    assert call() == want, (want, L.dash_last_error())
    assert len(L.dash_last_error()) > 10
flag.value = 0
"""
    import os
    r = subprocess.run([sys.executable, "-c", code, so, dash.library_path()], capture_output=True, text=True,
                       env=dict(os.environ, LD_PRELOAD=so), timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
