"""Decode of a batch that shares a prefix, on the GPU, against the 64-bit form of
the plain decode over each sequence's whole table (same bounds: P is rounded to
bf16 once, sums are 32-bit)."""
import math

import pytest
import torch

import deterministic_attention_backward_fa_gb300 as dash

import _packed as R

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(lens, prefix, hkv, D, page, seed=1, wide=False):
    """Pages in random order.  Whole pages of the prefix belong to all; the page that it fills in part is each
    sequence's own copy.  ``seen``: the table as the call sees it, whose entries for the prefix's whole pages are
    named by the first row alone.  ``wide``: a table of more than 4096 tokens, for which the prefix is attended apart
    from the tails however few the sequences are."""
    extra = 4096 // page + 1 if wide else 0
    full = prefix // page
    width = max([-(-n // page) for n in lens] + [-(-prefix // page)]) + extra
    need = [max(0, -(-max(n, prefix if b == 0 else 0) // page) - full) for b, n in enumerate(lens)]
    n_pages = full + sum(need) + 3
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), width), 2**31 - 1, dtype=torch.int32, device="cuda")
    table[:, :full] = order[:full]
    at = full
    for b, n in enumerate(need):
        table[b, full:full + n] = order[at:at + n]
        at += n
    kp, vp = R.normal(seed, n_pages, page, hkv, D), R.normal(seed + 1, n_pages, page, hkv, D)
    if prefix % page:
        for b, n in enumerate(lens):
            if b and n > full * page:
                for p in (kp, vp):
                    p[table[b, full].long(), :prefix % page] = p[table[0, full].long(), :prefix % page]
    seen = table.clone()
    seen[1:, :full] = -7
    return kp, vp, table, seen


def check(q, kp, vp, table, lens, o, lse):
    ro, rl, mag = R.decode(q, kp, vp, table, lens, 1 / math.sqrt(q.shape[2]))
    R.within("O", o, ro, mag)
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), none)
    assert (lse.double() - rl)[~none].abs().max() <= 1e-4 if (~none).any() else True


CASES = [(1, [0], 1, 1, 64, 16), (128, [0, 1], 4, 2, 128, 16), (127, [3, 0, 17], 4, 1, 64, 16),
         (129, [5], 8, 2, 128, 7), (700, [0, 300, 1000, 16], 16, 4, 128, 16), (1501, [0, 3, 17, 40], 16, 4, 128, 24),
         (257, [2] * 33, 4, 1, 64, 1), (5000, [9, 700] * 40, 8, 2, 128, 64), (3000, [1, 0, 5] * 50, 12, 2, 64, 16),
         (20000, [1, 2], 2, 1, 128, 16), (300, [4] * 70, 8, 1, 128, 32), (9000, [33, 0], 32, 32, 64, 128)]


both = pytest.mark.parametrize("wide", [False, True], ids=["", "wide"])


@both
@pytest.mark.parametrize("prefix,tails,hq,hkv,D,page", CASES, ids=lambda x: str(x)[:30])
def test_shared(prefix, tails, hq, hkv, D, page, wide):
    lens = [prefix + n for n in tails]
    kp, vp, table, seen = cache(lens, prefix, hkv, D, page, wide=wide)
    for b, n in enumerate(lens):  # whatever stands behind a sequence's last token is not read into its result
        if n % page:
            last = table[b, n // page].long()
            kp[last, n % page:], vp[last, n % page:] = NAN, NAN
    q = R.normal(9, len(lens), hq, D)
    o, lse = dash.attn_decode_shared(q, kp, vp, seen, i32(lens), prefix)
    dash.dash_sync_status()
    check(q, kp, vp, table, lens, o, lse)
    o2, lse2 = dash.attn_decode_shared(q, kp, vp, seen, i32(lens), prefix)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    dash.dash_sync_status()


@pytest.mark.parametrize("longest", [2000, 5000])
def test_sequences_that_end_inside_the_prefix(longest):
    prefix, hq, hkv, D, page = 900, 4, 2, 128, 16
    lens = [900, 0, 1, 127, 128, 129, 500, 899, 950, longest, 640]
    kp, vp, table, seen = cache(lens, prefix, hkv, D, page)
    q = R.normal(3, len(lens), hq, D)
    o, lse = dash.attn_decode_shared(q, kp, vp, seen, i32(lens), prefix)
    check(q, kp, vp, table, lens, o, lse)
    # out of range, clipped; lengths read when a captured call is replayed
    lengths, graph = i32([-5, 10**9] + lens[2:]), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = dash.attn_decode_shared(q, kp, vp, seen, lengths, prefix)
    cap = table.shape[1] * page
    for now in (lens, [cap if n == longest else min(n, 900) for n in lens]):
        lengths.copy_(i32(now))
        graph.replay()
        check(q, kp, vp, table, now, og, lg)
    dash.dash_sync_status()


def test_no_prefix_is_the_plain_decode_and_a_prefix_alone():
    lens, hq, hkv, D, page = [300, 40, 0], 8, 2, 64, 16
    kp, vp, table, _ = cache(lens, 0, hkv, D, page)
    q = R.normal(4, 3, hq, D)
    a, b = dash.attn_decode(q, kp, vp, table, i32(lens)), dash.attn_decode_shared(q, kp, vp, table, i32(lens), 0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # the table's whole width is the prefix
    kp, vp, table, seen = cache([320, 320], 320, hkv, D, page)
    o, lse = dash.attn_decode_shared(q[:2], kp, vp, seen, i32([320, 320]), 320)
    check(q[:2], kp, vp, table, [320, 320], o, lse)
    none = dash.attn_decode_shared(q[:0], kp, vp, seen[:0], i32([]), 320)
    assert none[0].shape == (0, hq, D) and none[1].shape == (0, hq)
    dash.dash_sync_status()


@both
def test_rows_whose_first_tiles_count_nothing(wide):
    # bad pages (reported), scores of -inf, then tokens that count, with scores far below zero
    prefix, hq, hkv, D, page = 128 * 7, 4, 1, 64, 64
    lens = [prefix + 10, prefix]
    kp, vp, table, seen = cache(lens, prefix, hkv, D, page, wide=wide)
    q = R.normal(5, 2, hq, D)
    bad = table.clone()
    bad[:, :3], bad[:, 9] = 10**6, -1
    o, lse = dash.attn_decode_shared(q, kp, vp, bad, i32(lens), prefix)
    with pytest.raises(dash.DashError, match="outside the cache"):
        dash.dash_sync_status()
    dash.dash_sync_status()  # cleared
    check(q, kp, vp, bad, lens, o, lse)
    q = q.abs() + 2.0
    kp[table[0, :4].long()] = -INF
    kp[table[0, 4:prefix // page].long()] = -kp[table[0, 4:prefix // page].long()].abs() - 20.0  # scores of some -500
    o, lse = dash.attn_decode_shared(q, kp, vp, seen, i32([prefix, prefix]), prefix)
    ro, rl, mag = R.decode(q, kp, vp, table, [prefix, prefix], 1 / math.sqrt(D))
    # 32-bit scores of this size are off by 2^-24 x 64 roundings of their terms' magnitudes: 2e-3 in a weight's
    # exponent at most, twice that in a weight over their sum
    assert (lse.double() - rl).abs().max() <= 2e-3 * 1.5
    err = (o.double() - ro).abs()
    assert (err <= R.bound(ro, mag) + 4e-3 * mag).all()
    kp[table[0, 4:prefix // page].long()] = -INF
    o, lse = dash.attn_decode_shared(q, kp, vp, seen, i32([prefix, prefix]), prefix)
    assert not o.any() and (lse == -INF).all()
    dash.dash_sync_status()


@both
def test_nan_and_infinite_scores_reach_their_rows_alone(wide):
    prefix, hq, hkv, D, page = 700, 4, 2, 128, 16
    lens = [prefix, prefix + 5, 200]
    kp, vp, table, seen = cache(lens, prefix, hkv, D, page, wide=wide)
    q = R.normal(6, 3, hq, D)
    good = dash.attn_decode_shared(q, kp, vp, seen, i32(lens), prefix)
    k1 = kp.clone()
    k1[table[0, 30].long(), 3, 1, 4] = NAN  # token 483 of head 1: the third sequence ends before it
    o, lse = dash.attn_decode_shared(q, k1, vp, seen, i32(lens), prefix)
    assert o[:2, 2:].isnan().all() and lse[:2, 2:].isnan().all()
    for a, b in ((o, good[0]), (lse, good[1])):
        assert torch.equal(a[:, :2], b[:, :2]) and torch.equal(a[2], b[2])
    for tok in (3, 600):
        k1 = kp.clone()
        k1[table[0, tok // page].long(), tok % page, 0, 0] = INF
        one = q.clone()
        one[:, 0, 0], one[:, 1, 0] = 1.0, -1.0  # +inf for head 0, -inf for head 1
        o, lse = dash.attn_decode_shared(one, k1, vp, seen, i32(lens), prefix)
        reached = [0, 1] if tok == 600 else [0, 1, 2]
        assert o[reached, 0].isnan().all() and lse[reached, 0].isnan().all() and o[:, 1:].isfinite().all()
    dash.dash_sync_status()


@both
def test_strides_streams_and_two_calls_at_once(wide):
    prefix, hq, hkv, D, page = 1000, 8, 2, 64, 16
    lens = [prefix + n for n in (0, 5, 300)]
    kp, vp, table, seen = cache(lens, prefix, hkv, D, page, wide=wide)
    q = R.normal(6, 3, hq, D)
    want = dash.attn_decode_shared(q, kp, vp, seen, i32(lens), prefix)
    kv = torch.full((kp.shape[0], 2, hkv, page, D), NAN, dtype=kp.dtype, device="cuda")
    k2, v2 = kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2)
    k2.copy_(kp)
    v2.copy_(vp)
    fused = torch.full((3, hq + 4, D), NAN, dtype=kp.dtype, device="cuda")
    q2 = fused[:, 2:2 + hq]
    q2.copy_(q)
    t2 = torch.full((3, table.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    t2[:, :table.shape[1]] = seen
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [dash.attn_decode_shared(q2, k2, v2, t2[:, :table.shape[1]], i32(lens), prefix, stream=s)
           for _ in range(3) for s in streams]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    # a workspace that starts at an odd multiple of 16 bytes; no lse
    o = torch.empty_like(q)
    need = dash.dash_decode_shared_workspace(3, hq, hkv, D, page, table.shape[1], prefix)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]
    dash.dash_attn_decode_shared(q, kp, vp, seen, i32(lens), prefix, o, None, 1 / math.sqrt(D), ws)
    assert torch.equal(o, want[0])
    dash.dash_sync_status()


@pytest.mark.parametrize("width", [4, 70])
def test_a_captured_first_call_and_large_offsets(width):
    # a cache of more than 2^31 elements
    hq, hkv, D, page = 4, 4, 128, 64
    n_pages = (2**31 // (page * hkv * D)) + 40
    kp = torch.zeros(n_pages, page, hkv, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    pages = [n_pages - 1, 3, n_pages - 20, n_pages - 2]
    for i, p in enumerate(pages):
        kp[p], vp[p] = R.normal(100 + i, page, hkv, D), R.normal(200 + i, page, hkv, D)
    q, table = R.normal(8, 2, hq, D), i32([pages + [0] * (width - 4)] * 2)
    o, lse = dash.attn_decode_shared(q, kp, vp, table, i32([250, 210]), 200)
    dash.dash_sync_status()
    check(q, kp, vp, table, [250, 210], o, lse)


def test_refusals():
    kp, vp, table, seen = cache([40, 40], 32, 2, 64, 16, wide=True)
    q, n = R.normal(1, 2, 4, 64), i32([40, 40])
    f = dash.attn_decode_shared
    for bad in (lambda: f(q.float(), kp, vp, table, n, 32), lambda: f(q, kp, vp, table, n, -1),
                lambda: f(q, kp, vp, table, n, 2**31), lambda: f(q, kp, vp, table, n.long(), 32),
                lambda: f(q, kp, vp[1:], table, n, 32)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dash.DashError, match="does not fit"):
        f(q, kp, vp, table, n, table.shape[1] * 16 + 1)
    with pytest.raises(dash.DashError, match="workspace"):
        dash.dash_attn_decode_shared(q, kp, vp, table, n, 32, torch.empty_like(q), None, 0.1)


@both
@pytest.mark.parametrize("bad", [NAN, INF, -INF], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 24)])
def test_values_that_a_sequence_does_not_attend_stay_out_of_its_rows(D, page, bad, wide):
    # tokens 250 and 699 of head 1 of V: behind the end of the shorter sequences, attended by the longer ones
    prefix, hq, hkv = 700, 4, 2
    lens = [prefix, 200, prefix + 5, 0, 250, 251, 249, 699, 1]
    kp, vp, table, seen = cache(lens, prefix, hkv, D, page, wide=wide)
    q = R.normal(6, len(lens), hq, D)
    v1 = vp.clone()
    for tok in (250, 699):
        for rows in (table[0, tok // page], *(table[b, tok // page] for b, n in enumerate(lens) if n > tok)):
            v1[rows.long(), tok % page, 1, 5:40:7] = bad
    o, lse = dash.attn_decode_shared(q, kp, v1, seen, i32(lens), prefix)
    ro, rl, mag = R.decode(q, kp, v1, table, lens, 1 / math.sqrt(D))
    assert torch.equal(o.double().isnan(), ro.isnan()) and torch.equal(o.double().isinf(), ro.isinf())
    some = rl.isfinite()
    assert (lse.double() - rl)[some].abs().max() <= 1e-4
    fine = ro.isfinite()
    assert fine[:, :2].all() and fine[1].all() and fine[[3, 4, 6, 8]].all() and not fine[[0, 2, 5, 7], 2:].all()
    R.within("O", torch.where(fine, o.double(), 0.0), torch.where(fine, ro, 0.0), torch.where(fine, mag, 0.0))
    assert not o[3].any() and lse[3].eq(-INF).all()
    dash.dash_sync_status()


@both
@pytest.mark.parametrize("D", [128, 64])
def test_pages_of_the_prefix_that_nobody_attends_may_hold_anything(D, wide):
    # every sequence ends inside the prefix; behind the longest, nothing was ever written
    prefix, hq, hkv, page = 1000, 8, 2, 16
    lens = [3, 0, 257, 128, 1, 300]
    kp, vp, table, seen = cache(lens, prefix, hkv, D, page, wide=wide)
    for pages in (kp, vp):
        flat = pages[table[0, :-(-prefix // page)].long()].flatten(0, 1)
        flat[max(lens):] = NAN
        pages[table[0, :-(-prefix // page)].long()] = flat.unflatten(0, (-1, page))
    q = R.normal(7, len(lens), hq, D)
    o, lse = dash.attn_decode_shared(q, kp, vp, seen, i32(lens), prefix)
    check(q, kp, vp, table[:1].expand(len(lens), -1), lens, o, lse)
    graph = torch.cuda.CUDAGraph()
    lengths = i32([0] * len(lens))
    with torch.cuda.graph(graph):
        og, lg = dash.attn_decode_shared(q, kp, vp, seen, lengths, prefix)
    for now in ([0] * len(lens), lens):
        lengths.copy_(i32(now))
        graph.replay()
        check(q, kp, vp, table[:1].expand(len(lens), -1), now, og, lg)
    assert torch.equal(og, o) and torch.equal(lg, lse)
    dash.dash_sync_status()


@pytest.mark.parametrize("what", ["samples", "batch", "batch of the 8-bit cache", "rows of the 8-bit cache", "norms"])
def test_the_first_call_of_a_process_may_be_captured(what):
    # one launch; the prefix, the tails and their join; items and their join; write, read and copy; two launches
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import sys
import torch, deterministic_attention_backward_fa_gb300 as dash
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
rand = lambda *s: torch.randn(*s, device="cuda").bfloat16()
what, D, page = sys.argv[1], 128, 16
q, kp, vp = rand(12, 8, D), rand(40, page, 2, D), rand(40, page, 2, D)
table = (torch.arange(12 * 1100, device="cuda").int() % 40).reshape(12, 1100)
table[:, :20] = torch.arange(20, device="cuda").int()
lens = i([300 + 29 * b for b in range(12)])
c8 = [rand(40, page, 2, D).to(torch.float8_e4m3fn) for _ in "kv"] + [torch.rand(40, page, 2, device="cuda") for _ in "kv"]
k, v = rand(25, 2, D), rand(25, 2, D)
x, w, rope, pos = rand(25, 8, D), rand(D), torch.rand(30, D, device="cuda"), torch.arange(25, device="cuda").int()

def call():
    if what == "samples":
        return dash.attn_decode_shared(q[:2], kp, vp, table[:2, :40], lens[:2], 310)
    if what == "batch":
        return dash.attn_decode_shared(q, kp, vp, table, lens, 310)
    if what == "batch of the 8-bit cache":
        return dash.attn_decode_fp8(q, *c8, table, lens)
    if what == "norms":
        return *dash.qk_norm_rope(x, k, w, w, rope, pos), *dash.qk_norm_rope_bwd(x, k, x, v, w, w, rope, pos)
    dash.cache_write_fp8(k, v, *c8, table[:2], lens[:2], i_cu)
    dash.cache_copy_fp8(*c8, [1, 2], [30, 31])
    return *dash.cache_read_fp8(*c8, table[:2], starts, i_cu, 25), *(t.view(torch.uint8).clone() for t in c8[:2])

i_cu, starts = i([0, 20, 25]), i([295, 300])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = call()
g.replay()
torch.cuda.synchronize()
again = call()
dash.dash_sync_status()
assert all(torch.equal(a, b) for a, b in zip(out, again))
assert all(t.float().abs().sum() > 0 for t in out)
"""
    r = subprocess.run([sys.executable, "-c", code, what], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
