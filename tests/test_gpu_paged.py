"""The paged cache on the GPU: decode attention, writing and copying pages,
against 64-bit plain forms and torch's own indexing."""
import math

import pytest
import torch

import deterministic_attention_backward_fa_gb300 as dash

import _packed as R

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(lens, hkv, D, page, seed=1, spare=3, width=None):
    """Pages in random order; page table entries behind a sequence's last page point nowhere."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), width or max(need + [1])), 2**31 - 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return R.normal(seed, n_pages, page, hkv, D), R.normal(seed + 1, n_pages, page, hkv, D), table


def check(q, kp, vp, table, lengths, scale, o, lse):
    ro, rl, mag = R.decode(q, kp, vp, table, lengths, scale)
    R.within("O", o, ro, mag)
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), none)
    assert (lse.double() - rl)[~none].abs().max() <= 1e-4 if (~none).any() else True


CASES = [([1], 1, 1, 64, 16), ([0, 5, 0], 4, 2, 128, 16), ([64, 63, 65, 256, 257, 255], 8, 2, 128, 16),
         ([300, 1000, 17], 6, 2, 64, 24), ([2000, 1], 32, 1, 128, 64), ([777] * 3, 20, 1, 64, 1),
         ([40000, 3], 4, 4, 128, 128), ([33000, 65], 3, 1, 64, 7), (list(range(0, 900, 5)), 2, 1, 64, 32)]


@pytest.mark.parametrize("lens,hq,hkv,D,page", CASES, ids=lambda x: str(x)[:40])
def test_decode(lens, hq, hkv, D, page):
    kp, vp, table = cache(lens, hkv, D, page)
    # whatever stands behind a sequence's last token is not read into its result
    for b, n in enumerate(lens):
        if n % page:
            last = table[b, n // page].long()
            kp[last, n % page:], vp[last, n % page:] = NAN, NAN
    q = R.normal(9, len(lens), hq, D)
    o, lse = dash.attn_decode(q, kp, vp, table, i32(lens))
    dash.dash_sync_status()
    check(q, kp, vp, table, lens, 1 / math.sqrt(D), o, lse)
    o2, lse2 = dash.attn_decode(q, kp, vp, table, i32(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_does_not_depend_on_the_batch():
    # the same bits alone, in a batch, and under a wider page table
    lens, hq, hkv, D, page = [5000, 130, 20000, 1], 8, 2, 128, 16
    kp, vp, table = cache(lens, hkv, D, page, width=4000)
    q = R.normal(5, 4, hq, D)
    o, lse = dash.attn_decode(q, kp, vp, table, i32(lens))
    for b, n in enumerate(lens):
        w = -(-n // page)
        ob, lb = dash.attn_decode(q[b:b + 1], kp, vp, table[b:b + 1, :w].contiguous(), i32([n]))
        assert torch.equal(o[b], ob[0]) and torch.equal(lse[b], lb[0])


@pytest.mark.parametrize("at,width", [(4096, 4200), (8192, 8300), (65536, 65600)])
def test_decode_beside_the_lengths_where_splits_grow(at, width):
    # shorter sequences may have more splits than the longest that the table has room for
    hq, hkv, D, page = 4, 2, 64, 4
    lens = [at, width, at - 1, at + 1, 5] * 3
    kp, vp, table = cache(lens, hkv, D, page, width=-(-width // page))
    q = R.normal(5, len(lens), hq, D)
    o, lse = dash.attn_decode(q, kp, vp, table, i32(lens))
    dash.dash_sync_status()
    check(q, kp, vp, table, lens, 1 / math.sqrt(D), o, lse)
    one, l1 = dash.attn_decode(q[:1], kp, vp, table[:1], i32(lens[:1]))
    assert torch.equal(o[:1], one) and torch.equal(lse[:1], l1)


@pytest.mark.parametrize("hq,hkv,D,page,width", [(16, 4, 128, 16, 44), (8, 1, 64, 16, 64), (20, 1, 128, 7, 90),
                                                 (2, 2, 64, 1, 2000), (16, 16, 128, 64, 30), (6, 3, 64, 32, 512)])
def test_decode_small_calls_join_with_the_same_bits(hq, hkv, D, page, width):
    # one sequence at a time (its splits are joined in the call's only kernel) and in a batch (by a second one)
    cap = page * width
    lens = sorted({0, 1, 255, 256, 257, 512, 513, 777, cap // 2 + 1, cap - 1, cap} & set(range(cap + 1))) * 6
    kp, vp, table = cache(lens, hkv, D, page, width=width)
    q = R.normal(15, len(lens), hq, D)
    o, lse = dash.attn_decode(q, kp, vp, table, i32(lens))
    dash.dash_sync_status()
    check(q, kp, vp, table, lens, 1 / math.sqrt(D), o, lse)
    assert dash.dash_decode_workspace(len(lens), hq, D, page, width) > 0
    for b, n in enumerate(lens):
        ob, lb = dash.attn_decode(q[b:b + 1], kp, vp, table[b:b + 1], i32([n]))
        assert torch.equal(o[b], ob[0]) and torch.equal(lse[b], lb[0]), n
    # captured, its length read when it is replayed
    if dash.dash_decode_workspace(1, hq, D, page, width) == 0:
        length, graph = i32([1]), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            og, lg = dash.attn_decode(q[-1:], kp, vp, table[-1:], length)
        length.copy_(i32(lens[-1:]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(og[0], o[-1]) and torch.equal(lg[0], lse[-1])
    dash.dash_sync_status()


def test_decode_strides_and_lengths_out_of_range():
    lens, hq, hkv, D, page = [100, 700, 31], 8, 2, 64, 16
    kp, vp, table = cache(lens, hkv, D, page)
    want = dash.attn_decode(R.normal(6, 3, hq, D), kp, vp, table, i32(lens))
    # a head-first cache, K and V side by side in one tensor, Q a part of a fused row, a table inside a larger one
    both = torch.full((kp.shape[0], 2, hkv, page, D), NAN, dtype=kp.dtype, device="cuda")
    k2, v2 = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    k2.copy_(kp)
    v2.copy_(vp)
    fused = torch.full((3, hq + 4, D), NAN, dtype=kp.dtype, device="cuda")
    q2 = fused[:, 2:2 + hq]
    q2.copy_(R.normal(6, 3, hq, D))
    t2 = torch.full((3, table.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    t2[:, :table.shape[1]] = table
    got = dash.attn_decode(q2, k2, v2, t2[:, :table.shape[1]], i32(lens))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # lengths are clipped to the table
    small, full = table[:, :2].contiguous(), i32([32, 32, 31])
    a = dash.attn_decode(q2, kp, vp, small, i32([-4, 10**9, 31]))
    b = dash.attn_decode(q2, kp, vp, small, full)
    dash.dash_sync_status()
    assert torch.equal(a[0][1:], b[0][1:]) and not a[0][0].any() and (a[1][0] == float("-inf")).all()


def test_bad_pages_are_reported_and_left_out():
    lens, hq, hkv, D, page = [70, 40], 4, 2, 128, 16
    kp, vp, table = cache(lens, hkv, D, page)
    q = R.normal(7, 2, hq, D)
    for bad in (-1, kp.shape[0], 2**31 - 1):
        t = table.clone()
        t[0, 1] = bad
        o, lse = dash.attn_decode(q, kp, vp, t, i32(lens))
        with pytest.raises(dash.DashError, match="outside the cache"):
            dash.dash_sync_status()
        dash.dash_sync_status()  # cleared
        check(q, kp, vp, t, lens, 1 / math.sqrt(D), o, lse)


def test_masked_out_scores_and_large_offsets():
    # scores of -inf (a K row of -inf against a positive Q) weigh nothing; a cache of more than 2^31 elements
    hq, hkv, D, page = 4, 4, 128, 64
    n_pages = (2**31 // (page * hkv * D)) + 40
    kp = torch.zeros(n_pages, page, hkv, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    pages = [n_pages - 1, 3, n_pages - 20, n_pages - 2]
    for i, p in enumerate(pages):
        kp[p], vp[p] = R.normal(100 + i, page, hkv, D), R.normal(200 + i, page, hkv, D)
    kp[pages[1], 5:9] = float("-inf")
    q = R.normal(8, 1, hq, D).abs()
    table = i32([pages])
    o, lse = dash.attn_decode(q, kp, vp, table, i32([250]))
    dash.dash_sync_status()
    check(q, kp, vp, table, [250], 1 / math.sqrt(D), o, lse)
    dash.cache_copy(kp, vp, [n_pages - 1, n_pages - 2], [0, n_pages - 5])
    assert torch.equal(kp[0], kp[-1]) and torch.equal(vp[-5], vp[-2])
    k1 = R.normal(300, 3, hkv, D)
    dash.cache_write(k1, k1, kp, vp, i32([[n_pages - 7]]), i32([61]), i32([0, 3]))
    dash.dash_sync_status()
    assert torch.equal(kp[-7, 61:], k1) and torch.equal(vp[-7, 61:], k1) and not kp[-7, :61].any()


@pytest.mark.parametrize("hkv,D,page", [(1, 64, 16), (8, 128, 16), (3, 64, 1), (2, 128, 7)])
def test_write(hkv, D, page):
    starts, news = [0, 5, 31, 0, 16], [1, 40, 0, 33, 16]
    lens = [a + b for a, b in zip(starts, news)]
    kp, vp, table = cache(lens, hkv, D, page, seed=3)
    cu = [sum(news[:i]) for i in range(len(news) + 1)]
    extra = 4  # tokens behind the last sequence
    fused = R.normal(4, cu[-1] + extra, 2 * hkv + 1, D)
    k, v = fused[:, 1:1 + hkv], fused[:, 1 + hkv:]
    wk, wv = kp.clone(), vp.clone()
    for b, n in enumerate(news):
        for i in range(n):
            pos = starts[b] + i
            wk[table[b, pos // page].long(), pos % page] = k[cu[b] + i]
            wv[table[b, pos // page].long(), pos % page] = v[cu[b] + i]
    dash.cache_write(k, v, kp, vp, table, i32(starts), i32(cu))
    dash.dash_sync_status()
    assert torch.equal(kp, wk) and torch.equal(vp, wv)


def test_write_outside_the_cache_is_reported():
    kp, vp, table = cache([32, 32], 2, 64, 16)
    k = R.normal(2, 4, 2, 64)
    table[1, 1] = -1
    for starts in ([0, 15], [0, 40], [0, -3]):
        wk = kp.clone()
        dash.cache_write(k, k, kp, vp, table, i32(starts), i32([0, 2, 4]))
        with pytest.raises(dash.DashError, match="outside the cache"):
            dash.dash_sync_status()
        wk[table[0, 0].long(), :2] = k[:2]
        for i in (2, 3):
            pos = starts[1] + i - 2
            if 0 <= pos < 16:
                wk[table[1, 0].long(), pos] = k[i]
        assert torch.equal(kp, wk)


@pytest.mark.parametrize("hkv,D,page,n", [(1, 64, 1, 5), (2, 128, 16, 64), (3, 64, 24, 65), (8, 128, 16, 3600)])
def test_copy(hkv, D, page, n):
    n_pages = 2 * n + 3
    kp, vp = R.normal(1, n_pages, page, hkv, D), R.normal(2, n_pages, page, hkv, D)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(5))
    src, dst = perm[:n], perm[n:2 * n]
    src[n // 2] = src[0]  # a page may be copied to several
    wk, wv = kp.clone(), vp.clone()
    wk[dst], wv[dst] = kp[src], vp[src]
    hk, hv = kp.transpose(1, 2).contiguous().transpose(1, 2), vp.transpose(1, 2).contiguous().transpose(1, 2)
    dash.cache_copy(kp, vp, src, dst)
    dash.cache_copy(hk, hv, src.tolist(), dst.tolist())
    dash.cache_copy(kp, vp, [], [])
    dash.dash_sync_status()
    for got, want in ((kp, wk), (vp, wv), (hk, wk), (hv, wv)):
        assert torch.equal(got, want)


def test_refusals():
    kp, vp, table = cache([32], 2, 64, 16)
    q = R.normal(1, 1, 4, 64)
    n = i32([32])
    for bad in (lambda: dash.attn_decode(q.float(), kp, vp, table, n), lambda: dash.attn_decode(q, kp, vp[1:], table, n),
                lambda: dash.attn_decode(q, kp, vp, table.long(), n), lambda: dash.attn_decode(q, kp, vp, table, n.long()),
                lambda: dash.attn_decode(q, kp, vp, table, i32([1, 2])),
                lambda: dash.attn_decode(q, kp, vp, table.cpu(), n), lambda: dash.cache_copy(kp, vp, [0], [1, 2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dash.DashError, match="overlap|strides"):
        dash.attn_decode(q, kp[:, :, :1].expand(-1, -1, 2, -1), vp, table, n)
    with pytest.raises(dash.DashError, match="twice"):
        dash.cache_copy(kp, vp, [0, 1], [2, 2])


def test_prompt_cache_fork_and_decode_together():
    # two prompts go through the packed forward and into the cache, the first is forked (sharing its full pages,
    # copying its last one), and all three take new tokens: each decode equals the last row of a packed forward
    hq, hkv, D, page, lens = 8, 2, 128, 16, [150, 37]
    q, k, v = R.normal(1, 187, hq, D), R.normal(2, 187, hkv, D), R.normal(3, 187, hkv, D)
    kp, vp, table = cache([200, 200, 200], hkv, D, page, seed=4)
    dash.cache_write(k, v, kp, vp, table[:2], i32([0, 0]), i32([0, 150, 187]))
    own = table[2, 150 // page].clone()
    table[2, :150 // page] = table[0, :150 // page]
    dash.cache_copy(kp, vp, [int(table[0, 150 // page])], [int(own)])
    hist = [[t[:150] for t in (k, v)], [t[150:] for t in (k, v)], [t[:150] for t in (k, v)]]
    n = i32([150, 37, 150])
    cu = i32([0, 1, 2, 3])
    side = torch.cuda.Stream()
    for step in range(20):
        kn, vn, qn = (R.normal(50 + 3 * step + i, 3, h, D) for i, h in enumerate((hkv, hkv, hq)))
        hist = [[torch.cat([a, x[b:b + 1]]) for a, x in zip(hist[b], (kn, vn))] for b in range(3)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # tensors made on another stream
            dash.cache_write(kn, vn, kp, vp, table, n, cu)
            n = n + 1
            o, lse = dash.attn_decode(qn, kp, vp, table, n)
        side.synchronize()
    dash.dash_sync_status()
    for b in range(3):
        kk, vv = hist[b]
        x = torch.einsum("hgd,thd->hgt", qn[b].double().view(hkv, -1, D), kk.double()) / math.sqrt(D)
        p = torch.softmax(x, -1)
        R.within("O", o[b], torch.einsum("hgt,thd->hgd", p, vv.double()).reshape(hq, D),
                 torch.einsum("hgt,thd->hgd", p, vv.double().abs()).reshape(hq, D))
        rows = len(kk)
        qq = torch.zeros(rows, hq, D, dtype=q.dtype, device="cuda")
        qq[-1] = qn[b]
        of, _ = dash.attn_packed_fwd(dash.PackedPlan([rows], hq, hkv, D), qq, kk, vv)
        R.within("decode and forward", of[-1], torch.einsum("hgt,thd->hgd", p, vv.double()).reshape(hq, D),
                 torch.einsum("hgt,thd->hgd", p, vv.double().abs()).reshape(hq, D))


def test_decode_in_captured_graphs():
    lens, hq, hkv, D, page = [3000, 41], 8, 2, 128, 16
    kp, vp, table = cache(lens, hkv, D, page)
    q, n = R.normal(3, 2, hq, D), i32(lens)
    kn, cu = R.normal(4, 2, hkv, D), i32([0, 1, 2])
    want = dash.attn_decode(q, kp, vp, table, n)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dash.attn_decode(q, kp, vp, table, n))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    # a replay reads the lengths and pages as they are then
    w = torch.cuda.CUDAGraph()
    with torch.cuda.graph(w):
        dash.cache_write(kn, kn, kp, vp, table, n - 1, cu)
        n2 = dash.attn_decode(q, kp, vp, table, n)
    w.replay()
    torch.cuda.synchronize()
    dash.dash_sync_status()
    check(q, kp, vp, table, lens, 1 / math.sqrt(D), *n2)
    n -= 5
    w.replay()
    torch.cuda.synchronize()
    dash.dash_sync_status()
    check(q, kp, vp, table, [x - 5 for x in lens], 1 / math.sqrt(D), *n2)


def test_the_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, deterministic_attention_backward_fa_gb300 as dash
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kp = torch.randn(4, 16, 2, 64, device="cuda").bfloat16()
vp = torch.randn(4, 16, 2, 64, device="cuda").bfloat16()
q = torch.randn(1, 4, 64, device="cuda").bfloat16()
table, n = i([[2, 0, 1]]), i([40])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    dash.cache_copy(kp, vp, [2], [3])
    o, lse = dash.attn_decode(q, kp, vp, table, n)
g.replay()
torch.cuda.synchronize()
o2, lse2 = dash.attn_decode(q, kp, vp, table, n)
dash.dash_sync_status()
assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(kp[2], kp[3])
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("n", [200, 2000])
@pytest.mark.parametrize("form", ["one kernel", "two kernels", "scanned"])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_keeps_non_finite_scores(n, form, D):
    # one cached key of NaN, one that makes a score of +inf, a query of NaN, a value of NaN: the rows that attend them
    # are NaN, as softmax makes them, and every other row keeps its bits
    B, hq, hkv = {"one kernel": (1, 4, 2), "two kernels": (1, 128, 2), "scanned": (40, 8, 2)}[form]
    page, lens = 16, [n] * B
    kp, vp, table = cache(lens, hkv, D, page, width=2048 // page)
    assert (dash.dash_decode_workspace(B, hq, D, page, 2048 // page) == 0) == (form == "one kernel")
    q = R.normal(9, B, hq, D).abs() + 0.1
    o, lse = dash.attn_decode(q, kp, vp, table, i32(lens))
    check(q, kp, vp, table, lens, 1 / math.sqrt(D), o, lse)
    b, head, t = B // 2, 1, n // 2 + 3
    where = (table[b, t // page].long(), t % page, head)
    group = slice(head * hq // hkv, (head + 1) * hq // hkv)
    bad = torch.zeros(B, hq, dtype=torch.bool, device="cuda")
    bad[b, group] = True

    def others(o2, lse2, wrong):
        assert torch.equal(o2[~wrong], o[~wrong]) and torch.equal(lse2[~wrong], lse[~wrong])

    for x in (NAN, float("inf")):
        k2 = kp.clone()
        k2[where] = x
        o2, lse2 = dash.attn_decode(q, k2, vp, table, i32(lens))
        assert o2[bad].isnan().all() and not (lse2[bad] < float("inf")).any()
        others(o2, lse2, bad)
    q2, wrong = q.clone(), torch.zeros_like(bad)
    q2[b, hq - 1], wrong[b, hq - 1] = NAN, True
    o2, lse2 = dash.attn_decode(q2, kp, vp, table, i32(lens))
    assert o2[wrong].isnan().all() and lse2[wrong].isnan().all()
    others(o2, lse2, wrong)
    v2 = vp.clone()
    v2[where][5] = NAN
    o2, lse2 = dash.attn_decode(q, kp, v2, table, i32(lens))
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[b, group, 5] = True
    assert o2[hit].isnan().all() and torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2, lse)
    dash.dash_sync_status()


def test_writes_and_copies_on_a_stream_wait_for_the_current_one():
    # the rows and pages are still being made on the current stream when the calls are
    hkv, D, page, side = 2, 64, 16, torch.cuda.Stream()
    kp, vp, table = cache([40], hkv, D, page)
    new = R.normal(21, 40, 2 * hkv, D)
    k, v = torch.zeros_like(new[:, :hkv]), torch.zeros_like(new[:, hkv:])
    pages, free = table[0].tolist(), sorted(set(range(kp.shape[0])) - set(table[0].tolist()))
    starts, cu = i32([0]), i32([0, 40])
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # 10 ms
    k.copy_(new[:, :hkv])
    v.copy_(new[:, hkv:])
    dash.cache_write(k, v, kp, vp, table, starts, cu, stream=side)
    side.synchronize()
    at = lambda c: c[table[0].long()].flatten(0, 1)[:40]
    assert torch.equal(at(kp), new[:, :hkv]) and torch.equal(at(vp), new[:, hkv:])
    fresh = R.normal(22, 2, page, hkv, D)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    kp[pages[0]].copy_(fresh[0])
    vp[pages[1]].copy_(fresh[1])
    dash.cache_copy(kp, vp, pages[:2], free[:2], stream=side)
    side.synchronize()
    assert torch.equal(kp[free[0]], fresh[0]) and torch.equal(vp[free[1]], fresh[1])
    dash.dash_sync_status()


def test_inputs_dropped_after_a_call_on_a_stream():
    # The caller's inputs go out of scope while the stream that reads them is still busy with other work: their
    # memory must not be handed to the current stream's next tensors before.
    hq, hkv, D, page, n, side = 4, 2, 64, 16, 300, torch.cuda.Stream()
    q, k, v, do = (R.normal(30 + i, n, h, D) for i, h in enumerate((hq, hkv, hkv, hq)))
    plan = dash.PackedPlan([n], hq, hkv, D, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    kp, vp, table = cache([n], hkv, D, page)
    one, length, starts, cu = q[:1].clone(), i32([n]), i32([0]), i32([0, n])

    def run(call, *tensors, stream=None):
        """The call on copies of the tensors, whose memory is overwritten as soon as the allocator gives it out."""
        copies = [t.clone() for t in tensors]
        if stream:
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)  # 10 ms
        got = call(*copies, stream=stream)
        shapes = [(t.shape, t.dtype) for t in copies]
        del copies
        junk = [torch.empty(s, dtype=d, device="cuda").fill_(77) for s, d in shapes for _ in range(2)]
        torch.cuda.synchronize()
        del junk
        return got

    # the pages are copies too, and kept: what is written has to come from the inputs
    def write(k, v, table, starts, cu, stream):
        a, b = torch.zeros_like(kp), torch.zeros_like(vp)
        dash.cache_write(k, v, a, b, table, starts, cu, stream=stream)
        return a, b

    for call, tensors in ((lambda *t, stream: dash.attn_packed_fwd(plan, *t, stream=stream), (q, k, v)),
                          (lambda *t, stream: dash.attn_packed_bwd(plan, *t, stream=stream), (q, k, v, o, do, lse)),
                          (lambda *t, stream: dash.attn_decode(*t, stream=stream), (one, kp, vp, table, length)),
                          (write, (k, v, table, starts, cu))):
        want = run(call, *tensors)
        got = run(call, *tensors, stream=side)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    dash.dash_sync_status()


def test_a_failed_call_does_not_fail_the_next():
    # a plan asked for inside a capture is refused (it allocates); the calls after it are none the worse for it
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import os
import torch, deterministic_attention_backward_fa_gb300 as dash
rand = lambda *s: torch.randn(*s, device="cuda").bfloat16()
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kp, vp, q, table, n, o = rand(4, 16, 2, 64), rand(4, 16, 2, 64), rand(1, 4, 64), i([[2, 0, 1]]), i([40]), rand(1, 4, 64)
kn, starts, cu = rand(1, 2, 64), i([39]), i([0, 1])
plan = dash.PackedPlan([40], 4, 2, 64, backward=True)
x, xo, xl = [rand(40, h, 64) for h in (4, 2, 2, 4)], rand(40, 4, 64), torch.empty(4, 40, device="cuda")
g, ws = [torch.empty_like(t) for t in x[:3]], torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
y, yo, yl = [rand(1, 2, 128, 64) for _ in range(3)], rand(1, 2, 128, 64), torch.empty(1, 2, 128, device="cuda")
calls = [lambda: dash.dash_attn_decode(q, kp, vp, table, n, o, None, 0.125),
         lambda: dash.dash_cache_write(kn, kn, kp, vp, table, starts, cu),
         lambda: dash.dash_cache_copy(kp, vp, [2], [3]),
         lambda: dash.dash_attn_packed_fwd(plan, *x[:3], xo, xl, 0.125),
         lambda: dash.dash_attn_packed_bwd(plan, *x[:3], xo, x[3], xl, *g, 0.125, ws),
         lambda: dash.dash_attn_fwd(*y, yo, yl, True, 0.125)]
for call in calls:
    call()
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph.capture_begin()
        try:
            dash.PackedPlan([5], 4, 2, 64)
            os._exit(3)
        except dash.DashError as e:
            assert "capturing" in str(e), e
        try:
            graph.capture_end()
        except RuntimeError:
            pass
    call()
    torch.cuda.synchronize()
dash.dash_sync_status()
os._exit(0)  # without the destructors of captures that failed
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
