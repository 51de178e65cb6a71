"""The 8-bit paged cache on the GPU: writing, reading, copying, and decode
attention, against 64-bit plain forms."""
import math

import pytest
import torch

import deterministic_attention_backward_fa_gb300 as dash

import _cache8 as R
import _packed as P

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.view(torch.uint8) if t.dtype == FP8 else t.view(torch.int32)


def pages_of(lens, page, seed=1, spare=3, width=None):
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
    return table, n_pages


def cache(lens, hkv, D, page, seed=1, width=None, spread=0.0, heads_first=True):
    """A filled 8-bit cache; ``spread``: standard deviation of the rows' own scales, in powers of two."""
    table, n_pages = pages_of(lens, page, seed, width=width)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 10)
    out = []
    for _ in range(2):
        x = torch.randn(n_pages, page, hkv, D, generator=g, device="cuda", dtype=torch.float64)
        x = x * torch.exp2(spread * torch.randn(n_pages, page, hkv, 1, generator=g, device="cuda", dtype=torch.float64))
        codes, scale = R.quantise(x)
        scale = scale.float()
        if heads_first:
            scale = scale.transpose(1, 2).contiguous().transpose(1, 2)
        out.append((codes.to(FP8), scale))
    (kp, ks), (vp, vs) = out
    return kp, vp, ks, vs, table


def check(q, c, lengths, scale, o, lse, lse_tol=1e-4):
    kp, vp, ks, vs, table = c
    ro, rl, mag, top = R.decode(q, (kp, vp), (ks, vs), table, lengths, scale)
    R.within("O", o, ro, mag, top)
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), none)
    assert (lse.double() - rl)[~none].abs().max() <= lse_tol if (~none).any() else True


# ------------------------------------------------------------ write, read
@pytest.mark.parametrize("hkv,D,page", [(1, 64, 16), (8, 128, 16), (3, 64, 1), (5, 128, 7)])
def test_write_and_read(hkv, D, page):
    starts, news = [0, 5, 31, 0, 16], [1, 40, 0, 33, 16]
    lens = [a + b for a, b in zip(starts, news)]
    kp, vp, ks, vs, table = cache(lens, hkv, D, page, seed=3, heads_first=page != 7)
    cu = [sum(news[:i]) for i in range(len(news) + 1)]
    extra = 4  # tokens behind the last sequence
    fused = P.normal(4, cu[-1] + extra, 2 * hkv + 1, D) * torch.exp2(
        torch.randint(-20, 20, (cu[-1] + extra, 2 * hkv + 1, 1), device="cuda").float()).bfloat16()
    k, v = fused[:, 1:1 + hkv], fused[:, 1 + hkv:]
    want = []
    for x, pages, scales in ((k, kp, ks), (v, vp, vs)):
        codes, scale = R.quantise(x)
        wp, ws = bits(pages).clone(), scales.clone()
        for b, n in enumerate(news):
            for i in range(n):
                pos = starts[b] + i
                at = (table[b, pos // page].long(), pos % page)
                wp[at], ws[at] = bits(codes[cu[b] + i].to(FP8)), scale[cu[b] + i].float()
        want += [wp, ws]
    dash.cache_write_fp8(k, v, kp, vp, ks, vs, table, i32(starts), i32(cu))
    dash.dash_sync_status()
    for got, ref in zip((bits(kp), ks, bits(vp), vs), want):
        assert torch.equal(got, ref)
    # what was written reads back as code times scale, exactly; rows behind the last sequence are zero
    rk, rv = dash.cache_read_fp8(kp, vp, ks, vs, table, i32(starts), i32(cu), cu[-1] + extra)
    dash.dash_sync_status()
    for x, back in ((k, rk), (v, rv)):
        codes, scale = R.quantise(x[:cu[-1]])
        assert torch.equal(back[:cu[-1]].double(), codes * scale[..., None]) and not back[cu[-1]:].any()
        # within half a step of what went in: 2^-4 of a value, or 2^-10 of the scale below the normal codes
        err = (back[:cu[-1]].double() - x[:cu[-1]].double()).abs()
        assert (err <= torch.maximum(2.0 ** -4 * x[:cu[-1]].double().abs(), 2.0 ** -10 * scale[..., None])).all()
    # from the middle of the sequences on
    mid = [min(3, n) for n in lens]
    left = [n - m for n, m in zip(lens, mid)]
    cu2 = [sum(left[:i]) for i in range(len(left) + 1)]
    rk, _ = dash.cache_read_fp8(kp, vp, ks, vs, table, i32(mid), i32(cu2), cu2[-1])
    vals = R.values(kp, ks)
    for b, n in enumerate(left):
        t = torch.arange(mid[b], lens[b], device="cuda")
        assert torch.equal(rk[cu2[b]:cu2[b + 1]].double(), vals[table[b].long()[t // page], t % page].bfloat16().double())


def test_quantisation_of_every_magnitude():
    # one row for each exponent of bf16 and for mantissas beside the limit of 448 = 1.75 x 2^8; zero, NaN, infinities
    D = 64
    raw = torch.arange(0, 0x7f80, 0x10, dtype=torch.int16, device="cuda")
    edge = torch.tensor([e << 7 | m for e in range(255) for m in (0x5f, 0x60, 0x61, 0x7f)], dtype=torch.int16,
                        device="cuda")
    tops = torch.cat([raw, edge]).view(torch.bfloat16)
    x = P.normal(7, tops.numel(), 1, D).clamp(-1, 1) * tops[:, None, None] / 2
    x[:, 0, 5] = tops * torch.where(torch.arange(tops.numel(), device="cuda") % 2 == 0, 1, -1).bfloat16()
    bad = torch.zeros(4, 1, D, dtype=torch.bfloat16, device="cuda")
    bad[1, 0, 9], bad[2, 0, 0], bad[3, 0, 63] = NAN, INF, -INF
    x = torch.cat([x, bad])
    n = x.shape[0]
    kp, vp = (torch.zeros(1, n, 1, D, device="cuda").to(FP8) for _ in range(2))
    ks, vs = (torch.full((1, n, 1), 5.0, device="cuda") for _ in range(2))
    dash.cache_write_fp8(x, -x, kp, vp, ks, vs, i32([[0]]), i32([0]), i32([0, n]))
    codes, scale = R.quantise(x)
    assert torch.equal(kp[0].double(), codes) and torch.equal(vp[0].double(), -codes)
    assert torch.equal(ks[0].nan_to_num(7), scale.float().nan_to_num(7)) and torch.equal(vs.nan_to_num(7), ks.nan_to_num(7))
    rk, rv = dash.cache_read_fp8(kp, vp, ks, vs, i32([[0]]), i32([0]), i32([0, n]), n)
    assert torch.equal(rk[:-3].double(), (codes * scale[..., None]).bfloat16().double()[:-3])
    assert rk[-3:].isnan().all() and rv[-3:].isnan().all()


def test_write_and_read_outside_the_cache_are_reported():
    kp, vp, ks, vs, table = cache([32, 32], 2, 64, 16)
    k = P.normal(2, 4, 2, 64)
    codes, scale = R.quantise(k)
    table[1, 1] = -1
    for starts in ([0, 15], [0, 40], [0, -3]):
        wk = bits(kp).clone()
        dash.cache_write_fp8(k, k, kp, vp, ks, vs, table, i32(starts), i32([0, 2, 4]))
        with pytest.raises(dash.DashError, match="outside the cache"):
            dash.dash_sync_status()
        wk[table[0, 0].long(), :2] = bits(codes[:2].to(FP8))
        for i in (2, 3):
            pos = starts[1] + i - 2
            if 0 <= pos < 16:
                wk[table[1, 0].long(), pos] = bits(codes[i].to(FP8))
        assert torch.equal(bits(kp), wk)
        rk, rv = dash.cache_read_fp8(kp, vp, ks, vs, table, i32(starts), i32([0, 2, 4]), 4)
        with pytest.raises(dash.DashError, match="outside the cache"):
            dash.dash_sync_status()
        for i in range(4):
            pos = starts[i // 2] + i % 2
            inside = i < 2 or 0 <= pos < 16
            assert torch.equal(rk[i].double(), codes[i] * scale[i][:, None]) if inside else not rk[i].any()
    assert not dash.cache_read_fp8(kp, vp, ks, vs, table[:0], i32([]), i32([0]), 3)[0].any()
    dash.dash_sync_status()


@pytest.mark.parametrize("hkv,D,page,n", [(1, 64, 1, 5), (2, 128, 16, 64), (3, 64, 24, 65), (8, 128, 16, 3600)])
def test_copy(hkv, D, page, n):
    n_pages = 2 * n + 3
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    pages = [torch.randint(0, 256, (n_pages, page, hkv, D), generator=g, device="cuda", dtype=torch.uint8).view(FP8)
             for _ in range(2)]
    scales = [torch.rand(n_pages, page, hkv, generator=g, device="cuda") for _ in range(2)]
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(5))
    src, dst = perm[:n], perm[n:2 * n]
    src[n // 2] = src[0]  # a page may be copied to several
    want = [bits(t).clone() for t in (*pages, *scales)]
    for t, w in zip((*pages, *scales), want):
        w[dst] = bits(t)[src]
    first = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (*pages, *scales)]
    dash.cache_copy_fp8(*pages, *scales, src, dst)
    dash.cache_copy_fp8(*first, src.tolist(), dst.tolist())
    dash.cache_copy_fp8(*pages, *scales, [], [])
    dash.dash_sync_status()
    for t, f, w in zip((*pages, *scales), first, want):
        assert torch.equal(bits(t), w) and torch.equal(bits(f.contiguous()), w)


# ----------------------------------------------------------------- decode
CASES = [([1], 1, 1, 64, 16), ([0, 5, 0], 4, 2, 128, 16), ([64, 63, 65, 256, 257, 255], 8, 2, 128, 16),
         ([300, 1000, 17], 6, 2, 64, 24), ([2000, 1], 32, 1, 128, 64), ([777] * 3, 20, 1, 64, 1), ([90, 513], 16, 1, 128, 16),
         ([40000, 3], 4, 4, 128, 128), ([33000, 65], 3, 1, 64, 7), (list(range(0, 900, 5)), 2, 1, 64, 32),
         (list(range(0, 900, 7)), 9, 1, 128, 16)]


# Room in the table alone decides between the forms for small calls and for those that fill the GPU: a table row of
# 16384 tokens has room for 64 splits.
ROOM = 16384


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("lens,hq,hkv,D,page", CASES, ids=lambda x: str(x)[:40])
def test_decode(lens, hq, hkv, D, page, room):
    if room:  # more sequences, so that there is room for more splits than CTAs
        lens = (lens * 10)[:max(len(lens), 10)] + [0, 1, 129]
    c = cache(lens, hkv, D, page, heads_first=hq != 3, width=max(room, max(lens)) // page + 1 if room else None)
    kp, vp, ks, vs, table = c
    # whatever stands behind a sequence's last token is not read into its result
    for b, n in enumerate(lens):
        if n % page:
            last = table[b, n // page].long()
            for pages, scales in ((kp, ks), (vp, vs)):
                bits(pages)[last, n % page:], scales[last, n % page:] = 0x7f, NAN
    q = P.normal(9, len(lens), hq, D)
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    dash.dash_sync_status()
    check(q, c, lens, 1 / math.sqrt(D), o, lse)
    o2, lse2 = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("page", [1, 8, 12, 24, 32, 48, 64, 128, 200, 256])
def test_decode_of_whole_tiles_in_pages_of_every_kind(page, D):
    # rows are fetched a page's part of a tile at a time where it has one, row by row elsewhere; one bad page
    lens, hq, hkv = [128, 1024, 1023, 640, 2500, 0, 127, 256, 1, 3000], 16, 2
    kp, vp, ks, vs, table = c = cache(lens, hkv, D, page, width=max(ROOM, 3000) // page + 1)
    q = P.normal(9, len(lens), hq, D)
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    dash.dash_sync_status()
    check(q, c, lens, 1 / math.sqrt(D), o, lse)
    # heads first, K and V side by side
    both = torch.zeros((kp.shape[0], 2, hkv, page, D), dtype=torch.uint8, device="cuda")
    both[:, 0], both[:, 1] = bits(kp).transpose(1, 2), bits(vp).transpose(1, 2)
    k2, v2 = both[:, 0].transpose(1, 2).view(FP8), both[:, 1].transpose(1, 2).view(FP8)
    o2, lse2 = dash.attn_decode_fp8(q, k2, v2, ks, vs, table, i32(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    table[4, 700 // page] = -1
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    with pytest.raises(dash.DashError, match="outside the cache"):
        dash.dash_sync_status()
    check(q, c, lens, 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("hq,hkv,D", [(16, 8, 64), (16, 8, 128), (3, 1, 64)])
def test_decode_of_many_long_sequences(hq, hkv, D):
    # loads run ahead of the products and the softmax as far as there is room, item after item
    lens, page = [4096, 5000, 3000, 4096, 100, 8192, 4097, 1] * 4, 16
    kp, vp, ks, vs, table = c = cache(lens, hkv, D, page, width=ROOM * (8 // hkv) // page)
    q = P.normal(2, len(lens), hq, D)
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    dash.dash_sync_status()
    few = slice(0, 8)
    check(q[few], (kp, vp, ks, vs, table[few]), lens[few], 1 / math.sqrt(D), o[few], lse[few])
    for _ in range(5):
        o2, lse2 = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    dash.dash_sync_status()


@pytest.mark.parametrize("n,D,top", [(256, 128, 900), (257, 128, 900), (1500, 128, 300), (1500, 64, 300), (3000, 128, 60)])
def test_decode_of_very_many_sequences(n, D, top):
    # up to 256 the lengths are held and the items sorted by them; sequences that are all short have a form of their own
    lens, hq, hkv, page = [i * 37 % (top + 1) for i in range(n)], 3, 1, 4
    c = cache(lens, hkv, D, page)
    q = P.normal(4, n, hq, D)
    o, lse = dash.attn_decode_fp8(q, *c, i32(lens))
    dash.dash_sync_status()
    check(q, c, lens, 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("spread", [3.0, 20.0])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (12, 1)])
def test_decode_of_rows_of_very_different_scales(hq, hkv, spread, room):
    # K's scale far down as well, so that scores stay small whatever the rows' scales are; V's as they come
    lens, D, page = [700, 65, 3000, 5, 128, 129], 128, 16
    kp, vp, ks, vs, table = cache(lens, hkv, D, page, spread=spread, width=room // page or None)
    ks = torch.ones_like(ks) * 2.0 ** -8
    # the largest V rows first, in the middle, and on tokens that hardly count
    c = (kp, vp, ks, vs, table)
    for seed in (1, 2):
        q = P.normal(seed, 6, hq, D)
        o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
        check(q, c, lens, 1 / math.sqrt(D), o, lse)
    # scales of zero weigh nothing in O and count in the sum; arbitrary (not power of two) scales
    vs[table[0, 3].long(), 2:9] = 0.0
    ks.mul_(1.37)
    vs.mul_(0.77)
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    check(q, c, lens, 1 / math.sqrt(D), o, lse)
    vs.zero_()
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    assert not o.any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("gain", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_decode_of_queries_of_any_magnitude(gain, room):
    lens, hq, hkv, D, page = [300, 40, 129, 0, 7], 4, 2, 64, 16
    kp, vp, ks, vs, table = cache(lens, hkv, D, page, width=room // page or None)
    q = (P.normal(3, 5, hq, D).double() * gain).bfloat16()
    ks = (ks.double() / gain).float()
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    check(q, (kp, vp, ks, vs, table), lens, 1 / math.sqrt(D), o, lse)
    o, lse = dash.attn_decode_fp8(torch.zeros_like(q), kp, vp, ks, vs, table, i32(lens))
    check(torch.zeros_like(q), (kp, vp, ks, vs, table), lens, 1 / math.sqrt(D), o, lse)


def test_decode_does_not_depend_on_the_other_sequences():
    lens, hq, hkv, D, page = [5000, 130, 20000, 1, 700], 8, 2, 128, 16
    kp, vp, ks, vs, table = cache(lens, hkv, D, page, width=4000)
    q = P.normal(5, 5, hq, D)
    # three of them in a small call, and each alone
    o, lse = dash.attn_decode_fp8(q[:3], kp, vp, ks, vs, table[:3], i32(lens[:3]))
    for b, n in enumerate(lens[:3]):
        w = -(-n // page)
        ob, lb = dash.attn_decode_fp8(q[b:b + 1], kp, vp, ks, vs, table[b:b + 1, :w].contiguous(), i32([n]))
        assert torch.equal(o[b], ob[0]) and torch.equal(lse[b], lb[0])
    # all in calls that fill the GPU, in another order, with other neighbours
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    order = torch.tensor([3, 0, 4, 2, 1, 0, 3, 3], device="cuda")
    oo, ll = dash.attn_decode_fp8(q[order], kp, vp, ks, vs, table[order], i32(lens)[order])
    assert torch.equal(oo, o[order]) and torch.equal(ll, lse[order])
    check(q, (kp, vp, ks, vs, table), lens, 1 / math.sqrt(D), o, lse)
    # more sequences than are sorted by their length
    many = torch.arange(1500, device="cuda") % 5
    small = torch.minimum(i32(lens), i32([300, 130, 299, 1, 257]))
    oo, ll = dash.attn_decode_fp8(q[many], kp, vp, ks, vs, table[many], small[many])
    o, lse = oo[:5], ll[:5]
    assert torch.equal(oo, o[many]) and torch.equal(ll, lse[many])
    check(q, (kp, vp, ks, vs, table), small.tolist(), 1 / math.sqrt(D), o, lse)


@pytest.mark.parametrize("hq,hkv,D,page,width", [(16, 4, 128, 16, 44), (8, 1, 64, 16, 64), (20, 1, 128, 7, 90),
                                                 (2, 2, 64, 1, 2000), (12, 1, 128, 64, 30)])
def test_decode_small_calls_and_captures(hq, hkv, D, page, width):
    cap = page * width
    lens = sorted({0, 1, 255, 256, 257, 512, 513, 777, cap // 2 + 1, cap - 1, cap} & set(range(cap + 1))) * 6
    c = cache(lens, hkv, D, page, width=width)
    kp, vp, ks, vs, table = c
    q = P.normal(15, len(lens), hq, D)
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    dash.dash_sync_status()
    check(q, c, lens, 1 / math.sqrt(D), o, lse)
    ones = [dash.attn_decode_fp8(q[b:b + 1], kp, vp, ks, vs, table[b:b + 1], i32([n])) for b, n in enumerate(lens)]
    o1, l1 = (torch.cat(t) for t in zip(*ones))
    check(q, c, lens, 1 / math.sqrt(D), o1, l1)
    for rows, want in ((slice(-1, None), (o1, l1)), (slice(None), (o, lse))):
        length, graph = i32([1] * len(lens))[rows], torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            og, lg = dash.attn_decode_fp8(q[rows], kp, vp, ks, vs, table[rows], length)
        length.copy_(i32(lens)[rows])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(og, want[0][rows]) and torch.equal(lg, want[1][rows])
    dash.dash_sync_status()


def test_decode_strides_streams_and_lengths_out_of_range():
    lens, hq, hkv, D, page = [100, 700, 31], 8, 2, 64, 16
    kp, vp, ks, vs, table = cache(lens, hkv, D, page)
    q = P.normal(6, 3, hq, D)
    want = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    # a head-first cache, K and V side by side, Q a part of a fused row, a table inside a larger one
    both = torch.zeros((kp.shape[0], 2, hkv, page, D), dtype=torch.uint8, device="cuda")
    both[:, 0], both[:, 1] = bits(kp).transpose(1, 2), bits(vp).transpose(1, 2)
    k2, v2 = both[:, 0].transpose(1, 2).view(FP8), both[:, 1].transpose(1, 2).view(FP8)
    s2 = torch.stack([ks, vs], 3)
    fused = torch.full((3, hq + 4, D), NAN, dtype=torch.bfloat16, device="cuda")
    q2 = fused[:, 2:2 + hq]
    q2.copy_(q)
    t2 = torch.full((3, table.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    t2[:, :table.shape[1]] = table
    side = torch.cuda.Stream()
    got = dash.attn_decode_fp8(q2, k2, v2, s2[..., 0], s2[..., 1], t2[:, :table.shape[1]], i32(lens), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    small, full = table[:, :2].contiguous(), i32([32, 32, 31])
    a = dash.attn_decode_fp8(q2, kp, vp, ks, vs, small, i32([-4, 10**9, 31]))
    b = dash.attn_decode_fp8(q2, kp, vp, ks, vs, small, full)
    dash.dash_sync_status()
    assert torch.equal(a[0][1:], b[0][1:]) and not a[0][0].any() and (a[1][0] == -INF).all()
    # without lse, into a given o
    o = torch.empty_like(q)
    ws = torch.empty(dash.dash_decode_workspace(3, hq, D, page, table.shape[1]), dtype=torch.uint8, device="cuda")
    dash.dash_attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens), o, None, 1 / math.sqrt(D), ws)
    assert torch.equal(o, want[0])


@pytest.mark.parametrize("room", [0, ROOM])
def test_decode_of_bad_pages_nan_and_infinite_scores(room):
    lens, hq, hkv, D, page = [70, 40, 300, 128, 700], 4, 2, 128, 16
    c = cache(lens, hkv, D, page, width=room // page or None)
    kp, vp, ks, vs, table = c
    q = P.normal(7, 5, hq, D)
    for bad in (-1, kp.shape[0], 2**31 - 1):
        t = table.clone()
        t[0, 1] = bad
        o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, t, i32(lens))
        with pytest.raises(dash.DashError, match="outside the cache"):
            dash.dash_sync_status()
        dash.dash_sync_status()  # cleared
        check(q, (kp, vp, ks, vs, t), lens, 1 / math.sqrt(D), o, lse)
    good = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    # a NaN row of K, a NaN row of V, a NaN code of V: heads of that K/V head and sequence alone
    for what, where in (("k", ks), ("v", vs), ("code", vp)):
        kept = where.clone()
        at = (table[0, 2].long(), 5, 1)
        if what == "code":
            bits(where)[(*at, 17)] = 0x7f
        else:
            where[at] = NAN
        o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
        assert torch.equal(o[1:], good[0][1:]) and torch.equal(o[0, :2], good[0][0, :2])
        if what == "code":
            assert o[0, 2:, 17].isnan().all() and o[0, 2:, 16].isfinite().all()
        else:
            assert o[0, 2:].isnan().all() and (lse[0, 2:].isnan().all() if what == "k" else lse[0, 2:].isfinite().all())
        bits(where).copy_(bits(kept))
    # a query with a NaN or an infinity makes its row NaN
    for bad in (NAN, INF, -INF):
        one = q.clone()
        one[0, 1, 3], one[4, 2, 100] = bad, bad
        o, lse = dash.attn_decode_fp8(one, kp, vp, ks, vs, table, i32(lens))
        for b, h in ((0, 1), (4, 2)):
            assert o[b, h].isnan().all() and lse[b, h].isnan()
            o[b, h], lse[b, h] = good[0][b, h], good[1][b, h]
        assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
    # rows far below the others, and a first tile that weighs next to nothing
    ks[table[4, :16].long()] *= 2.0 ** -20
    ks[table[4, 16:44].long()] *= 4.0
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32(lens))
    check(q, c, lens, 1 / math.sqrt(D), o, lse)
    dash.dash_sync_status()


def test_large_offsets():
    # a cache of more than 2^32 bytes
    hq, hkv, D, page = 4, 4, 128, 64
    n_pages = (2**32 // (page * hkv * D)) + 40
    kp, vp = (torch.zeros(n_pages, page, hkv, D, dtype=torch.uint8, device="cuda").view(FP8) for _ in range(2))
    ks, vs = (torch.ones(n_pages, page, hkv, device="cuda") for _ in range(2))
    table = i32([[n_pages - 1, 3, n_pages - 20, n_pages - 2]])
    k, v = P.normal(1, 250, hkv, D), P.normal(2, 250, hkv, D)
    dash.cache_write_fp8(k, v, kp, vp, ks, vs, table, i32([0]), i32([0, 250]))
    q = P.normal(8, 1, hq, D)
    o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, i32([250]))
    dash.cache_copy_fp8(kp, vp, ks, vs, [n_pages - 1, n_pages - 2], [0, n_pages - 5])
    rk, rv = dash.cache_read_fp8(kp, vp, ks, vs, i32([[0, 3, n_pages - 20, n_pages - 5]]), i32([0]), i32([0, 250]), 250)
    dash.dash_sync_status()
    small = [t[table[0].long()] for t in (bits(kp), bits(vp), ks, vs)]
    check(q, (small[0].view(FP8), small[1].view(FP8), small[2], small[3], i32([[0, 1, 2, 3]])), [250], 1 / math.sqrt(D),
          o, lse)
    for x, back in ((k, rk), (v, rv)):
        codes, scale = R.quantise(x)
        assert torch.equal(back.double(), codes * scale[..., None])


def test_refusals():
    kp, vp, ks, vs, table = cache([32], 2, 64, 16)
    q, n = P.normal(1, 1, 4, 64), i32([32])
    f = dash.attn_decode_fp8
    for bad in (lambda: f(q.float(), kp, vp, ks, vs, table, n), lambda: f(q, kp, vp[1:], ks, vs, table, n),
                lambda: f(q, kp.float().bfloat16(), vp, ks, vs, table, n), lambda: f(q, kp, vp, ks.double(), vs, table, n),
                lambda: f(q, kp, vp, ks, vs[1:], table, n), lambda: f(q, kp, vp, ks, vs, table.long(), n),
                lambda: f(q, kp, vp, ks.cpu(), vs, table, n), lambda: f(q, kp, vp, ks, vs, table, n.long()),
                lambda: f(P.normal(1, 1, 4, 128), kp, vp, ks, vs, table, n),
                lambda: dash.cache_copy_fp8(kp, vp, ks, vs, [0], [1, 2]),
                lambda: dash.cache_write_fp8(q, q, kp, vp, ks, vs, table, i32([0]), i32([0, 1])),
                lambda: dash.cache_read_fp8(kp, vp, ks, vs, table, i32([0]), i32([0]), 1),
                lambda: dash.attn_decode(q, kp, vp, table, n)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dash.DashError, match="overlap|strides"):
        f(q, kp, vp, ks[:, :, :1].expand(-1, -1, 2), vs, table, n)
    with pytest.raises(dash.DashError, match="twice"):
        dash.cache_copy_fp8(kp, vp, ks, vs, [0, 1], [2, 2])


def test_prompt_fork_and_decode_together():
    # two prompts go through the norms and into the 8-bit cache, the first is forked, all take a new token, and the
    # context read back gives the packed forward the same answer as the decode
    hq, hkv, D, page, lens = 8, 2, 128, 16, [150, 37]
    rows = sum(lens)
    fused = P.normal(3, rows + 3, hq + 2 * hkv, D)
    w = [torch.ones(D, device="cuda")] * 2
    rope = dash.rope_table(200, D)
    positions = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens] + [i32([150, 37, 150])])
    q, k = dash.qk_norm_rope(fused[:, :hq], fused[:, hq:hq + hkv], *w, rope, positions)
    v = fused[:, hq + hkv:]
    kp, vp = (torch.zeros(40, page, hkv, D, dtype=torch.uint8, device="cuda").view(FP8) for _ in range(2))
    ks, vs = (torch.zeros(40, hkv, page, device="cuda").transpose(1, 2) for _ in range(2))
    c = (kp, vp, ks, vs)
    table = torch.arange(36, dtype=torch.int32, device="cuda").reshape(3, 12)
    dash.cache_write_fp8(k[:rows], v[:rows], *c, table[:2], i32([0, 0]), i32([0, 150, 187]))
    table[2, :9] = table[0, :9]
    dash.cache_copy_fp8(*c, [int(table[0, 9])], [int(table[2, 9])])
    dash.cache_write_fp8(k[rows:], v[rows:], *c, table, i32([150, 37, 150]), i32([0, 1, 2, 3]))
    now = [151, 38, 151]
    o, lse = dash.attn_decode_fp8(q[rows:], *c, table, i32(now))
    dash.dash_sync_status()
    check(q[rows:], (*c, table), now, D ** -0.5, o, lse)
    cu = [0, 151, 189, 340]
    rk, rv = dash.cache_read_fp8(*c, table, i32([0, 0, 0]), i32(cu), 340)
    fq = torch.zeros(340, hq, D, dtype=torch.bfloat16, device="cuda")
    last = torch.tensor([150, 188, 339], device="cuda")
    fq[last] = q[rows:]
    po, pl = dash.attn_packed_fwd(dash.PackedPlan(now, hq, hkv, D), fq, rk, rv)
    ro, _, mag = P.decode(q[rows:], R.values(kp, ks), R.values(vp, vs), table, now, D ** -0.5)
    P.within("packed", po[last], ro, mag)
    assert (pl[:, last].T - lse).abs().max() <= 2e-4


# Very long sequences whose weights differ widely.  What a weight loses beyond U of itself does not add up over a long
# split: in two e4m3 terms it is 2^-14 where the weight that the maximum was last set by stands at 2^4, which is in the
# same 1024 tokens: 2^-18 of their largest (2^-82 of the largest of all, where that is more); in f16 it is 2^-25 of the
# largest of its split.
def check_long(q, c, n, scale, o, lse, form):
    kp, vp, ks, vs, row = c
    page, D, U = kp.shape[1], kp.shape[3], P.U
    x = (R.values(kp, ks)[row.long()].reshape(-1, D)[:n] @ q.double().T * scale).T          # [heads, n]
    codes = bits(vp)[row.long()].view(FP8).reshape(-1, D)[:n].double().abs()
    cs = vs[row.long()].reshape(-1)[:n].double()
    v = R.values(vp, vs)[row.long()].reshape(-1, D)[:n]
    rl = torch.logsumexp(x, 1)
    p = torch.exp(x - rl[:, None])
    ro, mag = p @ v, p @ v.abs()
    chunk = 1024 if form == "wide" else max(256, 1 << (-(-n // 64) - 1).bit_length())
    pad = -n % chunk
    tops = torch.nn.functional.pad(p * cs, (0, pad)).unflatten(1, (-1, chunk)).amax(2)        # [heads, pieces]
    sums = torch.nn.functional.pad(codes, (0, 0, 0, pad)).unflatten(0, (-1, chunk)).sum(1)    # [pieces, D]
    floor = (2.0 ** -18 if form == "wide" else 2.0 ** -25) * (tops @ sums)
    if form == "wide":
        floor += 2.0 ** -82 * tops.amax(1, keepdim=True) * codes.sum(0)
    assert (lse.double() - rl).abs().max() <= 1e-4
    err = (o.double() - ro).abs()
    bad = ~(err <= U * ro.abs() + (1 + U) * ((U + P.EPS) * mag + floor) + 1e-30)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside their bound, worst {(err / mag)[bad].max()} of it"


def long_cache(n, D, page=128):
    """One sequence's pages, K of zeros and V of ones, scales of 1, and a table row that names them in random order."""
    n_pages = -(-n // page)
    row = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)).int().cuda()
    kp = torch.zeros(n_pages, page, 1, D, dtype=torch.uint8, device="cuda").view(FP8)
    vp = torch.full((n_pages, page, 1, D), 0x38, dtype=torch.uint8, device="cuda").view(FP8)
    ks, vs = (torch.ones(n_pages, 1, page, device="cuda").transpose(1, 2) for _ in range(2))
    return kp, vp, ks, vs, row


# 12 sequences of 64 splits are more items than a GPU takes at once, 2 are not
FORMS = pytest.mark.parametrize("form,B", [("wide", 12), ("small", 2)], ids=["wide", "small"])


def put(pages, row, t, dim, codes):
    """Codes of tokens t in one dim."""
    page = pages.shape[1]
    bits(pages)[row[t // page].long(), t % page, 0, dim] = bits(codes.to(FP8))


@FORMS
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("n,D", [(262144, 128), (262144, 64), (1000003, 64)])
def test_decode_of_a_token_that_outweighs_a_long_sequence(n, D, where, form, B):
    hq = 8
    kp, vp, ks, vs, row = c = long_cache(n, D)
    t = torch.arange(n, device="cuda")
    at = {"first": 0, "middle": n // 2 + 77, "last": n - 1}[where]
    put(kp, row, t[at:at + 1], 0, torch.ones(1, device="cuda"))
    put(kp, row, t, 1, torch.randn(n, generator=torch.Generator("cuda").manual_seed(5), device="cuda") / 4)
    split = 1 << (-(-n // 64) - 1).bit_length()
    put(kp, row, t, 2, torch.where(t // split == at // split, 0.0, -60.0))
    # powers of two between that token's weight and the others', which are equal or (the last two) random; heads 2 and 3
    # have next to nothing in the other splits
    q = torch.zeros(B, hq, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = torch.tensor([16.0, 17.0, 18.0, 19.0, 20.0, 18.125, 18.125, 22.0])
    q[:, 6:, 1] = 1.0
    q[:, 2:4, 2] = 1.0
    lens, table = i32([n] * B), row[None].expand(B, -1).contiguous()
    g = torch.Generator("cuda").manual_seed(6)
    for values in ("ones", "positive"):
        if values == "positive":
            bits(vp).copy_(bits((torch.randn(vp.shape, generator=g, device="cuda").abs() * 100).clamp(max=448).to(FP8)))
            vs.copy_(torch.exp2(torch.randint(-3, 4, vs.shape, generator=g, device="cuda").float()))
        o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, lens, scale=math.log(2))
        dash.dash_sync_status()
        check_long(q[0], c, n, math.log(2), o[0], lse[0], form)
        assert torch.equal(o, o[:1].expand_as(o)) and torch.equal(lse, lse[:1].expand_as(lse))
        if values == "ones":
            # whole powers of two are held exactly, but for those within 1024 tokens of that one, which lose 2^-18 of it
            # each at most: what is left is the result's own rounding and the 32-bit arithmetic
            assert ((o[0, :5].double() - 1).abs() <= P.U + 2.0 * P.EPS + 1023 * 2.0 ** -18).all()


@FORMS
@pytest.mark.parametrize("D", [128, 64])
def test_decode_of_tiles_whose_weights_rise_and_fall(D, form, B):
    # each 128 tokens stand at a level of their own, up to 2^120 apart, and the levels of V's rows as well
    n, hq = 300001, 8
    kp, vp, ks, vs, row = c = long_cache(n, D)
    t, g = torch.arange(n, device="cuda"), torch.Generator("cuda").manual_seed(7)
    levels = torch.randn(n // 128 + 1, generator=g, device="cuda") * 18
    put(kp, row, t, 0, levels.clamp(-60, 60)[t // 128])
    put(kp, row, t, 1, torch.linspace(60, -60, n, device="cuda"))      # ever down, split by split and over all
    put(kp, row, t, 2, ((t % 4096) < 128).float() * 40)                # the first tile of a split above the others
    put(kp, row, t, 3, torch.randn(n, generator=g, device="cuda") * 2)
    bits(vp).copy_(bits((torch.randn(vp.shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(FP8)))
    q = torch.zeros(B, hq, D, dtype=torch.bfloat16, device="cuda")
    for h, w in enumerate([(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, -1, 0), (1, 0, 0, 1), (0, 0, 1, 1),
                           (0, 8, 0, 1), (0.25, 0, 0, 1)]):
        q[:, h, :4] = torch.tensor(w)
    lens, table = i32([n] * B), row[None].expand(B, -1).contiguous()
    for _ in range(2):
        o, lse = dash.attn_decode_fp8(q, kp, vp, ks, vs, table, lens, scale=math.log(2))
        dash.dash_sync_status()
        check_long(q[0], c, n, math.log(2), o[0], lse[0], form)
        assert torch.equal(o, o[:1].expand_as(o)) and torch.equal(lse, lse[:1].expand_as(lse))
        vs.copy_(torch.exp2(torch.randint(-30, 31, vs.shape, generator=g, device="cuda").float()))
