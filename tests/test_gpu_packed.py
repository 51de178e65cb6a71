"""Packed, grouped-head attention on the GPU against 64-bit plain forms: lengths
from none to several tiles, shared heads, strides, garbage around the sequences,
run-to-run bits, streams and captured graphs."""
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


def problem(lens, hq, hkv, D, extra=0, seed=1):
    rows = sum(lens) + extra
    q, do = R.normal(seed, rows, hq, D), R.normal(seed + 1, rows, hq, D)
    k, v = R.normal(seed + 2, rows, hkv, D), R.normal(seed + 3, rows, hkv, D)
    return q, k, v, do


def check_forward(lens, q, k, v, causal, scale, o, lse):
    n = sum(lens)
    ro, rl, mag = R.forward(lens, q[:n], k[:n], v[:n], causal, scale)
    R.within("O", o[:n], ro, mag)
    # a score is a 32-bit sum of D products: its error and that of the logarithm, in absolute terms
    assert (lse[:, :n].double() - rl[:, :n]).abs().max() <= 1e-4 if n else True


def check_backward(lens, q, k, v, o, do, lse, causal, scale, grads):
    n = sum(lens)
    ref, mags = R.backward(lens, *(t[:n] for t in (q, k, v, o, do)), lse[:, :n], causal, scale)
    for name, x, r, m in zip(("dQ", "dK", "dV"), grads, ref, mags):
        R.within(name, x[:n], r, m)


CASES = [([1], 1, 1, 64, True), ([128], 2, 1, 128, True), ([129, 1, 127], 4, 2, 64, True),
         ([0, 5, 0, 300, 0], 6, 2, 128, True), ([257, 64, 0, 1], 4, 4, 64, False), ([1000, 3], 8, 1, 128, True),
         ([200], 5, 1, 64, False), ([700, 513], 2, 2, 128, False), ([1300, 384, 31], 4, 4, 128, True),
         (list(range(1, 60, 3)), 8, 2, 128, True), ([2049], 16, 4, 64, True), ([640], 3, 3, 128, True),
         # few, long KV tiles: dK and dV are summed in parts
         ([1930, 70], 8, 1, 64, True), ([1300], 6, 1, 128, False), ([2000], 4, 2, 128, True)]


@pytest.mark.parametrize("lens,hq,hkv,D,causal", CASES, ids=str)
def test_forward_and_backward(lens, hq, hkv, D, causal):
    q, k, v, do = problem(lens, hq, hkv, D)
    scale = 1 / math.sqrt(D)
    plan = dash.PackedPlan(lens, hq, hkv, D, causal=causal, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    dash.dash_sync_status()
    check_forward(lens, q, k, v, causal, scale, o, lse)
    grads = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    dash.dash_sync_status()
    check_backward(lens, q, k, v, o, do, lse, causal, scale, grads)
    again = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    o2, lse2 = dash.attn_packed_fwd(plan, q, k, v)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_strides_garbage_and_rows_behind(D, causal):
    # parts of a fused projection whose every other element is NaN, rows behind the last sequence that must stay
    lens, hq, hkv, extra = [130, 1, 0, 300], 4, 2, 37
    n, rows = sum(lens), sum(lens) + extra
    src = problem(lens, hq, hkv, D, extra, seed=11)
    fused = torch.full((rows + 3, 3 * hq + 3, D), NAN, dtype=torch.bfloat16, device="cuda")
    q, k, v = fused[1:1 + rows, :hq], fused[1:1 + rows, hq:hq + hkv], fused[1:1 + rows, hq + hkv:hq + 2 * hkv]
    headfirst = torch.full((hq + 1, rows, D), NAN, dtype=torch.bfloat16, device="cuda")
    do = headfirst[:hq].transpose(0, 1)
    for dst, t in zip((q, k, v, do), src):
        dst[:n] = t[:n]
    keep = 3.0
    out = torch.full((rows, 2 * hq + 2 * hkv, D + 8), keep, dtype=torch.bfloat16, device="cuda")
    o, dq = out[:, :hq, :D], out[:, hq:2 * hq, :D]
    dk, dv = out[:, 2 * hq:2 * hq + hkv, :D], out[:, 2 * hq + hkv:, :D]
    lse = torch.full((hq, rows), keep, device="cuda")
    scale = 0.11
    plan = dash.PackedPlan(lens, hq, hkv, D, causal=causal, backward=True)
    ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")  # NaN in every float
    dash.dash_attn_packed_fwd(plan, q, k, v, o, lse, scale)
    dash.dash_attn_packed_bwd(plan, q, k, v, o, do, lse, dq, dk, dv, scale, ws)
    dash.dash_sync_status()
    check_forward(lens, q, k, v, causal, scale, o, lse)
    check_backward(lens, q, k, v, o, do, lse, causal, scale, (dq, dk, dv))
    assert (out[n:] == keep).all() and (out[:, :, D:] == keep).all() and (lse[:, n:] == keep).all()
    # contiguous tensors give the same bits
    oc, lc = dash.attn_packed_fwd(plan, *(t.contiguous() for t in (q, k, v)), scale)
    gc = dash.attn_packed_bwd(plan, *(t.contiguous() for t in (q, k, v, o, do)), lse.contiguous(), scale)
    for a, b in zip((oc, *gc), (o, dq, dk, dv)):
        assert torch.equal(a[:n], b[:n]) and not a[n:].any()
    assert torch.equal(lc[:, :n], lse[:, :n]) and (lc[:, n:] == float("-inf")).all()


def test_sequences_do_not_touch_each_other():
    # NaN and infinities in one sequence leave the others' bits as they are
    lens, hq, hkv, D = [70, 150, 40], 4, 2, 128
    q, k, v, do = problem(lens, hq, hkv, D, seed=21)
    plan = dash.PackedPlan(lens, hq, hkv, D, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    g = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    bad = [t.clone() for t in (q, k, v, do)]
    for t, x in zip(bad, (NAN, float("inf"), NAN, float("-inf"))):
        t[70:220] = x
    o2, lse2 = dash.attn_packed_fwd(plan, *bad[:3])
    g2 = dash.attn_packed_bwd(plan, *bad[:3], o2, bad[3], lse2)
    dash.dash_sync_status()
    for a, b in zip((o, *g), (o2, *g2)):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[220:], b[220:])
    assert torch.equal(lse[:, :70], lse2[:, :70]) and torch.equal(lse[:, 220:], lse2[:, 220:])


def test_forward_does_not_depend_on_the_batch():
    # a sequence's forward bits are the same alone and packed between others
    D, hq, hkv = 128, 6, 2
    q, k, v, _ = problem([333], hq, hkv, D, seed=31)
    alone = dash.attn_packed_fwd(dash.PackedPlan([333], hq, hkv, D), q, k, v)
    pad = [torch.cat([R.normal(40 + i, 200, t.shape[1], D), t, R.normal(50 + i, 55, t.shape[1], D)])
           for i, t in enumerate((q, k, v))]
    o, lse = dash.attn_packed_fwd(dash.PackedPlan([200, 333, 55], hq, hkv, D), *pad)
    assert torch.equal(o[200:533], alone[0]) and torch.equal(lse[:, 200:533], alone[1])


def test_scores_of_every_size():
    # rows whose maximum grows from tile to tile (the running maximum moves), and scores far from zero
    D, lens = 64, [900]
    q, k, v, do = problem(lens, 2, 1, D, seed=61)
    k = (k.float() * torch.linspace(0.1, 6.0, 900, device="cuda")[:, None, None]).bfloat16()
    q = (q.float() * 3).bfloat16()
    plan = dash.PackedPlan(lens, 2, 1, D, causal=False, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v, 0.5)
    dash.dash_sync_status()
    ro, rl, mag = R.forward(lens, q, k, v, False, 0.5)
    # scores reach 0.5 * 3 * 6 * 64 = 576 and more: a 32-bit sum of D products of that size is off by about
    # D * 2^-24 * 2000 < 2^-7 at most, which moves every p by less than 2^-6 of itself
    assert (lse.double() - rl).abs().max() <= 2 ** -7
    assert ((o.double() - ro).abs() <= R.bound(ro, mag) + 2 ** -6 * mag).all()


def test_against_the_dense_attention():
    # equal lengths: the framework's dense forward and backward on the same values
    B, H, S, D = 2, 3, 256, 128
    q, k, v, do = problem([S] * B, H, H, D, seed=71)
    plan = dash.PackedPlan([S] * B, H, H, D, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    g = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    dense = lambda t: t.reshape(B, S, H, D).transpose(1, 2).contiguous()
    do_, lse_ = dash.attn_fwd(dense(q), dense(k), dense(v), True)
    dg = dash.attn_bwd(dense(q), dense(k), dense(v), dense(o), dense(do),
                       lse.reshape(H, B, S).transpose(0, 1).contiguous(), True, schedule="serial")
    dash.dash_sync_status()
    for a, b in zip((o, *g), (do_, *dg)):
        # both are within U of the sums' magnitudes of the exact value; rows here have magnitudes below 8
        assert (dense(a).float() - b.float()).abs().max() <= 4 * R.U * 8
    assert (lse.reshape(H, B, S).transpose(0, 1) - lse_).abs().max() <= 1e-4


@pytest.mark.parametrize("D", [64, 128])
def test_rows_at_odd_multiples_of_16_bytes(D):
    # the same bits as with rows at multiples of 32 bytes, and nothing written beside the rows; few K/V heads of a
    # long sequence, whose dK and dV are summed in parts
    lens, hq, hkv = [2500, 3], 4, 1
    q, k, v, do = problem(lens, hq, hkv, D, seed=83)
    plan = dash.PackedPlan(lens, hq, hkv, D, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    want = (o, *dash.attn_packed_bwd(plan, q, k, v, o, do, lse))

    def odd(t):
        big = torch.full((t.shape[0], t.shape[1] * D + 24), 7.0, dtype=t.dtype, device="cuda")
        part = big[:, 8:8 + t.shape[1] * D].unflatten(1, t.shape[1:])
        assert part.data_ptr() % 32 == 16 and part.stride(0) % 16 == 8
        part.copy_(t)
        return big, part

    (_, o2), (_, do2), (_, q2), (_, k2), (_, v2) = (odd(t) for t in (o, do, q, k, v))
    outs = [odd(torch.zeros_like(t)) for t in want]
    lse2 = torch.empty_like(lse)
    ws = torch.empty(plan.workspace_bytes + 16, dtype=torch.uint8, device="cuda")[16:]
    scale = 1 / math.sqrt(D)
    dash.dash_attn_packed_fwd(plan, q2, k2, v2, outs[0][1], lse2, scale)
    dash.dash_attn_packed_bwd(plan, q2, k2, v2, o2, do2, lse, *(t for _, t in outs[1:]), scale, ws)
    dash.dash_sync_status()
    assert torch.equal(lse, lse2)
    for w, (big, got) in zip(want, outs):
        assert torch.equal(w, got)
        assert (big[:, :8] == 7).all() and (big[:, 8 + got.shape[1] * D:] == 7).all()


def test_streams_and_captured_graphs():
    lens, hq, hkv, D = [300, 77], 4, 2, 64
    q, k, v, do = problem(lens, hq, hkv, D, seed=81)
    plan = dash.PackedPlan(lens, hq, hkv, D, backward=True)

    def step():
        o, lse = dash.attn_packed_fwd(plan, q, k, v)
        return (o, lse, *dash.attn_packed_bwd(plan, q, k, v, o, do, lse))

    want = step()
    side = torch.cuda.Stream()
    o, lse = dash.attn_packed_fwd(plan, q, k, v, stream=side)
    g = dash.attn_packed_bwd(plan, q, k, v, o, do, lse, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (o, lse, *g)))
    # two captures whose replays overlap: each has its own workspace and outputs
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step())
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        eager = step()
    torch.cuda.synchronize()
    dash.dash_sync_status()
    for got in (*outs, eager):
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("hq,hkv,D,causal", [(8, 2, 128, True), (8, 2, 64, True), (3, 1, 128, False), (5, 5, 64, False),
                                             (5, 5, 128, True)])
def test_many_short_sequences(hq, hkv, D, causal):
    # dozens of one-tile items per CTA, each with a tail, so that warps run items ahead of each other; and the same
    # lengths with longer ones between, so that items of one and two tiles, with and without a second Q tile, alternate
    for lens in ([1 + (37 * i) % 127 for i in range(700)], [1 + (53 * i) % 300 for i in range(300)]):
        q, k, v, do = problem(lens, hq, hkv, D, seed=93)
        plan = dash.PackedPlan(lens, hq, hkv, D, causal=causal, backward=True)
        first = None
        for _ in range(5):
            o, lse = dash.attn_packed_fwd(plan, q, k, v)
            got = (o, lse, *dash.attn_packed_bwd(plan, q, k, v, o, do, lse))
            dash.dash_sync_status()
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        scale, few, n = 1 / math.sqrt(D), lens[:40], sum(lens[:40])
        cut = lambda *t: [x[:n].contiguous() for x in t]
        check_forward(few, *cut(q, k, v), causal, scale, o[:n], lse[:, :n])
        check_backward(few, *cut(q, k, v, o, do), lse[:, :n], causal, scale, [x[:n] for x in got[2:]])
        # the last ones, which end the CTAs' lists
        few, n = lens[-40:], sum(lens[-40:])
        cut = lambda *t: [x[-n:].contiguous() for x in t]
        check_forward(few, *cut(q, k, v), causal, scale, o[-n:], lse[:, -n:])
        check_backward(few, *cut(q, k, v, o, do), lse[:, -n:], causal, scale, [x[-n:] for x in got[2:]])


def test_a_long_sequence():
    # many KV tiles per row, several items per CTA, tails inside tiles
    lens, hq, hkv, D = [9001, 517], 4, 2, 128
    q, k, v, do = problem(lens, hq, hkv, D, seed=95)
    scale = 1 / math.sqrt(D)
    plan = dash.PackedPlan(lens, hq, hkv, D, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    g = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    dash.dash_sync_status()
    check_forward(lens, q, k, v, True, scale, o, lse)
    check_backward(lens, q, k, v, o, do, lse, True, scale, g)


def test_a_backward_captured_while_plans_come_and_go():
    # a plan that is dropped during a capture, and gradients of the same inputs in an eager call and in the graph
    lens, hq, hkv, D = [260], 4, 2, 128
    q, k, v, do = problem(lens, hq, hkv, D, seed=97)
    plan = dash.PackedPlan(lens, hq, hkv, D, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    eager = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    dropped = dash.PackedPlan([5, 6], hq, hkv, D, backward=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        del dropped
        captured = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, captured))
    # new values in the same tensors
    for t, i in ((q, 1), (k, 2), (v, 3)):
        t.copy_(R.normal(200 + i, *t.shape))
    o2, lse2 = dash.attn_packed_fwd(plan, q, k, v)
    o.copy_(o2)
    lse.copy_(lse2)
    graph.replay()
    torch.cuda.synchronize()
    again = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    assert all(torch.equal(a, b) for a, b in zip(again, captured))
    assert not torch.equal(eager[0], again[0])


def test_two_plans_on_two_streams():
    probs = [([700, 33], 4, 2, 64, 1), ([128, 1, 390], 6, 3, 64, 2)]
    data = [(dash.PackedPlan(l, hq, hkv, D, backward=True), *problem(l, hq, hkv, D, seed=300 + s))
            for l, hq, hkv, D, s in probs]

    def run(p, q, k, v, do, stream=None):
        o, lse = dash.attn_packed_fwd(p, q, k, v, stream=stream)
        return (o, lse, *dash.attn_packed_bwd(p, q, k, v, o, do, lse, stream=stream))

    want = [run(*d) for d in data]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    got = [[run(*d, stream=s) for d, s in zip(data, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    dash.dash_sync_status()
    for row in got:
        for w, g in zip(want, row):
            assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_empty_problems():
    for lens in ([], [0, 0]):
        plan = dash.PackedPlan(lens, 2, 1, 64, backward=True)
        q, k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda"), R.normal(1, 3, 1, 64)
        o, lse = dash.attn_packed_fwd(plan, q, k, k)
        assert not o.any() and (lse == float("-inf")).all()
        g = dash.attn_packed_bwd(plan, q, k, k, o, q, lse)
        assert not any(t.any() for t in g)


def test_refusals():
    q, k, v, do = problem([40], 4, 2, 64, seed=91)
    plan = dash.PackedPlan([40], 4, 2, 64)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    with pytest.raises(dash.DashError, match="without its backward"):
        dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    with pytest.raises(ValueError):
        dash.attn_packed_fwd(plan, q, k[:39], v)
    with pytest.raises(ValueError):
        dash.attn_packed_fwd(plan, q.float(), k, v)
    with pytest.raises(ValueError):
        dash.attn_packed_fwd(plan, q[:, :2], k, v)
    with pytest.raises(dash.DashError, match="fewer"):
        dash.attn_packed_fwd(plan, q[:39], k[:39], v[:39])
    with pytest.raises(dash.DashError, match="strides"):
        dash.attn_packed_fwd(plan, q, k[:, :1].expand(40, 2, 64), v)
    with pytest.raises(dash.DashError, match="aligned"):
        dash.attn_packed_fwd(plan, torch.empty(40 * 4 * 64 + 1, dtype=q.dtype, device="cuda")[1:].view(40, 4, 64), k, v)
    bp = dash.PackedPlan([40], 4, 2, 64, backward=True)
    ws = torch.empty(bp.workspace_bytes - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(dash.DashError, match="workspace"):
        dash.dash_attn_packed_bwd(bp, q, k, v, o, do, lse, torch.empty_like(q), torch.empty_like(k),
                                  torch.empty_like(v), 0.1, ws)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [500, 805])
def test_large_rows_outside_a_sequence_leave_its_bits(D, causal, n):
    # A sequence of several KV tiles that ends inside a warp's 32 rows.  The warp also computes the rows behind it,
    # whose scores here grow from tile to tile by far more than what makes it rescale: those of the next sequence,
    # then rows behind the last one.
    hq, hkv, more = 3, 1, 60
    q, k, v, do = problem([n], hq, hkv, D, seed=131)
    k = (k.float() * torch.linspace(0.2, 1.0, n, device="cuda")[:, None, None]).bfloat16()
    plan = dash.PackedPlan([n], hq, hkv, D, causal=causal, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    grads = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    check_forward([n], q, k, v, causal, 1 / math.sqrt(D), o, lse)
    behind = [torch.cat([t, (R.normal(140 + i, more, t.shape[1], D) * 100).bfloat16()])
              for i, t in enumerate((q, k, v))]
    # what the test is about: a row behind the sequence in the same 32 rows whose maximum moves, one inside that does
    # not but has grown (in powers of two, as far as 2^8)
    scores = torch.einsum("qhd,kd->hqk", behind[0][:(n + 31) // 32 * 32].float(), k[:, 0].float())
    scores = scores[:, n // 32 * 32:] / math.sqrt(D) * math.log2(math.e)
    grown = torch.stack([t.amax(-1) for t in scores.split(128, -1)], -1).diff(dim=-1)
    assert n % 32 and (grown[:, n % 32:] > 8).any() and ((grown[:, :n % 32] > 0) & (grown[:, :n % 32] < 8)).any()
    pad = torch.zeros_like(behind[0][n:])
    for lens in ([n, more], [n]):
        both = dash.PackedPlan(lens, hq, hkv, D, causal=causal, backward=True)
        o2, lse2 = dash.attn_packed_fwd(both, *behind)
        dash.dash_sync_status()
        assert torch.equal(o, o2[:n]) and torch.equal(lse, lse2[:, :n])
        g2 = dash.attn_packed_bwd(both, *behind, torch.cat([o, pad]), torch.cat([do, pad + 100]),
                                  torch.cat([lse, lse2[:, n:]], 1).contiguous())
        dash.dash_sync_status()
        assert torch.equal(grads[0], g2[0][:n])
        if len(lens) == 1:  # dK and dV too: the same lengths
            assert all(torch.equal(a, b[:n]) for a, b in zip(grads, g2))


def test_the_wait_for_dq_is_not_bounded():
    # Other work holds some SMs, so that dQ's CTAs for them start late and run their share after all others have
    # ended: dK and dV's CTAs on the freed SMs stand still for longer than any single wait may last, in a run where
    # nothing is stuck.  The held SMs belong to a dense backward on eight CTAs, which waits for nothing of this.
    limit_ms = 1
    lens, hq, hkv, D = [8192] * 16, 16, 4, 128
    q, k, v, do = problem(lens, hq, hkv, D, seed=151)
    plan = dash.PackedPlan(lens, hq, hkv, D, backward=True, spin_limit_ns=limit_ms * 10**6)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    want = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    dash.dash_sync_status()
    x = [R.normal(160 + i, 1, 8, 8192, D) for i in range(4)]
    xo, xl = dash.attn_fwd(*x[:3], False)
    grads = [torch.empty_like(x[0]) for _ in range(3)]
    held = torch.cuda.Stream()
    event = lambda: torch.cuda.Event(enable_timing=True)
    main, begin = (event(), event()), event()
    hold = lambda **kw: dash.dash_attn_bwd_ex(*x[:3], xo, x[3], xl, *grads, False, 1 / math.sqrt(D), "serial",
                                              num_ctas=8, stream=held, **kw)
    hold()  # its workspace and tables
    for e in main:
        e.record(held)

    def held_for(side, call):
        torch.cuda.synchronize()
        hold(main_events=main)
        side.wait_event(main[0])
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000)  # 0.2 ms: the eight CTAs stand
            begin.record(side)
        out = call()
        torch.cuda.synchronize()
        return begin.elapsed_time(main[1]), out

    # streams may share a hardware queue, where one waits for the other's kernel to end: one that does not
    streams = [torch.cuda.Stream(priority=-(i % 2)) for i in range(32)]
    side = next((s for s in streams if held_for(s, lambda: None)[0] > 2 * limit_ms), None)
    assert side is not None, "no stream runs beside the other"
    ms, got = held_for(side, lambda: dash.attn_packed_bwd(plan, q, k, v, o, do, lse, stream=side))
    assert ms > 2 * limit_ms, "the SMs were not held for long enough"
    dash.dash_sync_status()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_each_value_against_the_dense_attention(D, causal):
    # Equal lengths: the dense forward and backward on the same values.  Both sides round P, dS and the result to
    # bf16 once, so each value of either is within R.bound of the exact one, and the two within twice that.
    B, H, S, scale = 2, 3, 384, 1 / math.sqrt(D)
    q, k, v, do = problem([S] * B, H, H, D, seed=171)
    plan = dash.PackedPlan([S] * B, H, H, D, causal=causal, backward=True)
    o, lse = dash.attn_packed_fwd(plan, q, k, v)
    g = dash.attn_packed_bwd(plan, q, k, v, o, do, lse)
    dense = lambda t: t.reshape(B, S, H, D).transpose(1, 2).contiguous()
    packed = lambda t: t.transpose(1, 2).reshape(B * S, H, D)
    xo, xl = dash.attn_fwd(dense(q), dense(k), dense(v), causal)
    xg = dash.attn_bwd(dense(q), dense(k), dense(v), dense(o), dense(do),
                       lse.reshape(H, B, S).transpose(0, 1).contiguous(), causal, schedule="serial")
    dash.dash_sync_status()
    ro, _, mag = R.forward([S] * B, q, k, v, causal, scale)
    ref, mags = R.backward([S] * B, q, k, v, o, do, lse, causal, scale)
    for name, a, b, r, m in zip(("O", "dQ", "dK", "dV"), (o, *g), (xo, *xg), (ro, *ref), (mag, *mags)):
        far = (a.double() - packed(b).double()).abs() > 2 * R.bound(r, m)
        assert not far.any(), f"{name}: {int(far.sum())} of {far.numel()}"
    assert (lse.reshape(H, B, S).transpose(0, 1) - xl).abs().max() <= 1e-4
