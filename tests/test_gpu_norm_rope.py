"""Norms of queries and keys with their rotation on the GPU, forward and
backward, against the 64-bit form."""
import pytest
import torch

import deterministic_attention_backward_fa_gb300 as dash

import _norm_rope as R
import _packed as P

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def inputs(rows, hq, hkv, D, rot, seed=1, most=300, weight=torch.bfloat16):
    """Q, K, their outputs' gradients, weights, table and positions; all but the weights parts of larger tensors."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    fused = torch.full((rows + 1, hq + 2 * hkv + 1, D), NAN, dtype=torch.bfloat16, device="cuda")
    parts = [fused[:rows, :hq], fused[:rows, hq:hq + hkv]]
    for i, t in enumerate(parts):
        t.copy_(P.normal(seed + i, *t.shape) * 3)
    heads_first = [torch.full((h, rows, D), NAN, dtype=torch.bfloat16, device="cuda").transpose(0, 1) for h in (hq, hkv)]
    for i, t in enumerate(heads_first):
        t.copy_(P.normal(seed + 5 + i, *t.shape))
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(weight) for _ in range(2)]
    positions = torch.randint(0, most, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return parts, heads_first, w, dash.rope_table(most, rot), positions


def check(parts, grads, w, rope, positions, eps, pairs, z, back):
    for i, name in enumerate("qk"):
        R.within(name, z[i], *R.forward(parts[i], w[i], rope, positions, eps, pairs))
        (dx, dw), (mx, mw) = R.backward(parts[i], grads[i], w[i], rope, positions, eps, pairs)
        R.within("d" + name, back[i], dx, mx)
        # fp32, its own rounding 2^-24; a chain of the sum has a lane's rows and heads (at most 32 here), two steps
        # across lanes, eight warps and 32 + 32 parts: 106 roundings more on each term, below 2^-17 with EPS
        R.within("weight of " + name, back[2 + i], dw, mw, 2.0 ** -24, 2.0 ** -17)


CASES = [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (37, 5, 1, 128, 32), (1, 32, 8, 128, 128), (64, 16, 4, 64, 48),
         (300, 3, 3, 64, 8), (19, 40, 40, 128, 120), (2, 1, 7, 64, 16),
         (700, 5, 2, 128, 64), (4000, 3, 1, 64, 32), (3, 1000, 30, 128, 128)]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rows,hq,hkv,D,rot", CASES)
def test_against_64_bits(rows, hq, hkv, D, rot, pairs):
    for weight in (torch.bfloat16, torch.float32):
        parts, grads, w, rope, positions = inputs(rows, hq, hkv, D, rot, weight=weight)
        eps = 1e-5
        z = dash.qk_norm_rope(*parts, *w, rope, positions, eps, pairs)
        back = dash.qk_norm_rope_bwd(*parts, *grads, *w, rope, positions, eps, pairs)
        dash.dash_sync_status()
        check(parts, grads, w, rope, positions, eps, pairs, z, back)
        again = dash.qk_norm_rope(*parts, *w, rope, positions, eps, pairs)
        again += dash.qk_norm_rope_bwd(*parts, *grads, *w, rope, positions, eps, pairs)
        assert all(torch.equal(a, b) for a, b in zip((*z, *back), again))


def test_many_rows():
    # more rows than CTAs have warps: rows are taken in turn
    rows, hq, hkv, D = 12000, 3, 1, 64
    parts, grads, w, rope, positions = inputs(rows, hq, hkv, D, 64)
    z = dash.qk_norm_rope(*parts, *w, rope, positions)
    back = dash.qk_norm_rope_bwd(*parts, *grads, *w, rope, positions)
    dash.dash_sync_status()
    check(parts, grads, w, rope, positions, 1e-6, False, z, back)


def test_no_rows_and_zero_rows():
    parts, grads, w, rope, positions = inputs(4, 2, 1, 64, 64)
    none = [t[:0] for t in parts]
    assert [t.shape[0] for t in dash.qk_norm_rope(*none, *w, rope, positions[:0])] == [0, 0]
    back = dash.qk_norm_rope_bwd(*none, *none, *w, rope, positions[:0])
    assert not back[2].any() and not back[3].any() and back[0].shape == (0, 2, 64)
    # a row of zeros has the norm eps gives it: it stays zero, its gradient is finite
    zero = [torch.zeros_like(t) for t in parts]
    assert not any(t.any() for t in dash.qk_norm_rope(*zero, *w, rope, positions))
    back = dash.qk_norm_rope_bwd(*zero, *grads, *w, rope, positions)
    check(zero, grads, w, rope, positions, 1e-6, False, zero, back)
    dash.dash_sync_status()


def test_in_place_and_heads_first():
    parts, grads, w, rope, positions = inputs(50, 6, 2, 128, 128)
    want = dash.qk_norm_rope(*parts, *w, rope, positions)
    wback = dash.qk_norm_rope_bwd(*parts, *grads, *w, rope, positions)
    # gradients first, over their inputs, then the rows themselves
    ws = torch.empty(dash.dash_norm_rope_workspace(50, 6, 2, 128), dtype=torch.uint8, device="cuda")
    dws = [torch.empty(128, device="cuda") for _ in range(2)]
    dash.dash_qk_norm_rope_bwd(*parts, *grads, *grads, *w, *dws, rope, positions, 1e-6, ws)
    dash.dash_qk_norm_rope(*parts, *parts, *w, rope, positions, 1e-6)
    for got, ref in zip((*parts, *grads, *dws), (*want, *wback)):
        assert torch.equal(got, ref)


def test_positions_outside_the_table_are_reported():
    parts, grads, w, rope, positions = inputs(9, 4, 2, 64, 32, most=20)
    for bad in (-1, 20, 2**31 - 1, -2**31):
        positions[4] = bad
        ok = torch.arange(9, device="cuda") != 4
        z = dash.qk_norm_rope(*parts, *w, rope, positions)
        with pytest.raises(dash.DashError, match="rotation table"):
            dash.dash_sync_status()
        back = dash.qk_norm_rope_bwd(*parts, *grads, *w, rope, positions)
        with pytest.raises(dash.DashError, match="rotation table"):
            dash.dash_sync_status()
        dash.dash_sync_status()  # cleared
        for i in range(2):
            ref, mag = R.forward(parts[i][ok], w[i], rope, positions[ok], 1e-6, False)
            R.within("rows", z[i][ok], ref, mag)
            assert z[i][4].isnan().all() and back[i][4].isnan().all() and back[2 + i].isnan().all()
            assert back[i][ok].isfinite().all()


def test_captured_streams_and_two_calls_at_once():
    parts, grads, w, rope, positions = inputs(200, 8, 2, 128, 128)
    call = lambda **kw: (*dash.qk_norm_rope(*parts, *w, rope, positions, **kw),
                         *dash.qk_norm_rope_bwd(*parts, *grads, *w, rope, positions, **kw))
    want = call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [call(stream=s) for s in streams for _ in range(3)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for seed in (7, 8):  # replayed on other inputs
        for i, t in enumerate(parts):
            t.copy_(P.normal(seed + i, *t.shape))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, call()))
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


def test_large_offsets():
    # rows further apart than 2^31 elements
    rows, hq, D = 3, 2, 64
    step = 2**30 + 64
    big = torch.empty((rows - 1) * step + 4 * D, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((rows, hq, D), (step, D, 1))
    k = big.as_strided((rows, hq, D), (step, D, 1), 2 * D)
    q.copy_(P.normal(1, rows, hq, D))
    k.copy_(P.normal(2, rows, hq, D))
    w = [torch.ones(D, dtype=torch.bfloat16, device="cuda")] * 2
    rope, positions = dash.rope_table(10, 64), i32([0, 5, 9])
    z = dash.qk_norm_rope(q, k, *w, rope, positions)
    back = dash.qk_norm_rope_bwd(q, k, q, k, *w, rope, positions)
    check((q, k), (q, k), w, rope, positions, 1e-6, False, z, back)


def test_refusals():
    parts, grads, w, rope, positions = inputs(4, 4, 2, 64, 64)
    (q, k), call = parts, dash.qk_norm_rope
    for bad in (lambda: call(q.float(), k, *w, rope, positions), lambda: call(q, k[:3], *w, rope, positions),
                lambda: call(q, k, w[0], w[1].float(), rope, positions), lambda: call(q, k, w[0][:32], w[1], rope, positions),
                lambda: call(q, k, w[0].half(), w[1].half(), rope, positions),
                lambda: call(q, k, *w, rope.double(), positions), lambda: call(q, k, *w, rope[:, :32], positions),
                lambda: call(q, k, *w, rope, positions.long()), lambda: call(q, k, *w, rope, positions[:2]),
                lambda: call(q, k, *w, rope.cpu(), positions), lambda: call(q[..., ::2], k, *w, rope, positions),
                lambda: dash.qk_norm_rope_bwd(q, k, grads[0][:2], grads[1], *w, rope, positions),
                lambda: dash.qk_norm_rope_bwd(q, k, grads[1], grads[0], *w, rope, positions)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dash.DashError, match="multiple of 8"):
        call(q, k, *w, rope[:, :12].contiguous(), positions)
    with pytest.raises(dash.DashError, match="head dim"):
        call(q[..., :32], k[..., :32], w[0][:32], w[1][:32], rope[:, :32].contiguous(), positions)


def test_norms_cache_and_attention_together():
    # a prompt's projection goes through the norms into the packed forward and the cache; the decode of its last token
    # gives the forward's last row, and the gradients go back through both backwards
    hq, hkv, D, lens = 8, 2, 64, [70, 33]
    rows = sum(lens)
    fused = P.normal(3, rows, hq + 2 * hkv, D)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    w = [(1 + 0.2 * P.normal(11 + i, D).float()).to(torch.bfloat16) for i in range(2)]
    rope = dash.rope_table(100, D)
    positions = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens])
    plan = dash.PackedPlan(lens, hq, hkv, D, backward=True)
    qn, kn = dash.qk_norm_rope(q, k, *w, rope, positions)
    o, lse = dash.attn_packed_fwd(plan, qn, kn, v)
    do = P.normal(4, rows, hq, D)
    dqn, dkn, dv = dash.attn_packed_bwd(plan, qn, kn, v, o, do, lse)
    dq, dk, dwq, dwk = dash.qk_norm_rope_bwd(q, k, dqn, dkn, *w, rope, positions)
    kp, vp = (torch.zeros(12, 16, hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, cu = torch.arange(12, dtype=torch.int32, device="cuda").reshape(2, 6), i32([0, lens[0], rows])
    dash.cache_write(kn, v, kp, vp, table, i32([0, 0]), cu)
    last = torch.tensor([lens[0] - 1, rows - 1], device="cuda")
    od, _ = dash.attn_decode(qn[last], kp, vp, table, i32(lens))
    dash.dash_sync_status()
    ro, rl, mag = P.decode(qn[last], kp, vp, table, lens, D ** -0.5)
    P.within("decode", od, ro, mag)
    P.within("forward", o[last], ro, mag)
    for x, dz, dx, dw, wt in ((q, dqn, dq, dwq, w[0]), (k, dkn, dk, dwk, w[1])):
        (rx, rw), (mx, mw) = R.backward(x, dz, wt, rope, positions, 1e-6, False)
        R.within("dx", dx, rx, mx)
        R.within("dw", dw, rw, mw, 2.0 ** -24, 2.0 ** -17)
