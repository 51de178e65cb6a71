"""Measured cases of the packed, grouped-head attention and of the paged cache.

Five operators: attention over packed sequences with grouped heads (``fwd``),
its deterministic backward (``bwd``), attention of one new token per sequence
over a paged key-value cache (``decode``), writing new tokens into the cache's
pages (``write``) and copying pages inside the cache (``copy``).

``own`` selects what ``run`` calls: the plain form in elementary torch
operations, or this package's operators.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def _spread(total, parts):
    """Lengths that sum to ``total`` in the ratios ``parts`` (the last takes the rest)."""
    s = sum(parts)
    out = [max(1, total * p // s) for p in parts[:-1]]
    return out + [total - sum(out)]


def _attn(name, op, lens, hq, hkv, d, causal=True):
    case = {"op": op, "lens": ",".join(str(n) for n in lens), "hq": hq, "hkv": hkv, "d": d, "causal": causal}
    return dict(case, name=name) if name else case


def _decode(name, lens, hq, hkv, d, page):
    case = {"op": "decode", "lens": ",".join(str(n) for n in lens), "hq": hq, "hkv": hkv, "d": d, "page": page}
    return dict(case, name=name) if name else case


def _write(name, starts, news, hkv, d, page):
    case = {"op": "write", "starts": ",".join(str(n) for n in starts), "news": ",".join(str(n) for n in news),
            "hkv": hkv, "d": d, "page": page}
    return dict(case, name=name) if name else case


def _copy(name, pages, moves, hkv, d, page):
    case = {"op": "copy", "pages": pages, "moves": moves, "hkv": hkv, "d": d, "page": page}
    return dict(case, name=name) if name else case


# A document mixture of a training batch, in ratios: a few long ones and many short ones.
MIX = [1, 3, 9, 2, 31, 5, 17, 1, 7, 64, 4, 11, 2, 23, 6, 40]


def listed():
    ragged = [1 + (i * 2654435761 >> 7) % 8192 for i in range(64)]
    return [
        # a handful of short prompts in one call: latency
        _attn("fwd_short", "fwd", [1, 17, 128, 65], 8, 2, 64),
        # a training batch of 16384 tokens, hidden size 2048, documents of different lengths, grouped heads
        _attn("fwd_packed", "fwd", _spread(16384, MIX), 16, 4, 128),
        # one long prompt, as many K/V heads as Q heads
        _attn("fwd_long", "fwd", [16381], 16, 16, 128),
        # the same short prompts in training: latency
        _attn("bwd_short", "bwd", [1, 17, 128, 65], 8, 2, 64),
        # the backward of the training batch
        _attn("bwd_packed", "bwd", _spread(16384, MIX), 16, 4, 128),
        # long documents with head dimension 64
        _attn("bwd_d64", "bwd", [8192, 5000, 3191], 32, 8, 64),
        # one user's next token: latency
        _decode("decode_one", [701], 16, 4, 128, 16),
        # a serving batch: many users with one token to 8192, two with long contexts
        _decode("decode_batch", ragged + [131072, 65537], 32, 8, 128, 16),
        # the new token of every sequence of a serving batch: latency
        _write("write_step", ragged, [1] * 64, 8, 128, 16),
        # the prompts of a batch
        _write("write_prompt", [0] * 16, _spread(16384, MIX), 8, 128, 16),
        # compacting a fragmented cache
        _copy("copy_pages", 6000, 2500, 8, 128, 64),
        # forking a few sequences: each copies its last, partly filled page
        _copy("copy_fork", 512, 6, 8, 128, 16),
    ]


HEADS = [(8, 2), (16, 4), (16, 16), (32, 8), (32, 4), (8, 1), (12, 4), (4, 4)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "decode", "write", "copy"])
    d = rng.choice([64, 128])
    if op in ("fwd", "bwd"):
        hq, hkv = rng.choice(HEADS)
        total = _log(rng, 64, 12000)
        lens = []
        while sum(lens) < total and len(lens) < 64:
            lens.append(_log(rng, 1, max(1, total - sum(lens))))
        rng.shuffle(lens)
        causal = rng.random() < 0.8
        while work(_attn(None, op, lens, hq, hkv, d, causal))["flops"] > 1e12:   # no dearer than the listed ones
            lens[lens.index(max(lens))] = max(lens) * 2 // 3
        return _attn(None, op, lens, hq, hkv, d, causal)
    page = rng.choice([16, 32, 64, 24, 1])
    if op == "decode":
        hq, hkv = rng.choice(HEADS)
        top = _log(rng, 1, 100000)
        n = min(_log(rng, 1, 128), max(1, 1600000 // (top * hkv)))
        if page == 1:
            top = min(top, 20000)
        return _decode(None, [_log(rng, 1, top) for _ in range(n)], hq, hkv, d, page)
    hkv = rng.choice([1, 2, 4, 8])
    if op == "write":
        n = _log(rng, 1, 128)
        total = _log(rng, n, 16384)
        news = [max(1, total // n + rng.randint(-(total // n) // 2, total // n // 2)) for _ in range(n)]
        return _write(None, [_log(rng, 1, 4000) - 1 for _ in range(n)], news, hkv, d, page)
    pages = _log(rng, 64, 4000)
    return _copy(None, pages, _log(rng, 1, pages // 2), hkv, d, page)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _pairs(case):
    return sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _ints(case["lens"]))


def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op in ("fwd", "bwd"):
        t, hq = sum(_ints(case["lens"])), case["hq"]
        qb, kb, lse = 2 * t * hq * d, 2 * t * hkv * d, 4 * t * hq
        if op == "fwd":                                # Q, K, V in; O, LSE out
            return {"bytes": 2 * qb + 2 * kb + lse, "flops": 4 * d * hq * _pairs(case)}
        return {"bytes": 4 * qb + 4 * kb + lse, "flops": 10 * d * hq * _pairs(case)}
    if op == "decode":
        t, n, hq = sum(_ints(case["lens"])), len(_ints(case["lens"])), case["hq"]
        pages = sum(-(-x // case["page"]) for x in _ints(case["lens"]))
        return {"bytes": 4 * t * hkv * d + 4 * n * hq * d + 4 * n * hq + 4 * n + 4 * pages, "flops": 4 * t * hq * d}
    if op == "write":
        return {"bytes": 8 * sum(_ints(case["news"])) * hkv * d, "flops": 0}
    return {"bytes": 8 * case["moves"] * case["page"] * hkv * d, "flops": 0}


# ----------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _shuffled_table(g, lens, page, spare=7):
    """A page table whose pages lie in random order, and the number of pages of the cache."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, d, hkv = case["op"], case["d"], case["hkv"]
    s = {"op": op, "case": case}
    if op in ("fwd", "bwd"):
        lens, hq = _ints(case["lens"]), case["hq"]
        t = sum(lens)
        s["lens"], s["causal"], s["scale"] = lens, case["causal"], 1.0 / math.sqrt(d)
        s["q"], s["k"], s["v"] = _normal(g, t, hq, d), _normal(g, t, hkv, d), _normal(g, t, hkv, d)
        if op == "bwd":
            s["do"] = _normal(g, t, hq, d)
            s["o"], s["lse"] = _plain_fwd(s)
        if own:
            import deterministic_attention_backward_fa_gb300 as dash
            s["plan"] = dash.PackedPlan(lens, hq, hkv, d, causal=case["causal"], backward=op == "bwd")
        return s
    page = case["page"]
    if op == "decode":
        s["host_lens"] = _ints(case["lens"])
        s["lengths"] = torch.tensor(s["host_lens"], dtype=torch.int32, device=DEV)
        s["table"], n_pages = _shuffled_table(g, s["host_lens"], page)
        s["q"] = _normal(g, len(s["host_lens"]), case["hq"], d)
        s["scale"] = 1.0 / math.sqrt(d)
    elif op == "write":
        starts, news = _ints(case["starts"]), _ints(case["news"])
        s["host_starts"], s["host_news"] = starts, news
        s["table"], n_pages = _shuffled_table(g, [a + b for a, b in zip(starts, news)], page)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        s["cu_new"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["k"], s["v"] = _normal(g, cu[-1], hkv, d), _normal(g, cu[-1], hkv, d)
    else:
        n_pages = case["pages"]
        perm = torch.randperm(n_pages, generator=g, device=DEV).tolist()
        s["src"], s["dst"] = perm[:case["moves"]], perm[case["moves"]:2 * case["moves"]]
    s["k_pages"], s["v_pages"] = _normal(g, n_pages, page, hkv, d), _normal(g, n_pages, page, hkv, d)
    return s


# ------------------------------------------------------------ plain forms
def _chunks(n_rows, numel_per_row, cap=1 << 28):
    step = max(1, cap // max(1, numel_per_row))
    return [(i, min(n_rows, i + step)) for i in range(0, n_rows, step)]


def _plain_fwd(s):
    q, k, v, scale = s["q"], s["k"], s["v"], s["scale"]
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    o = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(hq, q.shape[0], dtype=torch.float32, device=DEV)
    at = 0
    for n in s["lens"]:
        kf = k[at:at + n].float().permute(1, 2, 0).unsqueeze(1)       # [hkv, 1, d, n]
        vf = v[at:at + n].float().permute(1, 0, 2).unsqueeze(1)       # [hkv, 1, n, d]
        for a, b in _chunks(n, hq * n):
            qf = q[at + a:at + b].float().permute(1, 0, 2).reshape(hkv, hq // hkv, b - a, d)
            x = torch.matmul(qf, kf) * scale
            if s["causal"]:
                rows = torch.arange(a, b, device=DEV).unsqueeze(1)
                x.masked_fill_(torch.arange(n, device=DEV).unsqueeze(0) > rows, float("-inf"))
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - m)
            total = p.sum(-1, keepdim=True)
            o[at + a:at + b] = (torch.matmul(p, vf) / total).reshape(hq, b - a, d).permute(1, 0, 2).to(torch.bfloat16)
            lse[:, at + a:at + b] = (m + torch.log(total)).reshape(hq, b - a)
        at += n
    return o, lse


def _plain_bwd(s):
    q, k, v, o, do, lse, scale = s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["scale"]
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    gr = hq // hkv
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    at = 0
    for n in s["lens"]:
        kf = k[at:at + n].float().permute(1, 0, 2).unsqueeze(1)       # [hkv, 1, n, d]
        vf = v[at:at + n].float().permute(1, 0, 2).unsqueeze(1)
        dka = torch.zeros(hkv, n, d, dtype=torch.float32, device=DEV)
        dva = torch.zeros(hkv, n, d, dtype=torch.float32, device=DEV)
        for a, b in _chunks(n, hq * n):
            shape = (hkv, gr, b - a, d)
            qf = q[at + a:at + b].float().permute(1, 0, 2).reshape(shape)
            of = o[at + a:at + b].float().permute(1, 0, 2).reshape(shape)
            gf = do[at + a:at + b].float().permute(1, 0, 2).reshape(shape)
            x = torch.matmul(qf, kf.transpose(2, 3)) * scale
            if s["causal"]:
                rows = torch.arange(a, b, device=DEV).unsqueeze(1)
                x.masked_fill_(torch.arange(n, device=DEV).unsqueeze(0) > rows, float("-inf"))
            p = torch.exp(x - lse[:, at + a:at + b].reshape(hkv, gr, b - a, 1))
            dva += torch.matmul(p.transpose(2, 3), gf).sum(1)
            ds = p * (torch.matmul(gf, vf.transpose(2, 3)) - (gf * of).sum(-1, keepdim=True))
            dka += torch.matmul(ds.transpose(2, 3), qf).sum(1)
            dq[at + a:at + b] = (torch.matmul(ds, kf) * scale).reshape(hq, b - a, d).permute(1, 0, 2).to(torch.bfloat16)
        dk[at:at + n] = (dka * scale).permute(1, 0, 2).to(torch.bfloat16)
        dv[at:at + n] = dva.permute(1, 0, 2).to(torch.bfloat16)
        at += n
    return dq, dk, dv


def _plain_decode(s):
    q, scale, page = s["q"], s["scale"], s["k_pages"].shape[1]
    hkv, d = s["k_pages"].shape[2], q.shape[2]
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    for b, n in enumerate(s["host_lens"]):
        pages = s["table"][b, :-(-n // page)].long()
        kf = s["k_pages"][pages].reshape(-1, hkv, d)[:n].float().permute(1, 2, 0)
        vf = s["v_pages"][pages].reshape(-1, hkv, d)[:n].float().permute(1, 0, 2)
        x = torch.matmul(q[b].float().reshape(hkv, -1, d), kf) * scale
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True)
        o[b] = (torch.matmul(p, vf) / total).reshape(-1, d).to(torch.bfloat16)
        lse[b] = (m + torch.log(total)).reshape(-1)
    return o, lse


def _plain_write(s):
    page = s["k_pages"].shape[1]
    seq = torch.repeat_interleave(torch.arange(len(s["host_news"]), device=DEV),
                                  (s["cu_new"][1:] - s["cu_new"][:-1]).long(), output_size=s["k"].shape[0])
    pos = torch.arange(s["k"].shape[0], device=DEV) - s["cu_new"].long()[seq] + s["starts"].long()[seq]
    where = (s["table"][seq, pos // page].long(), pos % page)
    s["k_pages"][where] = s["k"]
    s["v_pages"][where] = s["v"]
    return s["k_pages"], s["v_pages"]


def _plain_copy(s):
    src, dst = torch.tensor(s["src"], device=DEV), torch.tensor(s["dst"], device=DEV)
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]
    return s["k_pages"], s["v_pages"]


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode, "write": _plain_write,
                "copy": _plain_copy}[op](s)
    import deterministic_attention_backward_fa_gb300 as dash
    if op == "fwd":
        return dash.attn_packed_fwd(s["plan"], s["q"], s["k"], s["v"], s["scale"])
    if op == "bwd":
        return dash.attn_packed_bwd(s["plan"], s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["scale"])
    if op == "decode":
        return dash.attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["scale"])
    if op == "write":
        dash.cache_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["starts"], s["cu_new"])
    else:
        dash.cache_copy(s["k_pages"], s["v_pages"], s["src"], s["dst"])
    return s["k_pages"], s["v_pages"]


# -------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definition, sequence by sequence and head by head, in 64 bits; the cache's copies have no rounding."""
    op = case["op"]
    if op in ("write", "copy") or (op in ("fwd", "bwd") and work(case)["flops"] > 4e12):
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    q, scale = s["q"].double(), s["scale"]
    if op == "decode":
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=DEV)
        gr, page = case["hq"] // case["hkv"], case["page"]
        for b, n in enumerate(_ints(case["lens"])):
            tok = torch.arange(n, device=DEV)
            rows = s["table"][b].long()[tok // page] * page + tok % page
            for h in range(case["hq"]):
                kh = s["k_pages"].flatten(0, 1)[rows, h // gr].double()
                vh = s["v_pages"].flatten(0, 1)[rows, h // gr].double()
                x = (kh @ q[b, h]) * scale
                lse[b, h] = torch.logsumexp(x, 0)
                o[b, h] = torch.exp(x - lse[b, h]) @ vh
        return o, lse
    k, v = s["k"].double(), s["v"].double()
    gr = case["hq"] // case["hkv"]
    if op == "fwd":
        outs = (torch.empty_like(q), torch.empty(case["hq"], q.shape[0], dtype=torch.float64, device=DEV))
    else:
        o, do, stat = s["o"].double(), s["do"].double(), s["lse"].double()
        outs = (torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v))
    begin = 0
    for n in _ints(case["lens"]):
        end = begin + n
        for h in range(case["hq"]):
            kh, vh = k[begin:end, h // gr], v[begin:end, h // gr]
            for lo in range(begin, end, 4096):
                hi = min(end, lo + 4096)
                stop = hi if case["causal"] else end                   # keys past the last row are masked
                kk, vv = kh[:stop - begin], vh[:stop - begin]
                x = scale * (q[lo:hi, h] @ kk.T)
                if case["causal"]:
                    x += torch.full_like(x, float("-inf")).triu_(lo - begin + 1)
                if op == "fwd":
                    z = torch.logsumexp(x, 1)
                    outs[0][lo:hi, h] = torch.exp(x - z[:, None]) @ vv
                    outs[1][h, lo:hi] = z
                else:
                    p = torch.exp(x - stat[h, lo:hi, None])
                    gh = do[lo:hi, h]
                    delta = torch.sum(gh * o[lo:hi, h], 1)
                    ds = p * (gh @ vv.T - delta[:, None])
                    outs[0][lo:hi, h] = scale * (ds @ kk)
                    outs[1][begin:stop, h // gr] += scale * (ds.T @ q[lo:hi, h])
                    outs[2][begin:stop, h // gr] += p.T @ gh
        begin = end
    return outs
