"""Measured cases of the operators around the packed attention and the paged cache.

Six passes: the norms of queries and keys with their rotation by position
(``norm``) and its backward (``norm_bwd``), writing tokens into an 8-bit paged
cache (``write8``), reading them back (``read8``), attention of one new token
per sequence over that cache (``decode8``), and the same over a bf16 cache for
a batch whose sequences begin with the same tokens (``shared``).

``own`` selects what ``run`` calls: the plain form in elementary torch
operations, or this package's operators.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TOP = 448.0          # the largest 8-bit value (e4m3)


# ------------------------------------------------------------------ cases
def _spread(total, parts):
    """Lengths that sum to ``total`` in the ratios ``parts`` (the last takes the rest)."""
    s = sum(parts)
    out = [max(1, total * p // s) for p in parts[:-1]]
    return out + [total - sum(out)]


def _text(values):
    return ",".join(str(n) for n in values)


def _norm(op, lens, first, hq, hkv, d, rot, pairs):
    """``first``: the position of each sequence's first row; ``pairs``: neighbours rotate together, else halves."""
    return {"op": op, "lens": _text(lens), "first": _text(first), "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "pairs": pairs}


def _rows8(op, starts, news, hkv, d, page):
    return {"op": op, "starts": _text(starts), "news": _text(news), "hkv": hkv, "d": d, "page": page}


def _decode8(lens, hq, hkv, d, page):
    return {"op": "decode8", "lens": _text(lens), "hq": hq, "hkv": hkv, "d": d, "page": page}


def _shared(prefix, tails, hq, hkv, d, page):
    return {"op": "shared", "prefix": prefix, "tails": _text(tails), "hq": hq, "hkv": hkv, "d": d, "page": page}


# A document mixture of a training batch, in ratios: a few long ones and many short ones.
MIX = [1, 3, 9, 2, 31, 5, 17, 1, 7, 64, 4, 11, 2, 23, 6, 40]


def listed():
    ragged = [1 + (i * 2654435761 >> 7) % 8192 for i in range(64)]
    tails = [(i * 2654435761 >> 9) % 1024 for i in range(64)]
    return [
        # the new tokens of a serving batch, far into their sequences: latency
        dict(_norm("norm", [1] * 64, [16 * n for n in ragged], 32, 8, 128, 128, False), name="norm_step"),
        # a training batch of 16384 tokens, hidden size 2048, documents of different lengths
        dict(_norm("norm", _spread(16384, MIX), [0] * 16, 16, 4, 128, 128, False), name="norm_packed"),
        # a handful of short prompts in training: latency
        dict(_norm("norm_bwd", [1, 17, 128, 65], [0] * 4, 8, 2, 64, 64, False), name="norm_bwd_short"),
        # the backward of the training batch
        dict(_norm("norm_bwd", _spread(16384, MIX), [0] * 16, 16, 4, 128, 128, False), name="norm_bwd_packed"),
        # the new token of every sequence of a serving batch: latency
        dict(_rows8("write8", ragged, [1] * 64, 8, 128, 16), name="write8_step"),
        # the prompts of a batch
        dict(_rows8("write8", [0] * 16, _spread(16384, MIX), 8, 128, 16), name="write8_prompt"),
        # the context of a few short chats, for their next chunk of prompt: latency
        dict(_rows8("read8", [0, 0, 64, 0], [300, 41, 129, 7], 4, 64, 16), name="read8_chats"),
        # the context of a batch of long prompts
        dict(_rows8("read8", [0] * 16, _spread(16384, MIX), 8, 128, 16), name="read8_prompt"),
        # one user's next token: latency
        dict(_decode8([701], 16, 4, 128, 16), name="decode8_one"),
        # a serving batch: many users with one token to 8192, two with long contexts
        dict(_decode8(ragged + [131072, 65537], 32, 8, 128, 16), name="decode8_batch"),
        # four samples of one prompt, a few tokens in: latency
        dict(_shared(1501, [0, 3, 17, 40], 16, 4, 128, 16), name="shared_samples"),
        # a serving batch behind one long document
        dict(_shared(32000, tails, 32, 8, 128, 16), name="shared_batch"),
    ]


HEADS = [(8, 2), (16, 4), (16, 16), (32, 8), (32, 4), (8, 1), (12, 4), (4, 4), (16, 1)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "write8", "read8", "decode8", "decode8", "shared", "shared"])
    d = rng.choice([64, 128])
    hq, hkv = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 24, 1])
    if op in ("norm", "norm_bwd"):
        total = _log(rng, 1, 10000)
        lens = []
        while sum(lens) < total and len(lens) < 64:
            lens.append(_log(rng, 1, max(1, total - sum(lens))))
        rng.shuffle(lens)
        first = [_log(rng, 1, 40000) - 1 if rng.random() < 0.3 else 0 for _ in lens]
        return _norm(op, lens, first, hq, hkv, d, rng.choice([d, d, d // 2, 32, 48]), rng.random() < 0.3)
    if op in ("write8", "read8"):
        hkv = rng.choice([1, 2, 4, 8])
        n = _log(rng, 1, 128)
        total = _log(rng, n, 16384)
        news = [max(1, total // n + rng.randint(-(total // n) // 2, total // n // 2)) for _ in range(n)]
        while sum(news) > 16384:
            news[news.index(max(news))] //= 2
        return _rows8(op, [_log(rng, 1, 4000) - 1 for _ in range(n)], news, hkv, d, page)
    if op == "decode8":
        top = _log(rng, 1, 100000)
        n = min(_log(rng, 1, 128), max(1, 1600000 // (top * hkv)))
        if page == 1:
            top = min(top, 20000)
        return _decode8([_log(rng, 1, top) for _ in range(n)], hq, hkv, d, page)
    prefix = _log(rng, 100, 30000)
    n = min(_log(rng, 2, 128), max(2, 1900000 // (prefix * hq) * 32))
    top = _log(rng, 1, max(1, min(4000, 400000 // (n * hkv))))
    return _shared(prefix, [_log(rng, 1, top) - 1 for _ in range(n)], hq, hkv, d, page)


def _ints(text):
    return [int(x) for x in text.split(",")]


def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    if op in ("norm", "norm_bwd"):
        t, h = sum(_ints(case["lens"])), case["hq"] + hkv
        rows = set().union(*(range(f, f + n) for n, f in zip(_ints(case["lens"]), _ints(case["first"]))))
        moved = 4 * t + 4 * len(rows) * case["rot"] + 4 * d      # positions, the angles of each, two weights
        if op == "norm":
            return {"bytes": 4 * t * h * d + moved, "flops": 9 * t * h * d}
        return {"bytes": 6 * t * h * d + moved + 8 * d, "flops": 20 * t * h * d}
    if op in ("write8", "read8"):                      # K and V: 2 bytes and 1 a value, a scale per row
        return {"bytes": sum(_ints(case["news"])) * hkv * 2 * (3 * d + 4), "flops": 0}
    hq, page = case["hq"], case["page"]
    if op == "decode8":
        lens = _ints(case["lens"])
        t, n = sum(lens), len(lens)
        pages = sum(-(-x // page) for x in lens)
        return {"bytes": 2 * t * hkv * (d + 4) + 4 * n * hq * d + 4 * n * hq + 4 * n + 4 * pages,
                "flops": 4 * t * hq * d}
    tails = _ints(case["tails"])
    t, n, prefix = sum(tails), len(tails), case["prefix"]
    pages = -(-prefix // page) + sum(-(-(prefix + x) // page) - prefix // page for x in tails)
    return {"bytes": 4 * (prefix + t) * hkv * d + 4 * n * hq * d + 4 * n * hq + 4 * n + 4 * pages,
            "flops": 4 * (prefix * n + t) * hq * d}


# ----------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _keys(g, rows, hkv, d):
    """Keys as models have them: a few channels of each head are much larger than the others."""
    gain = torch.ones(hkv, d, device=DEV)
    at = torch.randint(0, d, (hkv, 3), generator=g, device=DEV)
    gain.scatter_(1, at, 6.0)
    return (_normal(g, rows, hkv, d) * gain).to(torch.bfloat16)


def _table(g, lens, page, spare=7):
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


def _codes(x):
    """e4m3 values and power-of-two scales, the smallest with |x| <= 448 scale, of rows in the last dimension."""
    top = x.float().abs().amax(-1)
    m, e = torch.frexp(top)                              # top = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    scale = torch.ldexp(torch.ones_like(top), e)
    return (x.float() / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _cache8(g, n_pages, page, hkv, d):
    """A filled 8-bit cache: pages [n_pages, page, hkv, d] and scales [n_pages, page, hkv], a head's side by side."""
    out = []
    for keys in (True, False):
        x = _keys(g, n_pages * page, hkv, d) if keys else _normal(g, n_pages * page, hkv, d).to(torch.bfloat16)
        codes, scale = _codes(x)
        out.append(codes.reshape(n_pages, page, hkv, d))
        out.append(scale.reshape(n_pages, page, hkv).transpose(1, 2).contiguous().transpose(1, 2))
    return {"k_pages": out[0], "k_scales": out[1], "v_pages": out[2], "v_scales": out[3]}


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pieces(lens, width):
    """Ranges of up to ``width`` tokens that cover the sequences: sequence, first token, tokens."""
    got = [(b, a, min(width, n - a)) for b, n in enumerate(lens) for a in range(0, n, width)] or [(0, 0, 0)]
    return torch.tensor(got, dtype=torch.int64, device=DEV).unbind(1)


def _width(lens):
    mean = max(1, sum(lens) // max(1, len(lens)))
    return min(1024, max(32, 1 << (mean - 1).bit_length()))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, d, hkv = case["op"], case["d"], case["hkv"]
    s = {"op": op}
    if op in ("norm", "norm_bwd"):
        lens, first, hq, rot = _ints(case["lens"]), _ints(case["first"]), case["hq"], case["rot"]
        s["positions"] = torch.cat([torch.arange(f, f + n, dtype=torch.int32, device=DEV)
                                    for n, f in zip(lens, first)])
        most = max(n + f for n, f in zip(lens, first))
        angle = (torch.arange(most, device=DEV, dtype=torch.float64).unsqueeze(1) *
                 torch.pow(10000.0, -2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot))
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["pairs"] = case["pairs"]
        t = sum(lens)
        fused = _normal(g, t, hq + 2 * hkv, d).mul_(1.5).to(torch.bfloat16)      # a projection's Q, K and V
        s["q"], s["k"] = fused[:, :hq], fused[:, hq:hq + hkv]
        s["wq"], s["wk"] = ((1 + 0.2 * _normal(g, d)).to(torch.bfloat16) for _ in range(2))
        if op == "norm_bwd":
            s["dq"], s["dk"] = (_normal(g, t, h, d).to(torch.bfloat16) for h in (hq, hkv))
        return s
    page = case["page"]
    if op in ("write8", "read8"):
        starts, news = _ints(case["starts"]), _ints(case["news"])
        s["table"], n_pages = _table(g, [a + b for a, b in zip(starts, news)], page)
        s["starts"] = _i32(starts)
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        s["cu"], s["rows"] = _i32(cu), cu[-1]
        s.update(_cache8(g, n_pages, page, hkv, d))
        if op == "write8":
            s["k"], s["v"] = _keys(g, cu[-1], hkv, d), _normal(g, cu[-1], hkv, d).to(torch.bfloat16)
        return s
    s["scale"] = 1.0 / math.sqrt(d)
    if op == "decode8":
        lens = tails = _ints(case["lens"])
        s["table"], n_pages = _table(g, lens, page)
        s.update(_cache8(g, n_pages, page, hkv, d))
        s["first"] = 0
    else:
        # every sequence's row of the table begins with the prefix's pages; a page that the prefix fills in part is
        # the sequence's own copy
        prefix, tails = case["prefix"], _ints(case["tails"])
        lens = [prefix + n for n in tails]
        full = prefix // page
        s["table"], n_pages = _table(g, [prefix + 1] + [n - full * page for n in lens], page)
        own_pages, width = s["table"][1:], max(-(-n // page) for n in lens)
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
        table[:, :full] = s["table"][0, :full]
        table[:, full:] = own_pages[:, :width - full]
        s["table"] = table
        s["k_pages"] = _keys(g, n_pages * page, hkv, d).reshape(n_pages, page, hkv, d)
        s["v_pages"] = _normal(g, n_pages, page, hkv, d).to(torch.bfloat16)
        if prefix % page:
            last = table[:, full].long()
            for p in (s["k_pages"], s["v_pages"]):
                p[last, :prefix % page] = p[last[0], :prefix % page].clone()
        s["first"] = prefix
    s["lengths"] = _i32(lens)
    s["q"] = _normal(g, len(lens), case["hq"], d).to(torch.bfloat16)
    s["pieces"] = _pieces(tails, _width(tails))
    s["width"] = _width(tails)
    return s


# ------------------------------------------------------------ plain forms
def _halves(x, pairs):
    return (x[..., 0::2], x[..., 1::2]) if pairs else x.chunk(2, -1)


def _whole(a, b, pairs):
    return torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)


def _rotate(x, s, sign):
    rot = s["rope"].shape[1]
    cos, sin = s["rope"][s["positions"].long()].unsqueeze(1).chunk(2, -1)
    a, b = _halves(x[..., :rot], s["pairs"])
    return torch.cat([_whole(a * cos - sign * b * sin, b * cos + sign * a * sin, s["pairs"]), x[..., rot:]], -1)


def _plain_norm_of(x, w, s):
    xf = x.float()
    n = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    return _rotate(n * w.float(), s, 1.0).to(torch.bfloat16)


def _plain_norm_bwd_of(x, dz, w, s):
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    n, grad = xf * r, _rotate(dz.float(), s, -1.0)
    a = grad * w.float()
    dx = r * (a - n * (a * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (grad * n).double().sum((0, 1)).float()


def _plain_norm(s):
    return _plain_norm_of(s["q"], s["wq"], s), _plain_norm_of(s["k"], s["wk"], s)


def _plain_norm_bwd(s):
    dq, dwq = _plain_norm_bwd_of(s["q"], s["dq"], s["wq"], s)
    dk, dwk = _plain_norm_bwd_of(s["k"], s["dk"], s["wk"], s)
    return dq, dk, dwq, dwk


def _where(s):
    """Page and place of every token of the ranges starts, cu."""
    seq = torch.repeat_interleave(torch.arange(s["starts"].shape[0], device=DEV), (s["cu"][1:] - s["cu"][:-1]).long(),
                                  output_size=s["rows"])
    pos = torch.arange(s["rows"], device=DEV) - s["cu"].long()[seq] + s["starts"].long()[seq]
    page = s["k_pages"].shape[1]
    return s["table"][seq, pos // page].long(), pos % page


def _plain_write8_of(x, pages, scales, where):
    codes, scale = _codes(x)
    pages.view(torch.uint8)[where] = codes.view(torch.uint8)
    scales[where] = scale


def _plain_write8(s):
    where = _where(s)
    _plain_write8_of(s["k"], s["k_pages"], s["k_scales"], where)
    _plain_write8_of(s["v"], s["v_pages"], s["v_scales"], where)
    return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]


def _values(s, name, where):
    """The cache's values at (page, place), in 32 bits."""
    pages = s[name + "_pages"]
    if pages.dtype != torch.float8_e4m3fn:
        return pages[where].float()
    return pages.view(torch.uint8)[where].view(pages.dtype).float() * s[name + "_scales"][where].unsqueeze(-1)


def _plain_read8(s):
    where = _where(s)
    return _values(s, "k", where).to(torch.bfloat16), _values(s, "v", where).to(torch.bfloat16)


def _plain_decode(s):
    """Attention piece by piece of the tails, and of the prefix at once, joined by the pieces' maxima and sums."""
    q, scale, page, first = s["q"].float(), s["scale"], s["k_pages"].shape[1], s["first"]
    B, hq, d = q.shape
    hkv = s["k_pages"].shape[2]
    q = q.reshape(B, hkv, hq // hkv, d)
    seq, begin, count = s["pieces"]
    at = torch.arange(s["width"], device=DEV)
    inside = at < count.unsqueeze(1)
    pos = first + begin.unsqueeze(1) + torch.where(inside, at, 0)
    where = (s["table"][seq.unsqueeze(1), (pos // page).clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0),
             pos % page)
    k, v = (_values(s, name, where).permute(0, 2, 1, 3) for name in ("k", "v"))          # [pieces, hkv, width, d]
    x = torch.matmul(q[seq], k.transpose(2, 3)) * scale
    x.masked_fill_(~inside[:, None, None], float("-inf"))
    m = x.amax(-1)
    p = torch.exp(x - m.clamp(min=-1e30).unsqueeze(-1))
    top = torch.full((B, hkv, hq // hkv), float("-inf"), device=DEV)
    top = top.scatter_reduce(0, seq[:, None, None].expand_as(m), m, "amax")
    if first:
        t = torch.arange(first, device=DEV)
        where = (s["table"][0, t // page].long(), t % page)
        k0, v0 = (_values(s, name, where).permute(1, 0, 2) for name in ("k", "v"))       # [hkv, prefix, d]
        q0 = q.permute(1, 0, 2, 3).reshape(hkv, -1, d)
        x0 = torch.matmul(q0, k0.transpose(1, 2)) * scale
        m0 = x0.amax(-1, keepdim=True)
        x0 = torch.exp(x0 - m0)
        shape = (hkv, B, hq // hkv)
        o0 = torch.matmul(x0, v0).reshape(*shape, d).transpose(0, 1)
        l0, m0 = (y.reshape(shape).transpose(0, 1) for y in (x0.sum(-1), m0))
        top = torch.maximum(top, m0)
    w = torch.exp(m - top[seq])
    total = torch.zeros_like(top).index_add_(0, seq, p.sum(-1) * w)
    o = torch.zeros_like(q).index_add_(0, seq, torch.matmul(p, v) * w.unsqueeze(-1))
    if first:
        w0 = torch.exp(m0 - top)
        total, o = total + l0 * w0, o + o0 * w0.unsqueeze(-1)
    return (o / total.unsqueeze(-1)).reshape(B, hq, d).to(torch.bfloat16), (top + torch.log(total)).reshape(B, hq)


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "write8": _plain_write8, "read8": _plain_read8,
                "decode8": _plain_decode, "shared": _plain_decode}[op](s)
    import deterministic_attention_backward_fa_gb300 as dash
    if op == "norm":
        return dash.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rope"], s["positions"], EPS, s["pairs"])
    if op == "norm_bwd":
        return dash.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], s["rope"], s["positions"],
                                     EPS, s["pairs"])
    if op == "write8":
        dash.cache_write_fp8(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                             s["starts"], s["cu"])
        return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    if op == "read8":
        return dash.cache_read_fp8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"], s["starts"],
                                   s["cu"], s["rows"])
    if op == "decode8":
        return dash.attn_decode_fp8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                                    s["lengths"], s["scale"])
    return dash.attn_decode_shared(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["first"],
                                   s["scale"])


# -------------------------------------------------------------- 64 bits
def _exact_norm(case, s):
    """Rows as complex numbers turned by e^(i angle); the backward as the transposed Jacobian, term by term."""
    d, rot, outs, sums = case["d"], case["rot"], [], []
    turn = torch.complex(*(t.double() for t in s["rope"][s["positions"].long()].split(rot // 2, 1)))[:, None]

    def rotated(y, by):
        head = y[..., :rot]
        if s["pairs"]:
            z = torch.view_as_complex(head.unflatten(-1, (rot // 2, 2)).contiguous()) * by
            return torch.cat([torch.view_as_real(z).flatten(-2), y[..., rot:]], -1)
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * by
        return torch.cat([z.real, z.imag, y[..., rot:]], -1)

    for x, w, dz in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.double(), w.double()
        rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + EPS) ** 0.5
        if dz is None:
            outs.append(rotated(x / rms * w, turn))
            continue
        back = rotated(dz.double(), turn.conj())
        sums.append(torch.einsum("rhd,rhd->d", back, x / rms))
        u = back * w
        outs.append(u / rms - x * torch.einsum("rhd,rhd->rh", u, x)[..., None] / (d * rms ** 3))
    return (*outs, *sums)


def _exact_codes(x):
    """The nearest e4m3 values (ties to even; steps of 2^-9 below 2^-6) of rows over their scales."""
    x = x.double()
    top = x.abs().amax(-1).clamp(min=TOP * 2.0 ** -126)
    scale = torch.exp2(torch.ceil(torch.log2(top / TOP) - 1e-12))
    y = x / scale[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, scale


def _exact_rows8(case, s):
    starts, cu, page = s["starts"].tolist(), s["cu"].tolist(), case["page"]
    if case["op"] == "write8":
        kp, vp, ks, vs = (s[n].double() for n in ("k_pages", "v_pages", "k_scales", "v_scales"))
        fresh = [(kp, ks, *_exact_codes(s["k"])), (vp, vs, *_exact_codes(s["v"]))]
        for b, first in enumerate(starts):
            t = torch.arange(first, first + cu[b + 1] - cu[b], device=DEV)
            at = s["table"][b].long()[t // page] * page + t % page
            for pages, scales, codes, scale in fresh:
                pages.flatten(0, 1)[at] = codes[cu[b]:cu[b + 1]]
                scales[at // page, at % page] = scale[cu[b]:cu[b + 1]]
        return kp, vp, ks, vs
    outs = [torch.empty(s["rows"], case["hkv"], case["d"], dtype=torch.float64, device=DEV) for _ in range(2)]
    for b, first in enumerate(starts):
        t = torch.arange(first, first + cu[b + 1] - cu[b], device=DEV)
        pg = s["table"][b].long()[t // page]
        for out, n in zip(outs, "kv"):
            pages, scales = s[n + "_pages"].view(torch.uint8), s[n + "_scales"]
            codes = pages[pg, t % page].view(torch.float8_e4m3fn).double()
            out[cu[b]:cu[b + 1]] = codes * scales[pg, t % page].double()[..., None]
    return tuple(outs)


def _exact_decode(case, s):
    """Sequence by sequence and K/V head by K/V head."""
    q, page, gr = s["q"].double(), case["page"], case["hq"] // case["hkv"]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lengths"].tolist()):
        t = torch.arange(n, device=DEV)
        at = (s["table"][b].long()[t // page], t % page)
        for h in range(case["hkv"]):
            kh, vh = s["k_pages"], s["v_pages"]
            if case["op"] == "decode8":
                kh, vh = (p.view(torch.uint8)[at[0], at[1], h].view(torch.float8_e4m3fn).double() for p in (kh, vh))
                kh, vh = kh * s["k_scales"][at[0], at[1], h][:, None], vh * s["v_scales"][at[0], at[1], h][:, None]
            else:
                kh, vh = kh[at[0], at[1], h].double(), vh[at[0], at[1], h].double()
            heads = slice(h * gr, (h + 1) * gr)
            x = s["scale"] * (q[b, heads] @ kh.T)
            lse[b, heads] = torch.logsumexp(x, 1)
            o[b, heads] = torch.softmax(x, 1) @ vh
    return o, lse


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(case, s)
    return (_exact_rows8 if case["op"] in ("write8", "read8") else _exact_decode)(case, s)
