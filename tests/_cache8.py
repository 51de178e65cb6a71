"""Plain 64-bit forms of the 8-bit paged cache, with bounds on the decode's errors.

A decode's result is rounded to bf16 (U = 2^-8 of the value).  Inside, the codes
are exact, sums and softmax are 32-bit, and Q and the weights 2^(x - m) c are
rounded.  Q: exact in f16 down to 2^-29 of its row's largest value, in two e4m3
terms down to 2^-14 and off by 2^-22 of the largest below, which EPS covers for
the standard normal rows of these tests.  Weights: in f16 by 2^-11 of themselves,
and by 2^-25 at least, counted against the largest of them, which stands at 2^-8
to 2^8 of 1: 2^-17 of the largest term at most; in two e4m3 terms by 2^-8 = U of
themselves (each term keeps 4 bits, so half a step is 2^-4 of what is left, twice),
and by 2^-14 at least (half of 2^-9, under a factor of 16) where the largest
stands at 16 at least: 2^-18 of it.  So U of each weight and 2^-17 of the largest
term for each of the n terms.  EPS = 2^-13 bounds the 32-bit arithmetic as for the
bf16 cache.
"""
import torch

import _packed as P

F64 = torch.float64
TOP = 448.0


def quantise(x):
    """Codes (as 64-bit values) and scales of rows in the last dimension, from the definition."""
    x = x.to(F64)
    scale = torch.full(x.shape[:-1], 2.0 ** -126, dtype=F64, device=x.device)
    top = x.abs().amax(-1)
    for e in range(-126, 121):
        scale = torch.where(TOP * 2.0 ** (e - 1) < top, 2.0 ** max(e, -126), scale)
    y = x / scale[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    codes = torch.round(y / step) * step  # ties to even
    finite = torch.isfinite(x).all(-1)
    return torch.where(finite[..., None], codes, 0.0), torch.where(finite, scale, float("nan"))


def values(pages, scales):
    return pages.view(torch.uint8).view(torch.float8_e4m3fn).to(F64) * scales.to(F64)[..., None]


def decode(q, pages, scales, table, lengths, scale):
    """O, LSE, magnitudes of O's terms and the terms' bound by their largest one."""
    kp, vp = (values(p, s) for p, s in zip(pages, scales))
    n_pages, page, hkv, D = kp.shape
    gr = q.shape[1] // hkv
    o, lse, mag = P.decode(q, kp, vp, table, lengths, scale)
    top = torch.zeros_like(mag)
    for b in range(q.shape[0]):
        n = max(0, min(int(lengths[b]), table.shape[1] * page))
        t = torch.arange(n, device=q.device)
        pg = table[b].long()[t // page] if n else t
        t = t[(pg >= 0) & (pg < n_pages)]
        if not len(t):
            continue
        pg = table[b].long()[t // page]
        for h in range(q.shape[1]):
            g = h // gr
            x = kp[pg, t % page, g] @ q[b, h].to(F64) * scale
            p = torch.exp(x - lse[b, h]) * scales[1][pg, t % page, g].to(F64)
            # n roundings of 2^-17 of the largest weight, each times a code of at most 448
            codes = pages[1].view(torch.uint8)[pg, t % page, g].view(torch.float8_e4m3fn).to(F64).abs()
            top[b, h] = 2.0 ** -17 * p.nan_to_num(0).amax() * codes.nan_to_num(0).sum(0)
    return o, lse, mag, top


def within(name, o, ref, mag, top):
    err = (o.to(F64) - ref).abs()
    bad = ~(err <= P.U * ref.abs() + (1 + P.U) * ((P.U + P.EPS) * mag + top) + 1e-30)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside their bound, worst {err[bad].max()}"
