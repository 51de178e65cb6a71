"""Plain 64-bit forms of the packed attention and the paged cache, with bounds
on the kernels' errors.

The kernels form products exactly and sum in 32 bits; what rounds to bf16 is the
second operand of a product (P, dS) and the result.  A rounding to bf16 is off
by at most U = 2^-8 of the value, so an output sum_j w_j x_j whose weights w were
rounded is off by at most U sum |w_j x_j|, and its own rounding adds U of the
(slightly wrong) result.  EPS bounds what the 32-bit arithmetic adds, relative
to the same sums of magnitudes: scores of standard normal rows, a few hundred
32-bit roundings (2^-24 each) and the exponential's 2^-22 stay below 2^-13.
"""
import torch

U = 2.0 ** -8
EPS = 2.0 ** -13
F64 = torch.float64


def bound(ref, mag):
    return U * ref.abs() + (U * (1 + U) + EPS) * mag + 1e-30


def within(name, x, ref, mag):
    err = (x.to(F64) - ref).abs()
    bad = ~(err <= bound(ref, mag))
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside their bound, worst error "
                           f"{err[bad].max() if torch.isfinite(err[bad]).any() else 'nan'}")


def forward(lens, q, k, v, causal, scale):
    """O, LSE and the magnitudes sum_j p_j |v_j| of O, in 64 bits."""
    gr = q.shape[1] // k.shape[1]
    o, mag = torch.zeros_like(q, dtype=F64), torch.zeros_like(q, dtype=F64)
    lse = torch.zeros(q.shape[1], q.shape[0], dtype=F64, device=q.device)
    at = 0
    for n in lens:
        for h in range(q.shape[1]):
            qq, kk, vv = (t[at:at + n, x].to(F64) for t, x in ((q, h), (k, h // gr), (v, h // gr)))
            x = qq @ kk.T * scale
            if causal:
                x = x.masked_fill(torch.ones_like(x, dtype=torch.bool).triu(1), float("-inf"))
            if n:
                lse[h, at:at + n] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[h, at:at + n, None])
            o[at:at + n, h], mag[at:at + n, h] = p @ vv, p @ vv.abs()
        at += n
    return o, lse, mag


def backward(lens, q, k, v, o, do, lse, causal, scale):
    """dQ, dK, dV and the magnitudes of their sums, in 64 bits."""
    gr = q.shape[1] // k.shape[1]
    outs = [torch.zeros_like(t, dtype=F64) for t in (q, k, v, q, k, v)]
    dq, dk, dv, mq, mk, mv = outs
    at = 0
    for n in lens:
        s = slice(at, at + n)
        for h in range(q.shape[1]):
            g = h // gr
            qq, kk, vv, oo, gg = (t[s, x].to(F64) for t, x in ((q, h), (k, g), (v, g), (o, h), (do, h)))
            x = qq @ kk.T * scale - lse[h, s].to(F64)[:, None]
            if causal:
                x = x.masked_fill(torch.ones_like(x, dtype=torch.bool).triu(1), float("-inf"))
            p = torch.exp(x)
            delta, dp = (gg * oo).sum(1, keepdim=True), gg @ vv.T
            ds = p * (dp - delta)
            # dP and delta are 32-bit sums of D products: their error goes with the products' magnitudes
            noise = p * (gg.abs() @ vv.abs().T + (gg * oo).abs().sum(1, keepdim=True)) * (EPS / U)
            ad = ds.abs() + noise
            dq[s, h], mq[s, h] = scale * (ds @ kk), scale * (ad @ kk.abs())
            dk[s, g] += scale * (ds.T @ qq)
            mk[s, g] += scale * (ad.T @ qq.abs())
            dv[s, g] += p.T @ gg
            mv[s, g] += p.T @ gg.abs()
        at += n
    return (dq, dk, dv), (mq, mk, mv)


def decode(q, k_pages, v_pages, table, lengths, scale):
    """O, LSE and magnitudes; tokens on pages outside the cache do not count."""
    n_pages, page, hkv, D = k_pages.shape
    gr = q.shape[1] // hkv
    o, mag = torch.zeros_like(q, dtype=F64), torch.zeros_like(q, dtype=F64)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=F64, device=q.device)
    for b in range(q.shape[0]):
        n = max(0, min(int(lengths[b]), table.shape[1] * page))
        t = torch.arange(n, device=q.device)
        pg = table[b].long()[t // page] if n else t
        t = t[(pg >= 0) & (pg < n_pages)]
        if not len(t):
            continue
        pg = table[b].long()[t // page]
        for h in range(q.shape[1]):
            kk, vv = k_pages[pg, t % page, h // gr].to(F64), v_pages[pg, t % page, h // gr].to(F64)
            x = kk @ q[b, h].to(F64) * scale
            lse[b, h] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[b, h])
            o[b, h], mag[b, h] = p @ vv, p @ vv.abs()
    return o, lse, mag


def normal(seed, *shape, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=device).to(torch.bfloat16)
