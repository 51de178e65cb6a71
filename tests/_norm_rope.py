"""Plain 64-bit form of the norms of queries and keys with their rotation, its
backward, and bounds on the kernels' errors.

A result is rounded to bf16 once (off by at most U = 2^-8 of the value).  What the
32-bit arithmetic adds is counted against the sums of magnitudes that a value is
made of: a sum of D <= 128 squares or products is eight additions in a lane and
four across lanes with a rounding each and one per product, rsqrt two steps, and
eight more products and sums stand on any path: at most 32 roundings of 2^-24 on
each term, so EPS = 2^-19 of the magnitudes.  (r comes from a sum of squares,
whose terms have one sign: its relative error is within the same count.)
"""
import torch

U = 2.0 ** -8
EPS = 2.0 ** -19
F64 = torch.float64


def table(positions, rot, base=10000.0, device="cpu"):
    i = torch.arange(rot // 2, dtype=F64, device=device)
    angle = torch.arange(positions, dtype=F64, device=device)[:, None] * base ** (-2.0 * i / rot)
    return torch.cat([angle.cos(), angle.sin()], 1)


def turn(y, rope, positions, pairs, sign):
    """y [rows, heads, D] turned, and the magnitudes of the terms of each value."""
    rot = rope.shape[1]
    c, s = rope.to(F64)[positions.long()][:, None].split(rot // 2, 2)
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if pairs else (y[..., :rot // 2], y[..., rot // 2:rot])
    out, mag = y.clone(), y.abs()
    for t, lo, hi in ((out, a * c - sign * b * s, b * c + sign * a * s),
                      (mag, (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs())):
        if pairs:
            t[..., 0:rot:2], t[..., 1:rot:2] = lo, hi
        else:
            t[..., :rot // 2], t[..., rot // 2:rot] = lo, hi
    return out, mag


def forward(x, w, rope, positions, eps, pairs):
    x, w = x.to(F64), w.to(F64)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return turn(w * (x * r), rope, positions, pairs, 1.0)


def backward(x, dz, w, rope, positions, eps, pairs):
    """(dx, dw) and the magnitudes of their terms."""
    x, dz, w = x.to(F64), dz.to(F64), w.to(F64)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    g, G = turn(dz, rope, positions, pairs, -1.0)
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    mag = r * (G * w.abs() + n.abs() * (G * w.abs() * n.abs()).mean(-1, keepdim=True))
    return (dx, (g * n).sum((0, 1))), (mag, (G * n.abs()).sum((0, 1)))


def within(name, x, ref, mag, rounding=U, eps=EPS):
    err = (x.to(F64) - ref).abs()
    bad = ~(err <= rounding * ref.abs() + (1 + rounding) * eps * mag + 1e-37)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside their bound, worst {err[bad].max()}"
