"""The activations of the gated feed-forward block in 64 bits, each with the
error that its evaluation in fp32 can show, and operands that carry one
pre-activation value an output column.

The errors are those of each function's own evaluation, relative to the value
where the function is small: a tail of 0, or one of the wrong sign, is outside.
"""
import math

import torch

from mix_oracle import U32, chain, half_step

TINY = 2.0 ** -126        # fp32 results below this may be flushed


def exp_error(a):
    """Relative error of exp(a) in fp32 as exp2(a log2 e): the constant and the
    product round, the exponent's error is relative in the result; an ulp more
    for the function."""
    return (2 * a.abs() + 4) * U32


def act(name, g):
    """(act(g), act'(g), error of each) for exact g (64 bits)."""
    a = g.abs()
    if name == "relu":
        return g.clamp_min(0), (g > 0).double(), torch.zeros_like(g), torch.zeros_like(g)
    if name == "gelu":
        q = 0.5 * torch.special.erfc(a / math.sqrt(2))          # Phi(-|g|)
        phi = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        # its form is good to 1.1e-5 of the value and 3.2e-7; the exponent g^2/2
        # rounds three times, the reciprocal and the polynomial's terms each once
        # more
        qe = torch.minimum(1.1e-5 * q, torch.full_like(q, 3.2e-7)) + q * (1.5 * a * a + 24) * U32 + TINY
        c = torch.where(g < 0, q, 1 - q)
        v, d = g * c, c + g * phi
        return v, d, a * qe + 4 * U32 * v.abs(), qe + a * phi * (1.5 * a * a + 8) * U32 + 2 * U32 * (c + a * phi)
    e = exp_error(g)
    s, t = torch.sigmoid(g), torch.sigmoid(-g)                  # s + t = 1
    r = t * e + 4 * U32                                         # relative error of s
    if name == "sigmoid":
        return s, s * t, s * (e + 4 * U32) + TINY, s * t * (2 * e + 10 * U32) + TINY
    v, d = g * s, s * (1 + g * t)
    # 1 - s rounds at the size of s
    return (v, d, v.abs() * (r + 2 * U32) + TINY,
            s * a * (s * r + U32) + (r + 4 * U32) * s * (1 + a * t) + TINY)


def rounded(t, v, e):
    """Largest distance from v of a value within e of it, rounded to t."""
    return e + half_step(t, v.abs() + e)


def values(n, t, top=12.0):
    """n pre-activations of type t in -top..top, half of them evenly spaced and
    half over the logarithm of their size."""
    m = n // 4
    log = torch.logspace(-6, math.log10(top), m, dtype=torch.float64)
    g = torch.cat([torch.linspace(-top, top, n - 2 * m, dtype=torch.float64), log, -log])
    return g.to(t)


# where g and u come from in a row of c channels: with c > 128 each from another
# 64-deep step of the reduction
def columns(c):
    return (c - 1, min(70, c - 2))


def operands(g, rows, c, t):
    """(x, wg, wu, dy) on the host: every row of x gives pre-activation g[j] and
    u = 1 in column j, exactly; dy is 1 in one row of each column."""
    f = len(g)
    kg, ku = columns(c)
    gen = torch.Generator().manual_seed(f + rows + c)
    row = torch.randint(-1, 2, (c,), generator=gen).to(t)       # met by zeros in both weights
    row[kg] = row[ku] = 1
    wg, wu = torch.zeros(f, c, dtype=t), torch.zeros(f, c, dtype=t)
    wg[:, kg] = g
    wu[:, ku] = 1
    dy = torch.zeros(rows, f, dtype=t)
    at = torch.arange(f)
    dy[at % rows, at] = 1
    return row.repeat(rows, 1), wg, wu, dy


def forward(name, g, t):
    """(y of any row, its bound)"""
    v, _, e, _ = act(name, g.double())
    return v, rounded(t, v, e)


def backward(name, g, x, rows, t):
    """((dx, dwg, dwu), their bounds): dg and du are act' and act, rounded to t,
    and every other term of their sums is 0."""
    g = g.double()
    f, c = len(g), x.shape[1]
    kg, ku = columns(c)
    v, d, ve, de = act(name, g)
    ve, de = rounded(t, v, ve), rounded(t, d, de)
    row = x[0].double()
    dwg, dwu = d[:, None] * row, v[:, None] * row
    at = torch.arange(f) % rows
    dx, bx, size = (torch.zeros(rows, c, dtype=torch.float64) for _ in range(3))
    for col, val, err in ((kg, d * g, de * g.abs()), (ku, v, ve)):
        dx[:, col].index_add_(0, at, val)
        bx[:, col].index_add_(0, at, err)
        size[:, col].index_add_(0, at, val.abs())
    bx = bx + chain(2 * f) * size
    return (dx, dwg, dwu), (bx + half_step(t, dx.abs() + bx), de[:, None] * row.abs(), ve[:, None] * row.abs())
