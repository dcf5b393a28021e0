"""The channel-mixing operators in 64 bits on the host, and the error bounds
their tests use.

Bounds count roundings.  A result rounded to type t is off by half a step,
eps(t)/2 relative (and half the smallest subnormal, for fp16); fp32 sums of n
terms are off by at most n * 2^-24 of the sum of absolute values, of which a
tree or a blocked sum of random terms realises a small multiple of sqrt(n).
"""
import math

import numpy as np
import torch

U32 = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SUBNORMAL = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def half_step(t, v):
    return torch.finfo(t).eps / 2 * v.abs() + SUBNORMAL[t]


def chain(n):
    """fp32 roundings that a sum of n terms can show."""
    return (8 * math.sqrt(n) + 64) * U32


# ---- layer norm -----------------------------------------------------------------

def layernorm(x, gamma, beta, eps):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layernorm_bound(x, gamma, beta, eps, t):
    y, mean, rstd = layernorm(x, gamma, beta, eps)
    g = torch.ones(x.shape[1], dtype=torch.float64) if gamma is None else gamma.abs()
    b = 0.0 if beta is None else beta.abs()
    k = chain(x.shape[1])
    mean_err = k * x.abs().mean(1) + U32 * mean.abs()
    # the deviations carry the mean's error: relative error of rstd
    spread = torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    # squared deviations err by 2 |d| e; their mean over spread^2 is at most 2 e / spread
    rstd_rel = k + mean_err / spread
    xhat = ((x - mean[:, None]) * rstd[:, None]).abs()
    y_err = (xhat * (rstd_rel[:, None] + 8 * U32) + (mean_err * rstd)[:, None] + U32) * g + 4 * U32 * (xhat * g + b)
    return half_step(t, y) + y_err, mean_err + U32 * mean.abs(), rstd * rstd_rel + U32 * rstd


def layernorm_bwd(dy, x, mean, rstd, gamma):
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    m1, m2 = g.mean(1), (g * xhat).mean(1)
    dx = rstd[:, None] * (g - m1[:, None] - xhat * m2[:, None])
    return dx, (dy * xhat).sum(0), dy.sum(0)


def layernorm_bwd_bound(dy, x, mean, rstd, gamma, t, pt):
    xhat = ((x - mean[:, None]) * rstd[:, None]).abs()
    # x - mean rounds once more when x and mean are far from their difference
    xhat_err = 4 * U32 * (xhat + (x.abs() + mean.abs()[:, None]) * rstd[:, None])
    g = (dy if gamma is None else dy * gamma).abs()
    k = chain(x.shape[1])
    m1, m2 = g.mean(1)[:, None], (g * xhat).mean(1)[:, None]
    m2_err = k * m2 + (g * xhat_err).mean(1)[:, None]
    dx, dgamma, dbeta = layernorm_bwd(dy, x, mean, rstd, gamma)
    dx_err = rstd[:, None] * (8 * U32 * (g + m1 + xhat * m2) + k * m1 + xhat * m2_err + xhat_err * m2)
    kr = chain(x.shape[0])
    return (half_step(t, dx) + dx_err,
            half_step(pt, dgamma) + kr * (dy.abs() * xhat).sum(0) + (dy.abs() * xhat_err).sum(0),
            half_step(pt, dbeta) + kr * dy.abs().sum(0))


# ---- gated feed-forward ---------------------------------------------------------

def act(name, g):
    if name == "relu":
        on = (g > 0).double()
        return torch.where(g > 0, g, torch.zeros_like(g)), on
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(g)
    if name == "sigmoid":
        return s, s * (1 - s)
    return g * s, s * (1 + g * (1 - s))


def gated(x, wg, wu, name):
    a, _ = act(name, x @ wg.t())
    return a * (x @ wu.t())


def gated_bwd(dy, x, wg, wu, name):
    u = x @ wu.t()
    a, da = act(name, x @ wg.t())
    dg, du = dy * u * da, dy * a
    return dg @ wg + du @ wu, dg.t() @ x, du.t() @ x


# |act'| <= 1.13 for gelu, 1.1 for silu; |act''| <= 0.8 (gelu: 2 phi(0))
LIP1, LIP2 = 1.13, 0.8


def _projections(x, wg, wu, name):
    g, u = x @ wg.t(), x @ wu.t()
    k = chain(x.shape[1])
    ge, ue = k * (x.abs() @ wg.abs().t()), k * (x.abs() @ wu.abs().t())
    a, da = act(name, g)
    # the fp32 activation: exp and erf to a few ulp of 1 (their argument's
    # rounding grows with |g|), scaled by g
    fe = 16 * U32 * (1 + g.abs()) ** 2
    ae = LIP1 * ge + fe + 4 * U32 * a.abs()
    de = LIP2 * ge + fe
    if name == "relu":
        de = (g.abs() <= ge).double()     # the slope jumps at 0
    return g, u, a, da, ge, ue, ae, de


def gated_bound(x, wg, wu, name, t):
    g, u, a, da, ge, ue, ae, de = _projections(x, wg, wu, name)
    y = a * u
    return half_step(t, y) + ae * u.abs() + a.abs() * ue + ae * ue + 4 * U32 * y.abs()


def gated_bwd_bound(dy, x, wg, wu, name, t):
    g, u, a, da, ge, ue, ae, de = _projections(x, wg, wu, name)
    dg, du = dy * u * da, dy * a
    # dg and du are rounded to t before the products
    dge = dy.abs() * (da.abs() * ue + de * (u.abs() + ue)) + 8 * U32 * dg.abs()
    dge = dge + half_step(t, dg.abs() + dge)
    due = dy.abs() * ae + 8 * U32 * du.abs()
    due = due + half_step(t, du.abs() + due)
    kf, kr = chain(2 * wg.shape[0]), chain(x.shape[0])
    dx, dwg, dwu = gated_bwd(dy, x, wg, wu, name)
    return (half_step(t, dx) + dge @ wg.abs() + due @ wu.abs() + kf * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()),
            half_step(t, dwg) + dge.t() @ x.abs() + kr * (dg.abs().t() @ x.abs()),
            half_step(t, dwu) + due.t() @ x.abs() + kr * (du.abs().t() @ x.abs()))


# ---- dropout ---------------------------------------------------------------------

def philox4x32(counter, key, rounds=10):
    """Philox4x32 on arrays of 32-bit words (Salmon, Moraes, Dror, Shaw 2011)."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    m = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & m,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep(first, n, p, seed, offset):
    """Mask of elements first..first+n-1."""
    b0, b1 = first // 4, (first + n + 3) // 4
    blocks = np.arange(b0, b1, dtype=np.uint64)
    m = np.uint64(0xFFFFFFFF)
    offset &= (1 << 64) - 1
    w = philox4x32([blocks & m, blocks >> np.uint64(32), np.full_like(blocks, offset & 0xFFFFFFFF),
                    np.full_like(blocks, offset >> 32)], (seed & 0xFFFFFFFF, seed >> 32))
    w = np.stack(w, 1).reshape(-1)[first - 4 * b0:][:n]
    return torch.from_numpy(w >= np.uint64(round(p * 2 ** 32)))


def dropout(x, p, seed, offset, residual=None, first=0):
    k = keep(first, x.numel(), p, seed, offset).reshape(x.shape)
    y = torch.where(k, x / (1 - p) if p < 1 else x, torch.zeros_like(x))
    return y if residual is None else y + residual
