"""Group norm's activations over the whole range of z, in both directions: tails that
have fallen to 0, and pixels far outside of their map."""
import pytest
import torch

import groupnorm_oracle as go
from convolution_nhwc_amd import api
from mix_oracle import TYPES

pytestmark = pytest.mark.gpu

ACTS = ["none", "silu", "gelu", "relu", "sigmoid"]


def within(got, ref, bound, what):
    err = (got.double().cpu().reshape(ref.shape) - ref).abs()
    bad = ~(err <= bound)     # (a NaN is not within)
    assert not bad.any(), "%s: %d of %d, %d of them not finite" % (what, int(bad.sum()), bad.numel(), int((~got.isfinite()).sum()))


def check(x, dy, groups, gamma, beta, dtype, act, tune):
    """y within its bound, and z of both directions' results."""
    n, c, t = x.shape[0], x.shape[-1], TYPES[dtype]
    x, dy, gamma, beta = x.to(t), dy.to(t), gamma.float(), beta.float()
    xd, dyd = (v.double().reshape(n, -1, c) for v in (x, dy))
    xg, gg, bg = x.cuda(), gamma.cuda(), beta.cuda()
    with api.override(tune=tune):
        y, mu, r = api.group_norm(xg, groups, gg, bg, act=act)
        grads = api.group_norm_bwd(dy.cuda(), xg, mu, r, groups, gg, bg, act=act)
    ref = go.forward(xd, groups, gamma, beta, 1e-5, act)
    for got, want, bound, what in zip((y, mu, r), ref, go.forward_bound(xd, groups, gamma, beta, 1e-5, act, t), ("y", "mean", "rstd")):
        within(got, want, bound, what)
    args = (dyd, xd, mu.double().cpu(), r.double().cpu(), groups, gamma, beta, act)
    for got, want, bound, what in zip(grads, go.backward(*args), go.backward_bound(*args, t, torch.float32), ("dx", "dgamma", "dbeta")):
        within(got, want, bound, what)
    return y, go.forward(xd, groups, gamma, beta, 1e-5, "none")[0]


@pytest.mark.parametrize("tune", [0, 1])
@pytest.mark.parametrize("each", [3, 8])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_every_z(dtype, act, each, tune):
    """beta takes z from -10000 to 10000, closely from 85 to 200 on both sides, where exponentials leave fp32."""
    g = torch.Generator().manual_seed(1)
    near = torch.linspace(85, 200, 300, dtype=torch.float64)
    beta = torch.cat([torch.linspace(-1e4, 1e4, 408, dtype=torch.float64), near, -near])
    c = beta.numel()
    beta = beta[torch.randperm(c, generator=g)]
    x, dy = (torch.randn(2, 5, 3, c, generator=g, dtype=torch.float64) for _ in range(2))
    y, z = check(x, dy, c // each, torch.full((c,), 0.01), beta, dtype, act, tune)
    low = z.reshape(y.shape) < -88
    if act in ("silu", "gelu", "sigmoid"):
        # the largest of them is silu's 88 exp(-88) = 5.4e-37
        assert int(low.sum()) > 1000 and float(y.cpu()[low].double().abs().max()) < 1e-36


@pytest.mark.parametrize("tune", [0, 1])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_one_pixel_far_out(dtype, act, tune):
    """A pixel of a 56 x 56 map that alone makes the group's spread: |xhat| nears the root of its elements."""
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(2, 56, 56, 8, generator=g, dtype=torch.float64) for _ in range(2))
    x[0, 20, 30, 3], x[1, 55, 55, 7] = 30000.0, -30000.0
    z = check(x, dy, 1, torch.ones(8), torch.zeros(8), dtype, act, tune)[1]
    assert float(z.max()) > 150 and float(z.min()) < -150
