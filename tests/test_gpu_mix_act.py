"""The gated feed-forward block's activations: pre-activations that overflow."""
import pytest
import torch

import mix_oracle as mo
from convolution_nhwc_amd import api

pytestmark = pytest.mark.gpu

NAMES = sorted(api.ACTS)

INF = float("inf")
# act(+inf); act(-inf) where the formula has a value there (silu and gelu: -inf * 0)
AT_INF = {"silu": (INF, None), "gelu": (INF, None), "relu": (INF, 0.0), "sigmoid": (1.0, 0.0)}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("rows,override", [
    (3, None), (40, None), (200, dict(tune=128, split_c=1)), (200, dict(tune=256, split_c=1)),
    (200, dict(tune=128, split_c=2)), (200, dict(tune=256, split_c=2))])
def test_overflowing_preactivations(rows, override, name):
    """Finite bf16 operands whose pre-activation is past fp32's largest value: every forward kernel gives
    the activation's value at infinity."""
    c, f = 128, 24
    x = torch.zeros(rows, c, dtype=torch.bfloat16)
    wg, wu = torch.zeros(f, c, dtype=torch.bfloat16), torch.zeros(f, c, dtype=torch.bfloat16)
    x[:, 5] = 2.0 ** 100
    x[:, 70] = 1.0
    wg[0::3, 5] = 2.0 ** 100          # g = +inf
    wg[1::3, 5] = -2.0 ** 100         # g = -inf
    wg[2::3, 70] = 1.0                # g = 1
    wu[:, 70] = 1.0                   # u = 1
    ops = x.cuda(), wg.cuda(), wu.cuda()
    if override is None:
        y = api.gated(*ops, act=name)
    else:
        with api.override(**override):
            y = api.gated(*ops, act=name)
    y = y.double().cpu()
    up, down = AT_INF[name]
    assert bool((y[:, 0::3] == up).all()), (name, y[0, 0])
    if down is not None:
        assert bool((y[:, 1::3] == down).all()), (name, y[0, 1])
    v = mo.act(name, torch.ones(1, dtype=torch.float64))[0]
    assert bool(((y[:, 2::3] - v).abs() <= 2 * mo.half_step(torch.bfloat16, v)).all())
