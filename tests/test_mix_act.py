"""The activation oracle on the CPU: its slopes against differences, forms that
its bounds have to accept, and wrong values that they have to refuse."""
import math

import pytest
import torch

import mix_act as ma
from mix_oracle import TYPES, act as plain_act, half_step

NAMES = ["silu", "gelu", "relu", "sigmoid"]


@pytest.mark.parametrize("name", NAMES)
def test_values_and_slopes(name):
    g = torch.linspace(-11.9, 12.1, 997, dtype=torch.float64)
    v, d, ve, de = ma.act(name, g)
    pv, pd = plain_act(name, g)
    torch.testing.assert_close(v, pv, rtol=1e-9, atol=0)
    torch.testing.assert_close(d, pd, rtol=1e-9, atol=1e-13)
    h = 1e-6
    torch.testing.assert_close(d, (ma.act(name, g + h)[0] - ma.act(name, g - h)[0]) / (2 * h), rtol=1e-6, atol=1e-9)
    assert bool((ve <= 1e-4 * v.abs() + 1e-30).all())            # relative, in the tails too
    if name != "relu":
        assert bool((ve > 0).all()) and bool((de > 0).all())


def refused(name, t, got_v, got_d):
    """(value refused, slope refused) where fp32 results are rounded to t."""
    t = TYPES[t]
    g = ma.values(4096, t).double()
    v, d, ve, de = ma.act(name, g)
    out = []
    for got, ref, err in ((got_v, v, ve), (got_d, d, de)):
        if got is None:
            out.append(None)
            continue
        off = (got(g).to(t).double() - ref).abs()
        out.append(not bool((off <= ma.rounded(t, ref, err)).all()))
    return tuple(out)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_the_definition_in_64_bits_is_accepted(name, t):
    assert refused(name, t, lambda g: plain_act(name, g)[0], lambda g: plain_act(name, g)[1]) == (False, False)


@pytest.mark.parametrize("name", ["silu", "gelu", "sigmoid"])
def test_a_tail_of_zero_or_of_the_wrong_sign_is_refused(name):
    for wrong in (0.0, -1.0):
        def tail(g):
            v = plain_act(name, g)[0]
            return torch.where(g < -5, wrong * v, v)
        assert refused(name, "bf16", tail, None)[0]


def test_gelu_with_an_absolute_error_in_its_tail_is_refused():
    """Abramowitz and Stegun 7.1.26 in 64 bits: 7.5e-8 of 1, 4.7e-4 of the value at -4."""
    def tail(g):
        z = g.abs() / math.sqrt(2)
        k = 1 / (1 + 0.3275911 * z)
        p = ((((1.061405429 * k - 1.453152027) * k + 1.421413741) * k - 0.284496736) * k + 0.254829592) * k
        return 0.5 * p * torch.exp(-z * z)

    def value(g):
        return torch.where(g < 0, g * tail(g), g * (1 - tail(g)))
    assert refused("gelu", "f16", value, None)[0] and refused("gelu", "bf16", value, None)[0]


def test_sigmoid_slope_of_a_rounded_difference_is_refused():
    def slope(g):
        s = torch.sigmoid(g).float()
        return s * (1 - s)
    assert refused("sigmoid", "bf16", None, slope)[1]

    def by_exp(g):
        e = torch.exp(-g.abs()).float()
        r = 1 / (1 + e)
        return e * r * r
    assert not refused("sigmoid", "bf16", None, by_exp)[1]


@pytest.mark.parametrize("c", [2, 8, 136])
def test_operands_carry_their_values(c):
    t = torch.bfloat16
    g = ma.values(257, t)
    x, wg, wu, dy = (v.double() for v in ma.operands(g, 5, c, t))
    assert torch.equal(x @ wg.t(), g.double().expand(5, -1)) and bool((x @ wu.t() == 1).all())
    assert bool((dy.sum(0) == 1).all())
    for name in NAMES:
        v, d = plain_act(name, g.double())
        dg, du = dy * d, dy * v
        for got, want in zip(ma.backward(name, g, x, 5, t)[0], (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x)):
            torch.testing.assert_close(got, want, rtol=1e-9, atol=1e-12)
    assert float(half_step(t, torch.ones(1, dtype=torch.float64))) >= 2.0 ** -8
