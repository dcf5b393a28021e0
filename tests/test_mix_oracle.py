"""The 64-bit oracle of the channel-mixing operators, pinned on the CPU: its
gradients against central differences, Philox against the published known
answers, and planted mistakes that the pins must catch."""
import numpy as np
import pytest
import torch

import mix_oracle as mo


def rnd(seed, *shape):
    return torch.from_numpy(np.random.Generator(np.random.PCG64(seed)).standard_normal(shape))


def differences(f, x, h=1e-5):
    """Gradient of the scalar f at x by central differences."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).reshape(-1)
        e[i] = h
        e = e.reshape(x.shape)
        g.reshape(-1)[i] = (f(x + e) - f(x - e)) / (2 * h)
    return g


@pytest.mark.parametrize("affine", [True, False])
def test_layernorm_gradient_against_differences(affine):
    x, dy = rnd(1, 3, 7), rnd(2, 3, 7)
    gamma, beta = (rnd(3, 7), rnd(4, 7)) if affine else (None, None)
    eps = 0.1
    _, mean, rstd = mo.layernorm(x, gamma, beta, eps)
    dx, dgamma, dbeta = mo.layernorm_bwd(dy, x, mean, rstd, gamma)
    loss = lambda a, b, c: float((mo.layernorm(a, b, c, eps)[0] * dy).sum())   # noqa: E731
    torch.testing.assert_close(dx, differences(lambda v: loss(v, gamma, beta), x), rtol=1e-7, atol=1e-8)
    if affine:
        torch.testing.assert_close(dgamma, differences(lambda v: loss(x, v, beta), gamma), rtol=1e-7, atol=1e-8)
        torch.testing.assert_close(dbeta, differences(lambda v: loss(x, gamma, v), beta), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("name", ["silu", "gelu", "relu", "sigmoid"])
def test_gated_gradient_against_differences(name):
    x, wg, wu, dy = rnd(5, 3, 4), rnd(6, 5, 4), rnd(7, 5, 4), rnd(8, 3, 5)
    dx, dwg, dwu = mo.gated_bwd(dy, x, wg, wu, name)
    loss = lambda a, b, c: float((mo.gated(a, b, c, name) * dy).sum())   # noqa: E731
    for got, ref in ((dx, differences(lambda v: loss(v, wg, wu), x)), (dwg, differences(lambda v: loss(x, v, wu), wg)),
                     (dwu, differences(lambda v: loss(x, wg, v), wu))):
        torch.testing.assert_close(got, ref, rtol=1e-6, atol=1e-7)


def test_a_wrong_gradient_is_caught():
    x, dy = rnd(1, 3, 7), rnd(2, 3, 7)
    _, mean, rstd = mo.layernorm(x, None, None, 0.1)
    xhat = (x - mean[:, None]) * rstd[:, None]
    wrong = rstd[:, None] * (dy - dy.mean(1)[:, None])       # the projection on xhat left out
    ref = differences(lambda v: float((mo.layernorm(v, None, None, 0.1)[0] * dy).sum()), x)
    assert (wrong - ref).abs().max() > 1e-2
    assert (wrong - rstd[:, None] * xhat * (dy * xhat).mean(1)[:, None] - ref).abs().max() < 1e-7


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, words):
    """The published test vectors of Philox4x32 with ten rounds."""
    assert tuple(int(w) for w in mo.philox4x32(counter, key)) == words


def test_keep_rate_and_independence():
    a = mo.keep(0, 1 << 20, 0.1, 7, 0).double()
    b = mo.keep(0, 1 << 20, 0.1, 7, 1).double()
    assert abs(float(a.mean()) - 0.9) < 5 * (0.09 / (1 << 20)) ** 0.5
    assert abs(float((a * b).mean()) - 0.81) < 5 * (0.1539 / (1 << 20)) ** 0.5
    assert bool(mo.keep(0, 64, 0.0, 7, 0).all()) and not bool(mo.keep(0, 64, 1.0, 7, 0).any())
    # a slice of the mask is the mask of the slice
    assert torch.equal(mo.keep(0, 100, 0.5, 9, 3)[37:80], mo.keep(37, 43, 0.5, 9, 3))
