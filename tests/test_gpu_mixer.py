"""The residual block that runs the channel-mixing operators with the
convolutions: its gradients against differences of its 64-bit definition, and a
short training run."""
import math

import pytest
import torch

import mix_oracle as mo
from convolution_nhwc_amd import mixer

pytestmark = pytest.mark.gpu

N, H, W, C, F = 2, 9, 8, 32, 72


def definition(x, w, p, seed, step, act):
    """The block in 64 bits on the host."""
    t = torch.nn.functional
    a = t.conv2d(x.permute(0, 3, 1, 2), w["dw"].permute(0, 3, 1, 2), padding=3, groups=C).permute(0, 2, 3, 1)
    n = mo.layernorm(a.reshape(-1, C), w["gamma"], w["beta"], 1e-5)[0]
    h = mo.gated(n, w["wg"], w["wu"], act)
    o = h @ w["down"].reshape(C, F).t()
    return mo.dropout(o, p, seed, step, x.reshape(-1, C)).reshape(x.shape)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_block_gradients(act):
    torch.manual_seed(0)
    block = mixer.ChannelMixer(N, H, W, C, F, dtype="f16", act=act, p=0.2, seed=3)
    x = torch.randn(N, H, W, C).half()
    dy = torch.randn(N, H, W, C).half()
    y = block.forward(x.cuda(), step=5)
    dx = block.backward(dy.cuda())
    w = {k: v.double().cpu() for k, v in block.weights.items()}
    x64 = x.double().requires_grad_()
    for v in w.values():
        v.requires_grad_()
    ref = definition(x64, w, 0.2, 3, 5, act)
    ref.backward(dy.double())
    # fp16 rounds each of the block's five stages by half a step (2^-11); the
    # sums of many rounded terms average that down, maxima stay within a few
    tol = 8 * 2.0 ** -11

    def close(got, want, what):
        err = (got.double().cpu() - want).abs().max() / want.abs().max()
        assert float(err) < tol, (what, float(err))
    close(y, ref.detach(), "y")
    close(dx, x64.grad, "dx")
    for k in mixer.ChannelMixer.NAMES:
        close(block.grads[k], w[k].grad, k)
    # the definition's own gradient against a difference along a random direction
    d = {k: torch.randn_like(v) for k, v in w.items()}
    e = 1e-5
    up = definition(x.double(), {k: v.detach() + e * d[k] for k, v in w.items()}, 0.2, 3, 5, act)
    down = definition(x.double(), {k: v.detach() - e * d[k] for k, v in w.items()}, 0.2, 3, 5, act)
    along = float(((up - down) * dy.double()).sum()) / (2 * e)
    want = sum(float((w[k].grad * d[k]).sum()) for k in w)
    assert math.isclose(along, want, rel_tol=1e-5, abs_tol=1e-4 * abs(want) + 1e-3)


def test_training_lowers_the_loss():
    losses = mixer.train(steps=20)
    assert all(math.isfinite(v) for v in losses)
    assert sum(losses[-3:]) < 0.7 * sum(losses[:3]), losses
