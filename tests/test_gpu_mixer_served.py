"""The served block's weights are the fp32 masters', rounded once."""
import pytest
import torch

from convolution_nhwc_amd import mixer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("adamw", [None, 32, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_products_are_of_the_masters(dtype, adamw):
    block = mixer.ChannelMixer(2, 5, 6, 32, 72, dtype=dtype, p=0.0, seed=1)
    if adamw:
        block.adamw(adamw)
    x = torch.randn(2, 5, 6, 32, device="cuda").to(block.dtype)
    for step in range(2):
        y = block.forward(x, step)
        block.backward(y)
        block.update(1e-3)
    served = block.serve()
    for k in ("wg", "wu", "down"):
        q, scale = served.products[k]
        w = block.master[k].double().reshape(block.master[k].shape[0], -1)
        # half a step of the code, and the scale's own rounding over 127 steps
        worst = (q.double() * scale.double()[:, None] - w).abs() / scale.double()[:, None]
        assert float(worst.max()) <= 0.5 + 127 * 2.0 ** -24, (k, float(worst.max()))
        # (the quotient in 64 bits, which rounds to fp32 as the exact one does)
        assert torch.equal(scale, (w.abs().amax(1) / 127).float())
    assert bool(torch.isfinite(served.forward(x)).all())
