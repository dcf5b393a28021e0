"""A channels-last residual block on the library's own operators, forward,
backward and training step:

    a = depthwise 7x7 convolution of x
    n = layer norm of a over the channels
    h = gated feed-forward, act(n wg^T) * (n wu^T)
    o = pointwise convolution of h back to the block's width
    y = x + dropout(o)

``python -m convolution_nhwc_amd.mixer`` trains one block for a few steps on
synthetic data and prints the loss.  Tensors are fp16 or bf16 on the GPU;
PyTorch holds them, adds the two branches of dx and updates the fp32 master
weights.
"""
import math

from . import api


class ChannelMixer:
    """One block.  ``forward(x, step)`` keeps what ``backward(dy)`` needs;
    ``backward`` returns dx and leaves the weights' gradients in ``grads``.
    The dropout mask of a step is drawn from (seed, step)."""

    NAMES = ("dw", "gamma", "beta", "wg", "wu", "down")

    def __init__(self, n, h, w, c, f, dtype="bf16", act="silu", p=0.1, seed=0, device="cuda"):
        import torch
        self.act, self.p, self.seed = act, p, seed
        self.spatial = dict(n=n, h=h, w=w, c=c, k=c, r=7, s=7, stride=1, pad_h=3, pad_w=3, groups=c, dtype=dtype)
        self.narrow = dict(n=n, h=h, w=w, c=f, k=c, r=1, s=1, stride=1, pad_h=0, pad_w=0, groups=1, dtype=dtype)
        t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        g = torch.Generator(device="cpu").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(device)
        self.master = {"dw": normal(c, 7, 7, 1, std=1 / 7.0), "gamma": torch.ones(c, device=device),
                       "beta": torch.zeros(c, device=device), "wg": normal(f, c, std=1 / math.sqrt(c)),
                       "wu": normal(f, c, std=1 / math.sqrt(c)), "down": normal(c, 1, 1, f, std=1 / math.sqrt(f))}
        self.dtype = t
        self.weights, self.grads, self.kept, self.ws = {}, {}, None, None
        self._round()

    def _round(self):
        # the norm's weights stay in fp32, the others are the products' operands
        self.weights = {k: v if k in ("gamma", "beta") else v.to(self.dtype) for k, v in self.master.items()}

    def forward(self, x, step=0):
        w = self.weights
        a = api.fwd(x, w["dw"], self.spatial)
        n, mean, rstd = api.layernorm(a, w["gamma"], w["beta"])
        h = api.gated(n, w["wg"], w["wu"], act=self.act)
        o = api.fwd(h, w["down"], self.narrow)
        self.kept = (x, a, mean, rstd, n, h, step)
        return api.dropout(o, self.p, self.seed, step, residual=x)

    def backward(self, dy):
        import torch
        w = self.weights
        x, a, mean, rstd, n, h, step = self.kept
        do = api.dropout_bwd(dy, self.p, self.seed, step)
        dh = api.dgrad(do, w["down"], self.narrow)
        down = api.wgrad(h, do, self.narrow)
        if self.ws is None:
            self.ws = torch.empty(api.gated_workspace(n, w["wg"], "bwd"), dtype=torch.uint8, device=x.device)
        dn, wg, wu = api.gated_bwd(dh, n, w["wg"], w["wu"], act=self.act, ws=self.ws)
        da, gamma, beta = api.layernorm_bwd(dn, a, mean, rstd, w["gamma"])
        dw = api.wgrad(x, da, self.spatial)
        self.grads = {"dw": dw, "gamma": gamma, "beta": beta, "wg": wg, "wu": wu, "down": down}
        return api.dgrad(da, w["dw"], self.spatial) + dy

    def update(self, rate):
        for k, g in self.grads.items():
            self.master[k] -= rate * g.float()
        self._round()


def train(steps=20, n=4, h=14, w=14, c=64, f=176, dtype="bf16", rate=1.0, seed=0):
    """Fits a block to another one's outputs; returns the mean squared error of
    each step."""
    import torch
    teacher = ChannelMixer(n, h, w, c, f, dtype=dtype, p=0.0, seed=seed + 1)
    block = ChannelMixer(n, h, w, c, f, dtype=dtype, p=0.05, seed=seed)
    g = torch.Generator(device="cpu").manual_seed(seed + 2)
    losses = []
    for step in range(steps):
        x = torch.randn((n, h, w, c), generator=g).to("cuda", block.dtype)
        diff = block.forward(x, step).float() - teacher.forward(x).float()
        losses.append(float((diff * diff).mean()))
        # the gradient of the sum over channels, averaged over pixels
        block.backward((diff * (2.0 / (n * h * w))).to(block.dtype))
        block.update(rate / c)
    return losses


if __name__ == "__main__":
    for i, v in enumerate(train()):
        print("step %2d  loss %.4f" % (i, v))
