"""A channels-last residual block on the library's own operators, forward,
backward and training step:

    a = depthwise 7x7 convolution of x
    n = layer norm of a over the channels, or group norm over a sample's map
    h = gated feed-forward, act(n wg^T) * (n wu^T)
    o = pointwise convolution of h back to the block's width
    y = x + dropout(o)

``python -m convolution_nhwc_amd.mixer`` trains one block for a few steps on
synthetic data and prints the loss; ``--norm group`` and ``--adamw 8`` choose the
norm and the update, and ``--serve`` then answers with the products in 8-bit
integers.  Tensors are fp16 or bf16 on the GPU; PyTorch holds them and adds the
two branches of dx.  The fp32 master weights are updated by a plain gradient
step in PyTorch, or by AdamW (``ChannelMixer.adamw``) in one launch that writes
the 16-bit weights too.
"""
import argparse
import math

from . import api


class ChannelMixer:
    """One block.  ``forward(x, step)`` keeps what ``backward(dy)`` needs;
    ``backward`` returns dx and leaves the weights' gradients in ``grads``.
    The dropout mask of a step is drawn from (seed, step).  ``norm`` is "layer" or
    "group" (of ``groups`` groups of channels)."""

    NAMES = ("dw", "gamma", "beta", "wg", "wu", "down")

    def __init__(self, n, h, w, c, f, dtype="bf16", act="silu", p=0.1, seed=0, device="cuda", norm="layer", groups=8):
        import torch
        if norm not in ("layer", "group"):
            raise ValueError('norm must be "layer" or "group" (got %r)' % (norm,))
        self.act, self.p, self.seed = act, p, seed
        self.groups = groups if norm == "group" else None
        self.optimizer = None
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

    def _norm(self, a):
        gamma, beta = self.weights["gamma"], self.weights["beta"]
        if self.groups:
            return api.group_norm(a, self.groups, gamma, beta)
        return api.layernorm(a, gamma, beta)

    def forward(self, x, step=0):
        w = self.weights
        a = api.fwd(x, w["dw"], self.spatial)
        n, mean, rstd = self._norm(a)
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
        if self.groups:
            da, gamma, beta = api.group_norm_bwd(dn, a, mean, rstd, self.groups, w["gamma"], w["beta"])
        else:
            da, gamma, beta = api.layernorm_bwd(dn, a, mean, rstd, w["gamma"])
        dw = api.wgrad(x, da, self.spatial)
        self.grads = {"dw": dw, "gamma": gamma, "beta": beta, "wg": wg, "wu": wu, "down": down}
        return api.dgrad(da, w["dw"], self.spatial) + dy

    def adamw(self, bits=32, weight_decay=0.01, seed=None, **kw):
        """Updates by AdamW from here on, with fp32 or 8-bit moments; the norm's
        weights do not decay.  The draws that round 8-bit moments come from seed (the
        block's), by a key of their own.  More arguments go to api.AdamW."""
        fp32 = ("gamma", "beta")   # these weights are their masters
        # both draw at (element / 4, step): under one key the first tensor's moments would
        # be rounded by the words of the dropout's mask
        key = (self.seed if seed is None else seed) ^ 1 << 63
        self.optimizer = api.AdamW([self.master[k] for k in self.NAMES], bits=bits, seed=key,
                                   weight_decay=[0.0 if k in fp32 else weight_decay for k in self.NAMES],
                                   copies=[None if k in fp32 else self.weights[k] for k in self.NAMES], **kw)
        return self.optimizer

    def update(self, rate, **kw):
        """One step along ``grads``; more arguments go to AdamW's step."""
        if self.optimizer is not None:
            self.optimizer.step(rate, [self.grads[k] for k in self.NAMES], **kw)
            return
        if kw:
            raise ValueError("%s needs AdamW (adamw())" % ", ".join(kw))
        for k, g in self.grads.items():
            self.master[k] -= rate * g.float()
        self._round()

    def serve(self):
        """The block as it stands, without dropout, its three products in 8 bits."""
        return ServedMixer(self)


class ServedMixer:
    """A ChannelMixer's weights for answering: the products' rows in 8-bit
    integers with a scale each (half the bytes that the 16-bit ones take), made of
    the fp32 masters, which are rounded once so, and laid out once.  The normed rows are quantized once for both projections; the residual
    is added as the last product leaves."""

    def __init__(self, block):
        self.block = block
        self.dw, self.gamma, self.beta = (block.weights[k].clone() for k in ("dw", "gamma", "beta"))
        w = block.master
        self.products = {k: api.quantize_rows(w[k].reshape(w[k].shape[0], -1)) for k in ("wg", "wu", "down")}

    def forward(self, x):
        b = self.block
        p = dict(b.spatial, n=x.shape[0], h=x.shape[1], w=x.shape[2])
        a = api.fwd(x, self.dw, p)
        if b.groups:
            n = api.group_norm(a, b.groups, self.gamma, self.beta)[0]
        else:
            n = api.layernorm(a, self.gamma, self.beta)[0]
        q, scale = api.quantize_rows(n)
        h = api.linear_i8(q, *self.products["wg"], x_scale=scale, act=b.act, dtype=b.dtype)
        h *= api.linear_i8(q, *self.products["wu"], x_scale=scale, dtype=b.dtype)
        return api.linear_i8(h, *self.products["down"], residual=x)


def train(steps=20, n=4, h=14, w=14, c=64, f=176, dtype="bf16", rate=1.0, seed=0, norm="layer", adamw=None, serve=False):
    """Fits a block to another one's outputs; returns the mean squared error of
    each step.  adamw: 32 or 8, the bits of AdamW's moments (and its rate), or
    None for plain steps of rate / c.  With serve a last value is the error of
    the block's answers in 8 bits."""
    import torch
    teacher = ChannelMixer(n, h, w, c, f, dtype=dtype, p=0.0, seed=seed + 1, norm=norm)
    block = ChannelMixer(n, h, w, c, f, dtype=dtype, p=0.05, seed=seed, norm=norm)
    if adamw:
        block.adamw(adamw)
    g = torch.Generator(device="cpu").manual_seed(seed + 2)
    losses = []

    def batch():
        return torch.randn((n, h, w, c), generator=g).to("cuda", block.dtype)
    for step in range(steps):
        x = batch()
        diff = block.forward(x, step).float() - teacher.forward(x).float()
        losses.append(float((diff * diff).mean()))
        # the gradient of the sum over channels, averaged over pixels
        block.backward((diff * (2.0 / (n * h * w))).to(block.dtype))
        block.update(0.01 * rate if adamw else rate / c)
    if serve:
        x = batch()
        diff = block.serve().forward(x).float() - teacher.forward(x).float()
        losses.append(float((diff * diff).mean()))
    return losses


def main():
    ap = argparse.ArgumentParser(description="Train a residual block on synthetic data.")
    ap.add_argument("--norm", choices=("layer", "group"), default="layer")
    ap.add_argument("--adamw", type=int, choices=(32, 8), help="update by AdamW with moments of so many bits")
    ap.add_argument("--serve", action="store_true", help="answer in 8 bits at the end")
    args = ap.parse_args()
    losses = train(norm=args.norm, adamw=args.adamw, serve=args.serve)
    served = losses.pop() if args.serve else None
    for i, v in enumerate(losses):
        print("step %2d  loss %.4f" % (i, v))
    if args.serve:
        print("in 8 bits  %.4f" % served)


if __name__ == "__main__":
    main()
