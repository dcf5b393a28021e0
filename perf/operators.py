"""The channel-mixing operators of a channels-last block, as measured workloads.

Next to its spatial convolutions a channels-last network normalises and mixes
the channels of every pixel (or token) by itself.  A tensor [N, H, W, C] is
then `rows` = N*H*W rows of `c` channels, and the operators are

  layernorm   y = (x - mean) * rstd * gamma + beta over a row's channels, the
              statistics kept for the backward pass; backward gives dx, dgamma
              and dbeta
  gated       y = act(x wg^T) * (x wu^T): the two widening projections of a
              gated feed-forward block, the activation and the product;
              backward gives dx, dwg and dwu
  dropout     y = residual + x * keep / (1 - p), keep drawn by a counter-based
              generator (Philox 4x32, 10 rounds) from (seed, offset, element
              index), so that the backward pass draws the same mask again

`run` computes them in plain torch operations (`own` false) or through
`convolution_nhwc_amd.api` (`own` true).
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}
_EPS = 1e-5
_MASK32 = 0xFFFFFFFF


# ---- cases -------------------------------------------------------------------

def _norm(op, rows, c, dtype, param, pad=0):
    return {"op": op, "rows": rows, "c": c, "dtype": dtype, "param": param, "pad": pad}


def _gated(op, rows, c, f, dtype, act):
    return {"op": op, "rows": rows, "c": c, "f": f, "dtype": dtype, "act": act}


def _drop(op, rows, c, dtype, p, residual, pad=0):
    return {"op": op, "rows": rows, "c": c, "dtype": dtype, "p": p, "residual": residual, "pad": pad}


def listed():
    cases = [
        # the deepest map of a batch of eight images (7 x 7 pixels, 2048 channels): a small call
        ("layernorm_fwd_map7", _norm("layernorm_fwd", 8 * 7 * 7, 2048, "bf16", "bf16")),
        # the norm after the depthwise 7x7 layer: 16 images of 56 x 56 pixels, 384 channels
        ("layernorm_fwd_map56", _norm("layernorm_fwd", 16 * 56 * 56, 384, "f16", "f16")),
        # its backward pass in training, weights and their gradients in fp32
        ("layernorm_bwd_map56", _norm("layernorm_bwd", 16 * 56 * 56, 384, "bf16", "f32")),
        # an odd width read out of a wider fp32 tensor
        ("layernorm_bwd_odd", _norm("layernorm_bwd", 4111, 1537, "f32", "f32", pad=11)),
        # one token, as in decoding: both weights are streamed once
        ("gated_fwd_token", _gated("gated_fwd", 1, 2048, 8192, "bf16", "silu")),
        # a serving batch of a few tokens, a hidden width that is no power of two
        ("gated_fwd_batch24", _gated("gated_fwd", 24, 2048, 5504, "f16", "silu")),
        # the block behind the depthwise 7x7 layer
        ("gated_fwd_map56", _gated("gated_fwd", 16 * 56 * 56, 384, 1024, "f16", "gelu")),
        # a long sequence through a wide block: the matrix cores' case
        ("gated_fwd_long", _gated("gated_fwd", 16384, 2048, 8192, "bf16", "silu")),
        # its training pass
        ("gated_bwd_long", _gated("gated_bwd", 8192, 2048, 8192, "bf16", "silu")),
        # a ragged training call: one more token than 56 x 56 pixels, odd channel counts
        ("gated_bwd_ragged", _gated("gated_bwd", 56 * 56 + 1, 385, 1027, "f16", "gelu")),
        # the residual join of the 56 x 56 block
        ("dropout_map56", _drop("dropout", 16 * 56 * 56, 384, "bf16", 0.1, True)),
        # the gradient of a small call's branch
        ("dropout_bwd_map7", _drop("dropout_bwd", 8 * 7 * 7, 2048, "f16", 0.25, False)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def _size(rng, lo, hi):
    """A size over the logarithm of its range: as it falls, or a multiple of 8 or of 64."""
    v = _log_int(rng, lo, hi)
    step = rng.choice((1, 1, 8, 8, 64))
    return min(max((v + step - 1) // step * step, lo), hi)


def draw(rng):
    op = rng.choice(("layernorm_fwd", "layernorm_bwd", "gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd",
                     "dropout", "dropout_bwd"))
    if op.startswith("gated"):
        limit = 16384 * 2048 * 8192 if op == "gated_fwd" else 8192 * 2048 * 8192
        c = _size(rng, 32, 4096)
        f = _size(rng, 32, 12288)
        rows = _size(rng, 1 if op == "gated_fwd" else 16, 65536)
        rows = max(1, min(rows, limit // (c * f)))
        return _gated(op, rows, c, f, rng.choice(("f16", "bf16")), rng.choice(("silu", "gelu", "relu", "sigmoid")))
    elems = 16 * 56 * 56 * 384
    c = _size(rng, 16, 8192)
    rows = max(1, min(_size(rng, 1, 262144), elems // c))
    dtype = rng.choice(("f16", "bf16", "bf16", "f32"))
    pad = rng.choice((0, 0, 0, 8, 5))
    if op.startswith("layernorm"):
        return _norm(op, rows, c, dtype, rng.choice((dtype, "f32")), pad)
    return _drop(op, rows, c, dtype, rng.choice((0.05, 0.1, 0.25, 0.5)), op == "dropout" and rng.random() < 0.7, pad)


def work(case):
    rows, c, b = case["rows"], case["c"], _BYTES[case["dtype"]]
    n = rows * c
    op = case["op"]
    if op == "layernorm_fwd":
        return {"bytes": 2 * n * b + 8 * rows + 2 * c * _BYTES[case["param"]], "flops": 8 * n}
    if op == "layernorm_bwd":
        return {"bytes": 3 * n * b + 8 * rows + 3 * c * _BYTES[case["param"]], "flops": 14 * n}
    if op == "gated_fwd":
        f = case["f"]
        return {"bytes": b * (n + 2 * f * c + rows * f), "flops": 4 * rows * f * c}
    if op == "gated_bwd":
        f = case["f"]
        # the projections again, the products with the weights and those with x
        return {"bytes": b * (2 * n + 4 * f * c + rows * f), "flops": 12 * rows * f * c}
    return {"bytes": n * b * (3 if case["residual"] else 2), "flops": (3 if case["residual"] else 2) * n}


# ---- inputs ------------------------------------------------------------------

def _inputs(case, seed):
    """The case's tensors on the GPU, from the seed alone (see prepare)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    rows, c = case["rows"], case["c"]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda") * std + mean

    def rowwise(width, pad=0, std=1.0, mean=0.0):
        t = normal(rows, width + pad, std=std, mean=mean).to(dt)
        return t[:, :width] if pad else t

    op = case["op"]
    d = {}
    if op.startswith("layernorm"):
        pd = _DTYPES[case["param"]]
        d["x"] = rowwise(c, case["pad"], std=1.5, mean=0.25)
        d["gamma"] = normal(c, std=0.2, mean=1.0).to(pd)
        if op == "layernorm_fwd":
            d["beta"] = normal(c, std=0.2).to(pd)
        else:
            d["dy"] = rowwise(c)
            # the forward pass's statistics
            x = d["x"].double()
            mean = x.mean(1)
            d["mean"] = mean.float()
            d["rstd"] = (1.0 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + _EPS)).float()
    elif op.startswith("gated"):
        f = case["f"]
        d["x"] = rowwise(c)
        d["wg"] = normal(f, c, std=c ** -0.5).to(dt)
        d["wu"] = normal(f, c, std=c ** -0.5).to(dt)
        if op == "gated_bwd":
            d["dy"] = rowwise(f)
    else:
        d["x"] = rowwise(c, case["pad"])
        if case["residual"]:
            d["residual"] = rowwise(c)
        d["seed"] = (seed * 0x9E3779B97F4A7C15 + 12345) & ((1 << 64) - 1)
        d["offset"] = (seed * 7919 + 5) & ((1 << 40) - 1)
    return d


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if own:
        from convolution_nhwc_amd import api
        # the workspace that a program keeps for its layer
        need = 0
        if case["op"] == "layernorm_bwd":
            need = api.layernorm_workspace(state["x"], state["gamma"])
        elif case["op"] == "gated_fwd":
            need = api.gated_workspace(state["x"], state["wg"], "fwd")
        elif case["op"] == "gated_bwd":
            need = api.gated_workspace(state["x"], state["wg"], "bwd")
        state["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return state


# ---- the operators -----------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from convolution_nhwc_amd import api
    case = s["case"]
    op = case["op"]
    if op == "layernorm_fwd":
        return api.layernorm(s["x"], s["gamma"], s["beta"], eps=_EPS)
    if op == "layernorm_bwd":
        return api.layernorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], ws=s["ws"])
    if op == "gated_fwd":
        return api.gated(s["x"], s["wg"], s["wu"], act=case["act"], ws=s["ws"])
    if op == "gated_bwd":
        return api.gated_bwd(s["dy"], s["x"], s["wg"], s["wu"], act=case["act"], ws=s["ws"])
    if op == "dropout":
        return api.dropout(s["x"], case["p"], s["seed"], s["offset"], residual=s.get("residual"))
    return api.dropout_bwd(s["x"], case["p"], s["seed"], s["offset"])


def _act(name, g):
    """act(g) and its derivative."""
    if name == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        pdf = torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
        return g * cdf, cdf + g * pdf
    s = 1.0 / (1.0 + torch.exp(-g))
    if name == "sigmoid":
        return s, s * (1.0 - s)
    return g * s, s * (1.0 + g * (1.0 - s))


def _philox_words(n, seed, offset):
    """Word i of the generator's stream for elements 0..n-1: four words a
    counter (element / 4, offset) under the key `seed`; int64 arithmetic whose
    wrapped 64-bit products keep all their bits."""
    blocks = torch.arange((n + 3) // 4, device="cuda", dtype=torch.int64)
    c0, c1 = blocks & _MASK32, blocks >> 32
    c2 = torch.full_like(blocks, offset & _MASK32)
    c3 = torch.full_like(blocks, (offset >> 32) & _MASK32)
    k0, k1 = seed & _MASK32, (seed >> 32) & _MASK32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & _MASK32) ^ c1 ^ k0, p1 & _MASK32,
                          ((p0 >> 32) & _MASK32) ^ c3 ^ k1, p0 & _MASK32)
        k0, k1 = (k0 + 0x9E3779B9) & _MASK32, (k1 + 0xBB67AE85) & _MASK32
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    dt = _DTYPES[case["dtype"]]
    if op == "layernorm_fwd":
        x = s["x"].float()
        mean = x.sum(1) / case["c"]
        d = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).sum(1) / case["c"] + _EPS)
        y = d * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        return y.to(dt), mean, rstd
    if op == "layernorm_bwd":
        pd = _DTYPES[case["param"]]
        dy = s["dy"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["gamma"].float()
        m1 = g.sum(1) / case["c"]
        m2 = (g * xhat).sum(1) / case["c"]
        dx = (g - m1[:, None] - xhat * m2[:, None]) * s["rstd"][:, None]
        return dx.to(dt), (dy * xhat).sum(0).to(pd), dy.sum(0).to(pd)
    if op == "gated_fwd":
        x = s["x"].float()
        a, _ = _act(case["act"], x @ s["wg"].float().t())
        return (a * (x @ s["wu"].float().t())).to(dt)
    if op == "gated_bwd":
        x, wg, wu, dy = (s[k].float() for k in ("x", "wg", "wu", "dy"))
        u = x @ wu.t()
        a, da = _act(case["act"], x @ wg.t())
        dg, du = dy * u * da, dy * a
        dx = dg @ wg + du @ wu
        return dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
    n = case["rows"] * case["c"]
    keep = _philox_words(n, s["seed"], s["offset"]) >= int(round(case["p"] * 2.0 ** 32))
    x = s["x"].float()
    y = torch.where(keep.reshape(x.shape), x * (1.0 / (1.0 - case["p"])), torch.zeros_like(x))
    if "residual" in s:
        y = y + s["residual"].float()
    return y.to(dt)


# ---- the definitions in 64 bits -----------------------------------------------

def _exact_keep(n, seed, offset, p):
    """The mask from Philox's published round function on 32-bit words held in
    numpy's unsigned 64-bit integers, on the host."""
    u = np.uint64
    low = u(_MASK32)
    e = np.arange((n + 3) // 4, dtype=np.uint64)
    x = [e & low, e >> u(32), np.full_like(e, offset & _MASK32), np.full_like(e, offset >> 32)]
    key = [seed & _MASK32, seed >> 32]
    for r in range(10):
        a = x[0] * u(0xD2511F53)
        b = x[2] * u(0xCD9E8D57)
        k0 = u((key[0] + r * 0x9E3779B9) & _MASK32)
        k1 = u((key[1] + r * 0xBB67AE85) & _MASK32)
        x = [(b >> u(32)) ^ x[1] ^ k0, b & low, (a >> u(32)) ^ x[3] ^ k1, a & low]
    words = np.stack(x, axis=1).reshape(-1)[:n]
    return words.astype(np.float64) >= float(round(p * 2.0 ** 32))


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    x = d["x"].double()
    if op == "layernorm_fwd":
        var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
        rstd = (var + _EPS).rsqrt()
        y = torch.addcmul(d["beta"].double(), (x - mean) * rstd, d["gamma"].double())
        return y, mean[:, 0], rstd[:, 0]
    if op == "layernorm_bwd":
        dy = d["dy"].double()
        r = d["rstd"].double()[:, None]
        xhat = (x - d["mean"].double()[:, None]) * r
        g = dy * d["gamma"].double()
        proj = torch.mean(g * xhat, dim=1, keepdim=True)
        dx = r * (g - torch.mean(g, dim=1, keepdim=True) - proj * xhat)
        return dx, torch.sum(dy * xhat, dim=0), torch.sum(dy, dim=0)
    if op.startswith("gated"):
        wg, wu = d["wg"].double(), d["wu"].double()
        g, u = torch.mm(x, wg.T), torch.mm(x, wu.T)
        act = case["act"]
        sg = torch.sigmoid(g)
        if act == "silu":
            a, da = g * sg, sg + g * sg * (1 - sg)
        elif act == "sigmoid":
            a, da = sg, sg * (1 - sg)
        elif act == "relu":
            a, da = g.clamp_min(0), (g > 0).double()
        else:
            phi = 0.5 * torch.erfc(-g / math.sqrt(2.0))
            a, da = g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        if op == "gated_fwd":
            return a * u
        dy = d["dy"].double()
        dg, du = dy * u * da, dy * a
        return torch.addmm(torch.mm(dg, wg), du, wu), torch.mm(dg.T, x), torch.mm(du.T, x)
    n = case["rows"] * case["c"]
    keep = torch.from_numpy(_exact_keep(n, d["seed"], d["offset"], case["p"])).cuda().reshape(x.shape)
    y = torch.where(keep, x / (1.0 - case["p"]), torch.zeros_like(x))
    return y + d["residual"].double() if case["residual"] else y
