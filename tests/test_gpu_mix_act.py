"""The gated feed-forward block's activations on every kernel that evaluates
them: one pre-activation value an output column, against 64 bits within each
function's own error, forward and backward; and pre-activations that overflow."""
import pytest
import torch

import mix_act as ma
import mix_oracle as mo
import test_gpu_mix as tm
from convolution_nhwc_amd import api

pytestmark = pytest.mark.gpu

TYPES = mo.TYPES
NAMES = sorted(api.ACTS)


def check(got, ref, bound, what):
    """Every element of a GPU tensor within its bound; compared on the GPU."""
    ref, bound = ref.cuda(), bound.cuda()
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int(torch.where(bad, err / bound.clamp_min(1e-300), torch.zeros_like(err)).argmax())
        raise AssertionError("%s: %d of %d off, worst %.6g for %.6g, allowed %.3g" % (
            what, int(bad.sum()), bad.numel(), float(got.reshape(-1)[i]),
            float(ref.expand_as(got).reshape(-1)[i]), float(bound.expand_as(got).reshape(-1)[i])))


def sweep(name, t, rows, c, f, kernel, kernel_bwd=None):
    """Forward and backward of f pre-activation values; `kernel` is part of the
    projections' name in the plan."""
    t = TYPES[t]
    g = ma.values(f, t)
    host = ma.operands(g, rows, c, t)
    x, wg, wu, dy = (v.cuda() for v in host)
    assert kernel in api.gated_plan(x, wg).split()[-1], api.gated_plan(x, wg)
    ref, bound = ma.forward(name, g, t)
    check(api.gated(x, wg, wu, act=name), ref, bound, "y")
    plan = api.gated_plan(x, wg, "bwd").replace("pack ", "").split()[0]
    assert (kernel_bwd or kernel) in plan, plan
    for got, r, b, n in zip(api.gated_bwd(dy, x, wg, wu, act=name), *ma.backward(name, g, host[0], rows, t),
                            ("dx", "dwg", "dwu")):
        check(got, r, b, n)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("rows,c,f", [(1, 8, 4096), (20, 136, 4095), (64, 72, 2048)])
def test_few_rows(rows, c, f, t, name):
    sweep(name, t, rows, c, f, "gated_rows")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("tile,rows,c,f", [
    # more tiles than blocks, so that a tile's stores are in flight in the next
    # one; f a multiple of 8 and odd: whole and cut vectors
    (256, 513, 136, 16384), (256, 530, 72, 16383), (128, 300, 136, 16384), (128, 257, 64, 16381)])
def test_tiles(tile, rows, c, f, t, name):
    with api.override(tune=tile, split_c=1):
        sweep(name, t, rows, c, f, "_t%d" % tile)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("tile", [128, 256])
def test_joined_splits(tile, t, name):
    with api.override(tune=tile, split_c=3):
        sweep(name, t, 70, 200, 2050, "split3")


@pytest.mark.parametrize("rows,c,f", [(4000, 200, 2100), (600, 136, 1027)])
@pytest.mark.parametrize("name", NAMES)
def test_large_tile_with_cut_vectors(rows, c, f, name):
    """Random fp16 operands on the 256 tile where f is no multiple of 8."""
    with api.override(tune=256, split_c=1):
        x, wg = tm.check_gated_fwd(rows, c, f, name, torch.float16)
        assert api.gated_plan(x, wg) == "gated_proj_f16_t256"
        x, wg = tm.check_gated_bwd(rows, c, f, name, torch.float16)
        assert api.gated_plan(x, wg, "bwd").count("_t256") == 3


# ---- pre-activations that overflow ------------------------------------------------

INF = float("inf")
# act(+inf); act(-inf) (None: not tested, the formula is -inf * 0)
AT_INF = {"silu": (INF, None), "gelu": (INF, 0.0), "relu": (INF, 0.0), "sigmoid": (1.0, 0.0)}


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
    v, bound = ma.forward(name, torch.ones(1, dtype=torch.bfloat16), torch.bfloat16)
    assert bool(((y[:, 2::3] - v).abs() <= bound).all())


@pytest.mark.parametrize("rows,override", [(4, None), (64, None), (256, dict(tune=128, split_c=1)),
                                           (256, dict(tune=256, split_c=1)), (256, dict(tune=128, split_c=2))])
@pytest.mark.parametrize("name,up,down", [("gelu", 1.0, 0.0), ("relu", 1.0, 0.0), ("sigmoid", 0.0, 0.0)])
def test_slopes_of_overflowing_preactivations(name, up, down, rows, override):
    """The slope at both infinities, through dwg = dg^T x with u = dy = 1."""
    c, f = 128, 24
    x = torch.zeros(rows, c, dtype=torch.bfloat16)
    wg, wu = torch.zeros(f, c, dtype=torch.bfloat16), torch.zeros(f, c, dtype=torch.bfloat16)
    x[:, 5] = 2.0 ** 100
    x[:, 70] = 1.0
    wg[0::2, 5] = 2.0 ** 100
    wg[1::2, 5] = -2.0 ** 100
    wu[:, 70] = 1.0
    dy = torch.ones(rows, f, dtype=torch.bfloat16).cuda()
    ops = dy, x.cuda(), wg.cuda(), wu.cuda()
    if override is None:
        dwg = api.gated_bwd(*ops, act=name)[1]
    else:
        with api.override(**override):
            dwg = api.gated_bwd(*ops, act=name)[1]
    dwg = dwg.double().cpu()
    assert bool((dwg[0::2, 70] == up * rows).all()) and bool((dwg[1::2, 70] == down * rows).all()), dwg[:2, 70]
    assert bool((dwg[0::2, 5] == up * rows * 2.0 ** 100).all()) and bool((dwg[1::2, 5] == 0).all())
