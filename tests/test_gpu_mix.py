"""Layer norm, gated feed-forward and dropout on the GPU against the 64-bit
oracle, every element within the bounds that mix_oracle derives."""
import numpy as np
import pytest
import torch

import mix_oracle as mo
from convolution_nhwc_amd import api

pytestmark = pytest.mark.gpu

TYPES = mo.TYPES


def rnd(seed, *shape, std=1.0, mean=0.0):
    g = np.random.Generator(np.random.PCG64(seed))
    return torch.from_numpy(g.standard_normal(shape) * std + mean)


def put(v, t, pad=0, shift=0):
    """(device tensor, its values in 64 bits) of v [rows, c] rounded to t, with
    `pad` poisoned columns between rows and its base moved by `shift` elements."""
    r = v.to(t)
    rows, c = r.shape
    buf = torch.full((shift + rows * (c + pad),), float("nan"), dtype=t, device="cuda")
    d = buf[shift:].view(rows, c + pad)[:, :c]
    d.copy_(r)
    return d, r.double()


def vec(v, t):
    r = v.to(t)
    return r.cuda(), r.double()


def check(got, ref, bound, what):
    got = got.double().cpu()
    assert got.shape == ref.shape, what
    err = (got - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g against %.3g" % (
        what, int(bad.sum()), bad.numel(), float(err[bad].max()), float(bound[bad][err[bad].argmax()]))


# ---- layer norm -----------------------------------------------------------------

EPS = 1e-5

LN_SHAPES = [  # rows, c: every lane count and vector count, its ends, the looped rows
    (1, 1), (3, 2), (1, 8), (5, 7), (130, 64), (17, 128), (33, 129), (9, 384), (64, 385), (20, 512), (7, 513),
    (6, 1000), (11, 1537), (5, 2048), (4, 2049), (3, 4104), (5, 8192), (3, 8193), (2, 16384), (3, 16385), (2, 32768),
    (2, 32771), (1, 70001), (4100, 33), (2500, 520)]


@pytest.mark.parametrize("t,pt", [("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,c", LN_SHAPES)
def test_layernorm(rows, c, t, pt):
    t, pt = TYPES[t], TYPES[pt]
    seed = rows * 7 + c
    x, xr = put(rnd(seed, rows, c, std=1.5, mean=0.5), t)
    dy, dyr = put(rnd(seed + 1, rows, c), t)
    gamma, gr = vec(rnd(seed + 2, c, std=0.3, mean=1.0), pt)
    beta, br = vec(rnd(seed + 3, c), pt)
    y, mean, rstd = api.layernorm(x, gamma, beta, eps=EPS)
    ref = mo.layernorm(xr, gr, br, EPS)
    for g, r, b, n in zip((y, mean, rstd), ref, mo.layernorm_bound(xr, gr, br, EPS, t), ("y", "mean", "rstd")):
        check(g, r, b, n)
    mr, rr = mean.double().cpu(), rstd.double().cpu()
    got = api.layernorm_bwd(dy, x, mean, rstd, gamma)
    again = api.layernorm_bwd(dy, x, mean, rstd, gamma)
    for g, h, r, b, n in zip(got, again, mo.layernorm_bwd(dyr, xr, mr, rr, gr),
                             mo.layernorm_bwd_bound(dyr, xr, mr, rr, gr, t, pt), ("dx", "dgamma", "dbeta")):
        assert g.dtype == (t if n == "dx" else pt)
        check(g, r, b, n)
        assert torch.equal(g, h), n


@pytest.mark.parametrize("c,pad,shift", [(384, 8, 0), (385, 6, 1), (8, 1, 3), (1536, 0, 5), (5000, 3, 0), (40000, 1, 1)])
@pytest.mark.parametrize("t", ["f16", "f32"])
def test_layernorm_strides_and_alignment(c, pad, shift, t):
    """Rows out of a wider tensor, bases off 16 bytes; the gaps hold NaN and stay as they are."""
    t = TYPES[t]
    rows = 19
    x, xr = put(rnd(c, rows, c), t, pad, shift)
    dy, dyr = put(rnd(c + 1, rows, c), t, 2 * pad, shift)
    y = torch.full((rows, c + 4), 7.0, dtype=t, device="cuda")
    api.layernorm(x, eps=EPS, y=y[:, :c])
    ref, mean, rstd = mo.layernorm(xr, None, None, EPS)
    check(y[:, :c], ref, mo.layernorm_bound(xr, None, None, EPS, t)[0], "y")
    assert bool((y[:, c:] == 7.0).all())
    m, r = mean.float().cuda(), rstd.float().cuda()
    got = api.layernorm_bwd(dy, x, m, r)
    m, r = m.double().cpu(), r.double().cpu()
    for g, h, b, n in zip(got, mo.layernorm_bwd(dyr, xr, m, r, None),
                          mo.layernorm_bwd_bound(dyr, xr, m, r, None, t, t), ("dx", "dgamma", "dbeta")):
        check(g, h, b, n)


def test_layernorm_parts():
    """gamma or beta alone, statistics not wanted, single gradients, NHWC shapes."""
    t = torch.bfloat16
    x = rnd(3, 2, 5, 6, 48).to(t).cuda()
    xr = x.double().cpu().reshape(-1, 48)
    gamma, gr = vec(rnd(4, 48), t)
    y, mean, rstd = api.layernorm(x, gamma)
    assert y.shape == x.shape and mean.shape == (2, 5, 6)
    check(y.reshape(-1, 48), mo.layernorm(xr, gr, None, EPS)[0], mo.layernorm_bound(xr, gr, None, EPS, t)[0], "gamma")
    y, _, _ = api.layernorm(x, None, gamma)
    check(y.reshape(-1, 48), mo.layernorm(xr, None, gr, EPS)[0], mo.layernorm_bound(xr, None, gr, EPS, t)[0], "beta")
    dy = rnd(5, 2, 5, 6, 48).to(t).cuda()
    full = api.layernorm_bwd(dy, x, mean, rstd, gamma)
    import ctypes
    q = api.LayernormProblem(60, 48, 48, 48, 0.0, api.BF16, api.BF16, 0)
    st = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    for i in range(3):
        out = torch.zeros_like(full[i])
        p = [None, None, None]
        p[i] = out.data_ptr()
        api._check(api.lib().cnhwc_layernorm_bwd(
            ctypes.byref(q), dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            *p, ws.data_ptr() if i else None, ws.numel() if i else 0, st))
        assert torch.equal(out, full[i]), i


def test_layernorm_of_no_rows():
    x = torch.empty(0, 24, dtype=torch.float16, device="cuda")
    y, mean, rstd = api.layernorm(x)
    assert y.shape == (0, 24) and mean.shape == (0,)
    dx, dgamma, dbeta = api.layernorm_bwd(x, x, mean, rstd)
    assert dx.shape == (0, 24) and bool((dgamma == 0).all()) and bool((dbeta == 0).all())


def test_layernorm_constant_large_and_nonfinite_rows():
    t = torch.float32
    v = rnd(9, 6, 100)
    v[0] = 3.0                       # no variance: xhat is 0
    v[1] = v[1] * 1e-3 + 1000.0      # a mean far above the spread
    v[2] *= 1e15                     # squares near 1e30
    x, xr = put(v, t)
    y, mean, rstd = api.layernorm(x, eps=EPS)
    for g, r, b in zip((y, mean, rstd), mo.layernorm(xr, None, None, EPS), mo.layernorm_bound(xr, None, None, EPS, t)):
        check(g, r, b, "rows")
    assert bool((y[0] == 0).all())
    x[3, 5] = float("nan")
    x[4, 6] = float("inf")
    z, _, _ = api.layernorm(x, eps=EPS)
    assert bool(z[3].isnan().all()) and bool(z[4].isnan().any())
    assert torch.equal(z[[0, 1, 2, 5]], y[[0, 1, 2, 5]])      # other rows do not notice


def test_layernorm_rows_past_32_bits():
    """A row stride that puts the last rows more than 2^32 elements after the first."""
    rows, c, stride = 4100, 40, 1 << 20
    buf = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, stride)[:, :c]
    v = rnd(11, rows, c).to(torch.bfloat16)
    x.copy_(v)
    y, mean, rstd = api.layernorm(x, eps=EPS)
    xr = v.double()
    check(y, mo.layernorm(xr, None, None, EPS)[0], mo.layernorm_bound(xr, None, None, EPS, torch.bfloat16)[0], "y")


# ---- gated feed-forward -----------------------------------------------------------

def gated_operands(seed, rows, c, f, t, pad=0, shift=0):
    x = put(rnd(seed, rows, c), t, pad, shift)
    wg = put(rnd(seed + 1, f, c, std=c ** -0.5), t, 0, shift)
    wu = put(rnd(seed + 2, f, c, std=c ** -0.5), t, 0, shift)
    dy = put(rnd(seed + 3, rows, f), t, pad, shift)
    return x, wg, wu, dy


def check_gated_fwd(rows, c, f, name, t, pad=0, shift=0, seed=0):
    (x, xr), (wg, gr), (wu, ur), _ = gated_operands(seed + rows + c + f, rows, c, f, t, pad, shift)
    y = api.gated(x, wg, wu, act=name)
    check(y, mo.gated(xr, gr, ur, name), mo.gated_bound(xr, gr, ur, name, t), "y")
    assert torch.equal(y, api.gated(x, wg, wu, act=name))
    return x, wg


def check_gated_bwd(rows, c, f, name, t, pad=0, shift=0, seed=0):
    (x, xr), (wg, gr), (wu, ur), (dy, dyr) = gated_operands(seed + rows + c + f, rows, c, f, t, pad, shift)
    got = api.gated_bwd(dy, x, wg, wu, act=name)
    again = api.gated_bwd(dy, x, wg, wu, act=name)
    for g, h, r, b, n in zip(got, again, mo.gated_bwd(dyr, xr, gr, ur, name),
                             mo.gated_bwd_bound(dyr, xr, gr, ur, name, t), ("dx", "dwg", "dwu")):
        check(g, r, b, n)
        assert torch.equal(g, h), n
    return x, wg


@pytest.mark.parametrize("rows,c,f", [
    (1, 1, 1), (1, 64, 16), (1, 2048, 300), (2, 63, 17), (15, 129, 40), (16, 640, 64), (17, 65, 33), (24, 200, 550),
    (32, 1024, 100), (33, 100, 31), (64, 520, 48)])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_gated_few_rows(rows, c, f, t):
    x, wg = check_gated_fwd(rows, c, f, "silu", TYPES[t])
    assert api.gated_plan(x, wg).startswith("gated_rows")


@pytest.mark.parametrize("rows,c,f,rows_kernel", [(16, 4104, 40, True), (33, 2056, 72, False), (17, 2056, 65, False),
                                                  (40, 2061, 33, True), (64, 2048, 24, True)])
def test_gated_few_rows_of_many_channels(rows, c, f, rows_kernel):
    """Where x does not stay in registers: one 16-row tile, operands that tiles would copy first."""
    x, wg = check_gated_fwd(rows, c, f, "silu", torch.bfloat16)
    assert api.gated_plan(x, wg).startswith("gated_rows") == rows_kernel


@pytest.mark.parametrize("rows,c,f,rows_kernel", [
    (1, 1, 1, True), (1, 2048, 300, True), (9, 2049, 17, True), (16, 4200, 40, True), (17, 65, 33, True),
    (32, 2040, 100, True), (32, 2056, 48, False), (50, 2048, 20, True), (64, 520, 49, True), (60, 2056, 24, False)])
@pytest.mark.parametrize("name", ["silu", "relu"])
def test_gated_backward_projections_of_few_rows(rows, c, f, rows_kernel, name):
    x, wg = check_gated_bwd(rows, c, f, name, torch.float16)
    assert ("gated_rows" in api.gated_plan(x, wg, "bwd")) == rows_kernel


@pytest.mark.parametrize("name", sorted(api.ACTS))
def test_gated_activations(name):
    check_gated_fwd(9, 72, 40, name, torch.float16)
    check_gated_fwd(150, 72, 100, name, torch.bfloat16)
    check_gated_bwd(150, 72, 100, name, torch.float16)


@pytest.mark.parametrize("rows,c,f", [
    (65, 8, 8), (65, 64, 64), (128, 128, 64), (129, 72, 65), (200, 136, 72), (257, 200, 190), (300, 1, 1), (100, 7, 9),
    (130, 65, 129), (513, 264, 40), (97, 1000, 24)])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_gated_tiles(rows, c, f, t):
    check_gated_fwd(rows, c, f, "silu", TYPES[t])
    check_gated_bwd(rows, c, f, "silu", TYPES[t])


@pytest.mark.parametrize("rows,c,f", [(1, 24, 40), (2, 65, 9), (16, 128, 128), (63, 40, 200)])
def test_gated_backward_of_few_rows(rows, c, f):
    check_gated_bwd(rows, c, f, "gelu", torch.bfloat16)


@pytest.mark.parametrize("rows,c,f,t", [(4096, 72, 2048, "bf16"), (4000, 200, 2100, "f16")])
def test_gated_projections_on_the_large_tile(rows, c, f, t):
    x, wg = check_gated_fwd(rows, c, f, "silu", TYPES[t])
    assert "_t256" in api.gated_plan(x, wg) or c == 200


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("rows,c,f,splits", [
    (65, 8, 8, 1), (300, 200, 190, 1), (513, 130, 260, 1), (257, 520, 129, 1), (600, 72, 40, 1), (100, 7, 9, 1),
    (300, 650, 330, 2), (515, 330, 200, 3), (129, 1032, 65, 5), (1500, 64, 72, 4)])
def test_gated_tile_shapes(rows, c, f, splits, tile):
    """Both tiles, one to many steps (odd counts too), with and without split reductions."""
    with api.override(tune=tile, split_c=splits):
        x, wg = check_gated_bwd(rows, c, f, "silu", torch.bfloat16)
        check_gated_fwd(rows, c, f, "gelu", torch.float16)
        assert api.gated_plan(x, wg, "bwd").count("_t%d" % tile) == 3


@pytest.mark.parametrize("rows,c,f", [(8192, 2048, 40), (72, 4096, 2048), (200, 4000, 2100)])
def test_gated_gradients_of_many_tiles(rows, c, f):
    check_gated_bwd(rows, c, f, "silu", torch.bfloat16)


@pytest.mark.parametrize("rows,c,f,which", [(4500, 264, 2100, 0), (4480, 265, 2100, 0), (8400, 2048, 136, 1),
                                            (8300, 2040, 72, 1)])
def test_gated_rows_behind_whole_rounds(rows, c, f, which):
    """The rows past the last whole round of large tiles run on small ones."""
    x, wg = check_gated_bwd(rows, c, f, "silu", torch.float16)
    plan = api.gated_plan(x, wg, "bwd").replace("pack ", "").split()
    assert "+t128" in plan[which], plan
    if which == 0:
        check_gated_fwd(rows, c, f, "silu", torch.bfloat16)


@pytest.mark.parametrize("rows,c,f,which", [(70, 4096, 64, 0), (66, 2049, 40, 0), (65, 64, 4096, 1), (70, 40, 2050, 1),
                                            (6000, 64, 40, 2), (5001, 72, 65, 2)])
def test_gated_split_reductions(rows, c, f, which):
    x, wg = check_gated_bwd(rows, c, f, "silu", torch.float16)
    plan = api.gated_plan(x, wg, "bwd").replace("pack ", "").split()
    assert "split" in plan[which], plan
    if which == 0:
        check_gated_fwd(rows, c, f, "silu", torch.bfloat16)


@pytest.mark.parametrize("rows,c,f,joins", [(129, 513, 130, ()), (300, 512, 2048, ("dx",)), (4096, 64, 64, ("dw",)),
                                            (2000, 200, 700, ("dx", "dw")), (3137, 385, 1027, ("dx", "dw"))])
def test_gated_gradients_in_one_launch(rows, c, f, joins):
    """dx and the weights' gradients share a launch where neither fills the GPU; alone each has its own."""
    t = torch.bfloat16
    x, wg = check_gated_bwd(rows, c, f, "gelu", t)
    plan = api.gated_plan(x, wg, "bwd").split()
    assert {w for w in ("dx", "dw") if any(p.startswith("pair:gated_%s" % w) for p in plan)} == {"dx", "dw"}, plan
    assert {w for w in ("dx", "dw") if any("gated_%s" % w in p and "join" in p for p in plan)} == set(joins), plan
    (x, xr), (wg, gr), (wu, ur), (dy, dyr) = gated_operands(rows, rows, c, f, t)
    ref, bound = mo.gated_bwd(dyr, xr, gr, ur, "gelu"), mo.gated_bwd_bound(dyr, xr, gr, ur, "gelu", t)
    check(api.gated_bwd(dy, x, wg, wu, act="gelu", need_dw=False)[0], ref[0], bound[0], "dx")
    got = api.gated_bwd(dy, x, wg, wu, act="gelu", need_dx=False)
    check(got[1], ref[1], bound[1], "dwg")
    check(got[2], ref[2], bound[2], "dwu")


@pytest.mark.parametrize("rows,c,f,pad,shift", [(90, 64, 48, 8, 0), (90, 64, 48, 3, 0), (90, 64, 48, 0, 1),
                                                (90, 61, 45, 5, 3), (20, 64, 48, 3, 1)])
def test_gated_strides_and_alignment(rows, c, f, pad, shift):
    check_gated_fwd(rows, c, f, "silu", torch.float16, pad, shift)
    check_gated_bwd(rows, c, f, "silu", torch.float16, pad, shift)


def test_gated_writes_into_a_wider_tensor():
    t = torch.bfloat16
    (x, xr), (wg, gr), (wu, ur), _ = gated_operands(5, 100, 64, 72, t)
    y = torch.full((100, 80), 7.0, dtype=t, device="cuda")
    api.gated(x, wg, wu, y=y[:, :72])
    check(y[:, :72], mo.gated(xr, gr, ur, "silu"), mo.gated_bound(xr, gr, ur, "silu", t), "y")
    assert bool((y[:, 72:] == 7.0).all())


def test_gated_parts_and_filters():
    """Single gradients equal the full call's; [f, 1, 1, c] filters and NHWC shapes."""
    t = torch.float16
    (x, _), (wg, _), (wu, _), (dy, _) = gated_operands(6, 120, 40, 56, t)
    full = api.gated_bwd(dy, x, wg, wu)
    dx, none1, none2 = api.gated_bwd(dy, x, wg, wu, need_dw=False)
    assert none1 is None and none2 is None and torch.equal(dx, full[0])
    none, dwg, dwu = api.gated_bwd(dy, x, wg, wu, need_dx=False)
    assert none is None and torch.equal(dwg, full[1]) and torch.equal(dwu, full[2])
    y = api.gated(x.view(2, 6, 10, 40), wg.view(56, 1, 1, 40), wu.view(56, 1, 1, 40))
    assert y.shape == (2, 6, 10, 56) and torch.equal(y.view(120, 56), api.gated(x, wg, wu))


def test_gated_of_no_rows():
    t = torch.float16
    x = torch.empty(0, 24, dtype=t, device="cuda")
    w = torch.ones(30, 24, dtype=t, device="cuda")
    assert api.gated(x, w, w).shape == (0, 30)
    dx, dwg, dwu = api.gated_bwd(torch.empty(0, 30, dtype=t, device="cuda"), x, w, w)
    assert dx.shape == (0, 24) and bool((dwg == 0).all()) and bool((dwu == 0).all())


@pytest.mark.parametrize("rows", [10, 300])
def test_gated_nonfinite_rows_stay_in_their_rows(rows):
    t = torch.bfloat16
    (x, _), (wg, _), (wu, _), (dy, _) = gated_operands(7, rows, 40, 60, t)
    y = api.gated(x, wg, wu)
    dx = api.gated_bwd(dy, x, wg, wu, need_dw=False)[0]
    x2 = x.clone()
    x2[3, 7] = float("nan")
    x2[5, 8] = float("inf")
    other = [r for r in range(rows) if r not in (3, 5)]
    y2 = api.gated(x2, wg, wu)
    assert bool(y2[3].isnan().all()) and torch.equal(y2[other], y[other])
    dx2 = api.gated_bwd(dy, x2, wg, wu, need_dw=False)[0]
    assert bool(dx2[3].isnan().all()) and torch.equal(dx2[other], dx[other])


def test_gated_saturated_activations():
    """Pre-activations of some hundred: exp over- and underflows, results do not."""
    t = torch.bfloat16
    x, xr = put(torch.tensor([[300.0], [-300.0], [80.0], [-80.0], [0.0]]).double().repeat(20, 1), t)
    w, wr = put(torch.ones(8, 1).double(), t)
    for name in api.ACTS:
        for n in (5, 100):
            y = api.gated(x[:n], w, w, act=name)
            check(y, mo.gated(xr[:n], wr, wr, name), mo.gated_bound(xr[:n], wr, wr, name, t), name)
        dy = torch.ones(100, 8, dtype=t, device="cuda")
        got = api.gated_bwd(dy, x, w, w, act=name)
        for g, r, b in zip(got, mo.gated_bwd(dy.double().cpu(), xr, wr, wr, name),
                           mo.gated_bwd_bound(dy.double().cpu(), xr, wr, wr, name, t)):
            check(g, r, b, name)


def test_gated_rows_past_32_bits():
    rows, c, f, stride = 2100, 40, 24, 1 << 21
    t = torch.bfloat16
    buf = torch.empty(rows * stride, dtype=t, device="cuda")
    x = buf.view(rows, stride)[:, :c]
    _, (wg, gr), (wu, ur), (dy, dyr) = gated_operands(8, rows, c, f, t)
    v = rnd(12, rows, c).to(t)
    x.copy_(v)
    xr = v.double()
    check(api.gated(x, wg, wu), mo.gated(xr, gr, ur, "silu"), mo.gated_bound(xr, gr, ur, "silu", t), "y")
    for g, r, b in zip(api.gated_bwd(dy, x, wg, wu), mo.gated_bwd(dyr, xr, gr, ur, "silu"),
                       mo.gated_bwd_bound(dyr, xr, gr, ur, "silu", t)):
        check(g, r, b, "gradients")


# ---- dropout -----------------------------------------------------------------------

def check_dropout(rows, c, t, p, seed, offset, residual, pad=0, shift=0):
    t = TYPES[t]
    x, xr = put(rnd(rows + c, rows, c), t, pad, shift)
    r, rr = put(rnd(rows + c + 1, rows, c), t, 2 * pad, shift) if residual else (None, None)
    y = api.dropout(x, p, seed, offset, residual=r)
    ref = mo.dropout(xr, p, seed, offset, rr)
    scale = 1 / (1 - p) if p < 1 else 0.0
    # the scale, the product and the sum round in fp32
    bound = mo.half_step(t, ref) + 4 * mo.U32 * (xr.abs() * scale + (0 if rr is None else rr.abs()))
    check(y, ref, bound, "y")
    keep = mo.keep(0, rows * c, p, seed, offset).reshape(rows, c)
    want = torch.zeros(rows, c, dtype=t) if r is None else r.cpu()
    assert torch.equal(y.cpu()[~keep], want[~keep])


@pytest.mark.parametrize("rows,c", [(1, 1), (1, 3), (3, 5), (7, 8), (2, 1000), (13, 385), (600, 384), (50, 2048)])
@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(rows, c, t, residual):
    check_dropout(rows, c, t, 0.1, 0x123456789ABCDEF0, (5 << 40) + 3, residual)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -40, 0.5, 1 - 2.0 ** -33, 1.0])
def test_dropout_probabilities(p):
    check_dropout(11, 100, "f32", p, (1 << 64) - 1, (1 << 64) - 1, True)


@pytest.mark.parametrize("c,pad,shift", [(384, 8, 0), (385, 3, 1), (3, 1, 0), (1, 4, 1), (8, 1, 3), (1000, 0, 5)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_dropout_strides_and_alignment(c, pad, shift, t):
    """The mask does not depend on where rows lie."""
    check_dropout(23, c, t, 0.25, 77, 9, True, pad, shift)
    check_dropout(23, c, t, 0.25, 77, 9, False, pad, shift)


def test_dropout_backward_draws_the_same_mask():
    x = torch.ones(40, 96, device="cuda")
    y = api.dropout(x, 0.3, 5, 6)
    dx = api.dropout_bwd(torch.full_like(x, 2.0), 0.3, 5, 6)
    assert torch.equal(dx, 2 * y) and not torch.equal(y, api.dropout(x, 0.3, 5, 7))


def test_dropout_drops_nonfinite_values():
    x = torch.ones(64, 64, device="cuda")
    keep = mo.keep(0, 4096, 0.5, 1, 0).reshape(64, 64).cuda()
    x[~keep] = float("nan")
    x[0][~keep[0]] = float("inf")
    assert torch.equal(api.dropout(x, 0.5, 1), torch.where(keep, 2.0, 0.0))
    assert bool((api.dropout(torch.full_like(x, float("nan")), 1.0, 1) == 0).all())


def test_dropout_in_place():
    x, r = rnd(1, 30, 70).float().cuda(), rnd(2, 30, 70).float().cuda()
    want = api.dropout(x, 0.4, 3, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(api.dropout(a, 0.4, 3, residual=r, y=a), want)
    assert torch.equal(api.dropout(x, 0.4, 3, residual=b, y=b), want)


def test_dropout_elements_past_32_bits():
    """The last elements of a tensor of more than 2^32."""
    rows, c = (1 << 17) + 3, 32771
    x = torch.ones(rows, c, dtype=torch.float16, device="cuda")
    y = api.dropout(x, 0.5, 21, 4, y=x)
    first = (rows - 4) * c
    assert first > 1 << 32
    keep = mo.keep(first, 4 * c, 0.5, 21, 4).reshape(4, c)
    assert torch.equal(y[-4:].cpu(), torch.where(keep, 2.0, 0.0).half())


# ---- streams and graphs ---------------------------------------------------------------

def test_another_stream():
    t = torch.bfloat16
    (x, _), (wg, _), (wu, _), (dy, _) = gated_operands(9, 200, 64, 96, t)
    gamma = torch.ones(64, dtype=t, device="cuda")

    def everything():
        n, mean, rstd = api.layernorm(x, gamma)
        h = api.gated(n, wg, wu)
        g = api.gated_bwd(dy, n, wg, wu)
        return (h, *g, *api.layernorm_bwd(g[0], x, mean, rstd, gamma), api.dropout(h, 0.2, 4))
    want = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = everything()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_graph_replays():
    """A captured step: each replay equals the eager calls on the inputs of the
    moment, and device_offset gives it a new mask."""
    t = torch.float16
    (x, _), (wg, _), (wu, _), (dy, _) = gated_operands(10, 6000, 40, 65, t)   # split dw, packed operands
    gamma = torch.ones(40, dtype=t, device="cuda")
    count = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        n, mean, rstd = api.layernorm(x, gamma)
        h = api.dropout(api.gated(n, wg, wu), 0.2, 4, 100, device_offset=count)
        g = api.gated_bwd(api.dropout_bwd(dy, 0.2, 4, 100, device_offset=count), n, wg, wu)
        return (h, *g, *api.layernorm_bwd(g[0], x, mean, rstd, gamma))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    masks = []
    for i in range(4):
        x.copy_(rnd(100 + i, 6000, 40).to(t))
        count.fill_(i)
        want = [v.clone() for v in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i
        masks.append(out[0] == 0)
    assert not torch.equal(masks[0], masks[1])
