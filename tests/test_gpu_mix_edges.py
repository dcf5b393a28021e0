"""Calls at the edges of the channel-mixing operators: what the ordinary tests'
sizes, values and arguments do not reach."""
import ctypes

import pytest
import torch

import mix_oracle as mo
from convolution_nhwc_amd import api

pytestmark = pytest.mark.gpu

TYPES = mo.TYPES


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("c", [1, 8, 24, 70, 385, 1537, 2056, 5001, 9000, 20001])
def test_layernorm_backward_of_constant_rows_far_from_zero(c, t):
    """mean * rstd is past fp32's largest value, (x - mean) * rstd is 0: lanes without a column
    must not bring the former into the row's sums."""
    t = TYPES[t]
    rows, big, rstd = 21, 2.0 ** 110, 2.0 ** 20
    x = torch.full((rows, c), big, dtype=t)
    mean, r = torch.full((rows,), big), torch.full((rows,), rstd)
    dy = rnd(c, rows, c).to(t)
    g = dy.double()
    dx, dgamma, dbeta = api.layernorm_bwd(dy.cuda(), x.cuda(), mean.cuda(), r.cuda())
    m1 = g.mean(1, keepdim=True)
    ref = rstd * (g - m1)
    size = g.abs().mean(1, keepdim=True)
    # m1 by a sum of c terms and a division, the difference and the product
    bound = mo.half_step(t, ref) + rstd * (mo.chain(c) * size + 4 * mo.U32 * (g.abs() + size))
    assert bool(((dx.double().cpu() - ref).abs() <= bound).all())
    assert bool((dgamma == 0).all())
    sums = mo.half_step(t, g.sum(0)) + mo.chain(rows) * g.abs().sum(0)
    assert bool(((dbeta.double().cpu() - g.sum(0)).abs() <= sums).all())


@pytest.mark.parametrize("rows", [9, 90])
def test_gated_workspace_of_weights_apart(rows):
    """wu off a 16-byte boundary beside an aligned wg, as in one buffer of many weights."""
    t = torch.bfloat16
    c, f = 64, 40
    x = rnd(1, rows, c).to(t).cuda()
    flat = torch.empty(2 * f * c + 3, dtype=t, device="cuda")
    wg, wu = flat[:f * c].view(f, c), flat[f * c + 3:].view(f, c)
    wg.copy_(rnd(2, f, c))
    wu.copy_(rnd(3, f, c))
    dy = rnd(4, rows, f).to(t).cuda()
    same = wu.clone()
    for which, call in (("fwd", lambda u, ws: (api.gated(x, wg, u, ws=ws),)),
                        ("bwd", lambda u, ws: api.gated_bwd(dy, x, wg, u, ws=ws))):
        ws = torch.empty(api.gated_workspace(x, wg, which, wu), dtype=torch.uint8, device="cuda")
        for got, want in zip(call(wu, ws), call(same, None)):
            assert torch.equal(got, want)


@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,c", [(1, 1), (37, 70), (300, 384), (5, 2056), (3, 9000), (2, 40000)])
def test_layernorm_without_statistics(rows, c, t):
    """mean, rstd or both NULL: y has the same bits, and the statistic that is asked for too."""
    code, t = {"f16": api.F16, "bf16": api.BF16, "f32": api.F32}[t], TYPES[t]
    x, gamma, beta = (rnd(i, *s).to(t).cuda() for i, s in enumerate(((rows, c), (c,), (c,))))
    want = api.layernorm(x, gamma, beta)
    q = api.LayernormProblem(rows, c, 0, 0, 1e-5, code, code, 0)
    for asked in ((0, 0), (1, 0), (0, 1)):
        y = torch.full_like(x, float("nan"))
        stats = [torch.full((rows,), float("nan"), device="cuda") for _ in range(2)]
        api._check(api.lib().cnhwc_layernorm_fwd(
            ctypes.byref(q), x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), y.data_ptr(),
            *(s.data_ptr() if a else None for s, a in zip(stats, asked)), torch.cuda.current_stream().cuda_stream))
        assert torch.equal(y, want[0]), asked
        for s, a, w in zip(stats, asked, want[1:]):
            assert torch.equal(s, w) if a else bool(s.isnan().all()), asked
