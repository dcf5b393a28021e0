"""Host checks of the channel-mixing entry points: refusals with their reasons,
workspace sizes and kernel choices.  Nothing here launches a kernel."""
import ctypes

import pytest
import torch

from convolution_nhwc_amd import api

OK, BAD, SMALL, MIS = api.OK, api.INVALID_ARG, api.WORKSPACE_TOO_SMALL, api.MISALIGNED
A, B, C, D, E, F = (1 << 40, 2 << 40, 3 << 40, 4 << 40, 5 << 40, 6 << 40)   # far apart, never dereferenced


def ln(rows=4, c=16, xs=0, ys=0, eps=1e-5, dtype=api.F16, param=api.F16, reserved=0):
    return api.LayernormProblem(rows, c, xs, ys, eps, dtype, param, reserved)


def gp(rows=100, c=64, f=96, xs=0, ys=0, act=0, dtype=api.BF16, reserved=0):
    return api.GatedProblem(rows, c, f, xs, ys, act, dtype, reserved)


def dp(rows=4, c=16, xs=0, rs=0, ys=0, p=0.5, dtype=api.F16, reserved=0):
    return api.DropoutProblem(rows, c, xs, rs, ys, p, 1, 2, dtype, reserved)


def refused(status, code, reason):
    assert status == code, (status, api.last_error())
    assert reason in api.last_error(), api.last_error()


def ln_fwd(q, x=A, gamma=None, beta=None, y=B, mean=None, rstd=None):
    return api.lib().cnhwc_layernorm_fwd(ctypes.byref(q), x, gamma, beta, y, mean, rstd, None)


def ln_bwd(q, dy=A, x=B, gamma=None, mean=C, rstd=D, dx=E, dgamma=None, dbeta=None, ws=None, n=0):
    return api.lib().cnhwc_layernorm_bwd(ctypes.byref(q), dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, n, None)


@pytest.mark.parametrize("q,reason", [
    (ln(rows=-1), "rows must be >= 0"), (ln(c=0), "c must be in"), (ln(c=1 << 31), "c must be in"),
    (ln(eps=-1.0), "eps"), (ln(eps=float("nan")), "eps"), (ln(eps=float("inf")), "eps"), (ln(dtype=7), "dtype"),
    (ln(param=api.BF16), "param_dtype"), (ln(xs=15), "x_stride"), (ln(ys=-16), "y_stride"), (ln(reserved=1), "reserved"),
    (ln(rows=1 << 40, xs=1 << 40), "address range")])
def test_layernorm_refuses_descriptors(q, reason):
    refused(ln_fwd(q), BAD, reason)
    refused(ln_bwd(q), BAD, reason)
    refused(api.lib().cnhwc_layernorm_workspace_size(ctypes.byref(q), None), BAD, reason)


def test_layernorm_refuses_pointers():
    refused(ln_fwd(ln(), x=None), BAD, "x is NULL")
    refused(ln_fwd(ln(), y=None), BAD, "y is NULL")
    refused(ln_fwd(ln(), x=A + 1), MIS, "x is not 2-byte")
    refused(ln_fwd(ln(dtype=api.F32, param=api.F32), y=B + 2), MIS, "y is not 4-byte")
    refused(ln_fwd(ln(), y=A + 64), BAD, "y overlaps x")
    refused(ln_fwd(ln(), mean=C, rstd=C + 12), BAD, "rstd overlaps mean")
    refused(ln_fwd(ln(), mean=C + 2), MIS, "mean")
    refused(ln_bwd(ln(), dx=None), BAD, "all NULL")
    refused(ln_bwd(ln(), mean=None), BAD, "mean is NULL")
    refused(ln_bwd(ln(), dx=A), BAD, "dx overlaps dy")
    need = ctypes.c_size_t()
    assert api.lib().cnhwc_layernorm_workspace_size(ctypes.byref(ln()), ctypes.byref(need)) == OK
    assert need.value == 4 * 2 * 16 * 4 or need.value == 2 * 16 * 4     # at most one partial row a row
    refused(ln_bwd(ln(), dgamma=F), BAD, "workspace is NULL")
    refused(ln_bwd(ln(), dgamma=F, ws=7 << 40, n=need.value - 1), SMALL, "workspace needs")
    refused(ln_bwd(ln(), dgamma=F, ws=(7 << 40) + 8, n=need.value), MIS, "workspace")
    refused(ln_bwd(ln(), dgamma=F, ws=E, n=need.value), BAD, "workspace overlaps dx")


def test_layernorm_of_no_rows_needs_no_pointers():
    assert ln_fwd(ln(rows=0), x=None, y=None) == OK
    assert ln_bwd(ln(rows=0), dy=None, x=None, mean=None, rstd=None, dx=E) == OK


def test_layernorm_workspace_is_bounded():
    """The partial sums stay a small part of the tensors, whatever the shape."""
    need = ctypes.c_size_t()
    for rows in (1, 2, 255, 4096, 50176, 1 << 24):
        for c in (1, 7, 384, 1537, 8192, 16385, 40000):
            assert api.lib().cnhwc_layernorm_workspace_size(ctypes.byref(ln(rows, c)), ctypes.byref(need)) == OK
            assert 8 * c <= need.value <= 8 * c * min(rows, 1024)


def g_fwd(q, x=A, wg=B, wu=C, y=D, ws=None, n=0):
    return api.lib().cnhwc_gated_fwd(ctypes.byref(q), x, wg, wu, y, ws, n, None)


def g_bwd(q, dy=A, x=B, wg=C, wu=D, dx=E, dwg=F, dwu=7 << 40, ws=None, n=0):
    return api.lib().cnhwc_gated_bwd(ctypes.byref(q), dy, x, wg, wu, dx, dwg, dwu, ws, n, None)


def g_need(q, op=api.OP_FWD, unaligned=0):
    b = ctypes.c_size_t()
    assert api.lib().cnhwc_gated_workspace_size(ctypes.byref(q), op, unaligned, ctypes.byref(b)) == OK
    return b.value


def g_plan(q, op=api.OP_FWD):
    buf = ctypes.create_string_buffer(256)
    assert api.lib().cnhwc_gated_plan(ctypes.byref(q), op, buf, 256) == OK
    return buf.value.decode()


@pytest.mark.parametrize("q,reason", [
    (gp(rows=-2), "rows must be >= 0"), (gp(rows=1 << 31), "rows must be < 2^31"), (gp(c=0), "c must be"),
    (gp(f=(1 << 20) + 1), "f must be"), (gp(act=4), "act"), (gp(act=-1), "act"), (gp(dtype=api.F32), "dtype"),
    (gp(xs=63), "x_stride"), (gp(ys=95), "y_stride"), (gp(xs=(1 << 21) + 8), "x_stride"), (gp(reserved=3), "reserved")])
def test_gated_refuses_descriptors(q, reason):
    refused(g_fwd(q), BAD, reason)
    refused(g_bwd(q), BAD, reason)
    refused(api.lib().cnhwc_gated_workspace_size(ctypes.byref(q), api.OP_FWD, 0, None), BAD, reason)
    refused(api.lib().cnhwc_gated_plan(ctypes.byref(q), api.OP_FWD, None, 0), BAD, reason)


def test_gated_refuses_pointers_and_workspaces():
    refused(g_fwd(gp(), x=None), BAD, "x is NULL")
    refused(g_fwd(gp(), wu=None), BAD, "wu is NULL")
    refused(g_fwd(gp(), y=D + 1), MIS, "y is not 2-byte")
    refused(g_fwd(gp(), y=B), BAD, "y overlaps wg")
    refused(g_bwd(gp(), dwu=None), BAD, "both")
    refused(g_bwd(gp(), dx=None, dwg=None, dwu=None), BAD, "all NULL")
    refused(g_bwd(gp(), dwg=E + 2), BAD, "dwg overlaps dx")
    need = g_need(gp(), api.OP_DGRAD)
    assert need >= 100 * 2 * 96 * 2
    refused(g_bwd(gp()), BAD, "workspace is NULL")
    refused(g_bwd(gp(), ws=8 << 40, n=need - 1), SMALL, "workspace needs")
    refused(g_bwd(gp(), ws=C, n=need), BAD, "workspace overlaps wg")
    # the copies that odd widths and unaligned bases need
    odd = gp(c=63)
    assert g_need(odd) >= (100 + 2 * 96) * 64 * 2
    assert g_need(gp(), unaligned=1) >= g_need(gp()) + (100 + 2 * 96) * 64 * 2
    refused(g_fwd(odd), BAD, "workspace is NULL")
    refused(g_fwd(gp(), x=A + 2), BAD, "workspace is NULL")
    refused(api.lib().cnhwc_gated_workspace_size(ctypes.byref(gp()), api.OP_WGRAD, 0, None), BAD, "op must be")


def test_gated_of_no_rows():
    assert g_fwd(gp(rows=0), x=None, y=None) == OK
    assert g_bwd(gp(rows=0), dy=None, x=None, dx=E, dwg=None, dwu=None) == OK
    assert g_plan(gp(rows=0)) == "none" and g_need(gp(rows=0), api.OP_DGRAD) == 0


def test_gated_plans():
    for rows in (1, 16, 17, 64):
        assert g_plan(gp(rows=rows, c=2048, f=8192)) == "gated_rows_bf16"
        assert g_need(gp(rows=rows, c=2047, f=8191), unaligned=1) == 0
    assert g_plan(gp(rows=16384, c=2048, f=8192)) == "gated_proj_bf16_t256"
    for i, part in enumerate(g_plan(gp(rows=8192, c=2048, f=8192), api.OP_DGRAD).split()):
        assert part == "gated_%s_bf16_t256" % ("proj", "dx", "dw")[i]
    assert g_plan(gp(rows=200, c=65, f=96)).startswith("pack ")
    # few tiles over a deep reduction are split
    assert "split" in g_plan(gp(rows=65, c=8192, f=256))
    assert "dw_bf16" in g_plan(gp(rows=50176, c=64, f=64), api.OP_DGRAD) and \
        "split" in g_plan(gp(rows=50176, c=64, f=64), api.OP_DGRAD).split()[-1]


def drop(q, x=A, res=None, y=B, off=None):
    return api.lib().cnhwc_dropout(ctypes.byref(q), x, res, y, off, None)


@pytest.mark.parametrize("q,reason", [
    (dp(rows=-1), "rows"), (dp(c=0), "c must be"), (dp(p=-0.1), "p must be"), (dp(p=1.5), "p must be"),
    (dp(p=float("nan")), "p must be"), (dp(dtype=5), "dtype"), (dp(xs=3), "x_stride"), (dp(rs=3), "residual_stride"),
    (dp(ys=3), "y_stride"), (dp(reserved=1), "reserved")])
def test_dropout_refuses_descriptors(q, reason):
    refused(drop(q), BAD, reason)


def test_dropout_refuses_pointers():
    refused(drop(dp(), x=None), BAD, "x is NULL")
    refused(drop(dp(), y=None), BAD, "y is NULL")
    refused(drop(dp(), y=A + 2), BAD, "y overlaps x")
    refused(drop(dp(ys=32), y=A), BAD, "y overlaps x")
    refused(drop(dp(), res=B + 2), BAD, "y overlaps residual")
    refused(drop(dp(), off=C + 4), MIS, "device_offset")
    assert drop(dp(rows=0), x=None, y=None) == OK


def test_python_layer_refuses():
    """The tensor conveniences check before they call."""
    x = torch.zeros(4, 8, dtype=torch.float16)
    for call in (lambda: api.layernorm(x), lambda: api.gated(x, x, x), lambda: api.dropout(x, 0.5, 1)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="GPU tensor"):
        api.layernorm_workspace(x)
    with pytest.raises(ValueError, match="not contiguous"):
        api._rows(torch.zeros(4, 8).t(), "x")
    with pytest.raises(ValueError, match="step evenly"):
        api._rows(torch.zeros(2, 3, 8).transpose(0, 1), "x")
    with pytest.raises(ValueError, match="overlap"):
        api._rows(torch.zeros(8).as_strided((4, 4), (1, 1)), "x")
    assert api._rows(torch.zeros(2, 3, 5, 8)[..., 2:6], "x") == (30, 4, 8)
    assert api._rows(torch.zeros(2, 1, 5, 8)[:, :, 1:2], "x") == (2, 8, 40)
    assert api._rows(torch.zeros(8), "x") == (1, 8, 8)
    assert api._rows(torch.zeros(0, 8), "x") == (0, 8, 8)
    with pytest.raises(ValueError, match="rows overlap"):
        api._rows(torch.zeros(1, 8).expand(4, 8), "x")
