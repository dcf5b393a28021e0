"""One workspace for a product with every activation, at sizes whose division depends on it."""
import pytest
import torch

from convolution_nhwc_amd import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,c,f", [(2622, 8316, 1685), (632, 7981, 6726), (700, 640, 1000)])
def test_a_workspace_for_every_act(rows, c, f):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, c, generator=g, device="cuda").bfloat16()
    w, scale = api.quantize_rows(torch.randn(f, c, generator=g, device="cuda"))
    need = api.linear_i8_workspace(x, w)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for act in api.ACTS_OR_NONE:
        y = api.linear_i8(x, w, scale, act=act, ws=ws)
        assert torch.equal(y, api.linear_i8(x, w, scale, act=act))
        # the act's own size suffices, and no less does
        own = api.linear_i8_workspace(x, w, act=act)
        assert own <= need
        assert torch.equal(y, api.linear_i8(x, w, scale, act=act, ws=ws[:own]))
        with pytest.raises(api.CnhwcError, match="workspace needs"):
            api.linear_i8(x, w, scale, act=act, ws=ws[:own - 1])
