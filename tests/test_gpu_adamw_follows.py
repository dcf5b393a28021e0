"""AdamW with tensors whose memory is exchanged between steps, against one whose is not."""
import pytest
import torch

from convolution_nhwc_amd import api

pytestmark = pytest.mark.gpu

SIZES = (1000, 300, 5000)


def new(bits):
    g = torch.Generator().manual_seed(4)
    p = [torch.randn(n, generator=g).cuda() for n in SIZES]
    copies = [v.bfloat16() for v in p]
    grads = [torch.randn(n, generator=g).cuda() for n in SIZES]
    opt = api.AdamW(p, bits=bits, copies=copies, seed=9)
    opt.bind(grads)
    return p, copies, grads, opt


@pytest.mark.parametrize("bits", [32, 8])
def test_results_do_not_depend_on_where_tensors_lie(bits):
    ours, theirs = new(bits), new(bits)

    def step():
        for _, _, _, opt in (ours, theirs):
            opt.step(0.01)
        for a, b in zip(ours[:2], theirs[:2]):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
        assert all(torch.equal(u, v) for u, v in zip(ours[3].moments(), theirs[3].moments()))
    step()
    p, copies, grads, opt = ours
    old = [t.clone() for t in (p[1], copies[2])]
    kept = [p[1].data, copies[2].data]
    p[1].data = p[1].data.clone()
    copies[2].set_(copies[2].clone())
    grads[0].data = grads[0].data.clone()
    step()
    assert all(torch.equal(a, b) for a, b in zip(old, kept))     # the memory of before is left alone
    opt.m = opt.m.clone()
    opt.v = opt.v.clone()
    if bits == 8:
        opt.scales = opt.scales.clone()
    step()
    # a run that goes on from saved moments
    saved = [t.clone() for t in (opt.m, opt.v) + ((opt.scales,) if bits == 8 else ())]
    values = [[t.clone() for t in ts] for ts in (p, copies)]
    step()
    after = [t.clone() for t in p]
    for ts, vs in zip((p, copies), values):
        for t, v in zip(ts, vs):
            t.copy_(v)
    for name, t in zip(("m", "v", "scales"), saved):
        setattr(opt, name, t)
    opt.steps -= 1
    opt.step(0.01)
    assert all(torch.equal(a, b) for a, b in zip(p, after))
