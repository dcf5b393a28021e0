"""AdamW's step goes to where its tensors lie when it is made.  The tensors are on the
CPU and no kernel is launched: the step's list of addresses is what is looked at."""
import gc

import pytest

torch = pytest.importorskip("torch")

from convolution_nhwc_amd import api  # noqa: E402


@pytest.fixture
def steps(monkeypatch):
    """Every step's tensors as (p, p's type, g, m, v, scales, copy) of addresses."""
    made = []
    types = {torch.float32: api.F32, torch.float16: api.F16, torch.bfloat16: api.BF16}

    def operand(t, what):
        if t.dtype not in types:
            raise ValueError("%s must be float16, bfloat16 or float32" % what)
        return types[t.dtype]

    def enqueue(fn, device, prob, tensors, *scalars):
        made.append([(t.p, t.p_dtype, t.g, t.m, t.v, t.m_scale, t.v_scale, t.copy) for t in tensors])
    monkeypatch.setattr(api, "_operand", operand)
    monkeypatch.setattr(api, "_enqueue", enqueue)
    return made


class Case:
    def __init__(self, bits):
        self.p = [torch.zeros(n) for n in (1000, 300, 77)]
        self.copies = [None, torch.zeros(300).half(), torch.zeros(77).bfloat16()]
        self.g = [torch.ones(n) for n in (1000, 300, 77)]
        self.opt = api.AdamW(self.p, bits=bits, copies=self.copies)
        self.opt.bind(self.g)

    def where(self):
        """The addresses as the tensors have them now."""
        o, out = self.opt, []
        size = o.m.element_size()
        for i, (p, g, copy, at) in enumerate(zip(self.p, self.g, self.copies, o.offsets)):
            scales = [s.data_ptr() + at // 256 * 4 for s in o.scales] if o.bits == 8 else [None, None]
            out.append((p.data_ptr(), {torch.float32: api.F32, torch.float16: api.F16}[p.dtype], g.data_ptr(),
                        o.m.data_ptr() + at * size, o.v.data_ptr() + at * size, *scales, copy.data_ptr() if copy is not None else None))
        return out


@pytest.mark.parametrize("bits", [32, 8])
def test_exchanged_memory_is_followed(bits, steps):
    c = Case(bits)

    def check():
        c.opt.step(0.1)
        assert steps[-1] == c.where()
    check()
    keep = [c.p[0].data, c.copies[1].data, c.g[2].data]     # (so that none of it is given out again)
    c.p[0].data = torch.zeros(1000)
    check()
    c.p[1].data = torch.zeros(300).half()                    # of another type
    check()
    c.copies[1].set_(torch.zeros(300).half())
    check()
    c.g[2].data = torch.zeros(77)
    check()
    c.opt.m.data = c.opt.m.data.clone()
    check()
    c.opt.v.set_(c.opt.v.clone())
    check()
    assert c.opt.steps == 7 and keep


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_can_be_assigned(bits, steps):
    c = Case(bits)
    for name in ("m", "v") + ("scales",) * (bits == 8):
        t = torch.ones_like(getattr(c.opt, name))
        setattr(c.opt, name, t)
        assert getattr(c.opt, name) is t
        c.opt.step(0.1)
        assert steps[-1] == c.where()
        for bad in (t[:-1], t.double(), None):
            with pytest.raises(ValueError):
                setattr(c.opt, name, bad)
        assert getattr(c.opt, name) is t
        c.opt.step(0.1)
        assert steps[-1] == c.where()
    if bits == 32:
        assert c.opt.scales is None
        with pytest.raises(ValueError, match="scales"):
            c.opt.scales = torch.ones(2, 6)


def test_gradients_of_one_step_and_of_the_next(steps):
    """Tensors are followed whichever way their gradients come."""
    c = Case(32)
    keep = []

    def exchange(t):
        keep.append(t.data)
        t.data = t.data.clone()
    c.g = [torch.ones_like(p) for p in c.p]
    exchange(c.p[0])
    c.opt.step(0.1, c.g)
    assert steps[-1] == c.where()
    exchange(c.g[1])                      # used again without being given
    c.opt.step(0.1)
    assert steps[-1] == c.where()
    exchange(c.g[1])
    c.opt.step(0.1)
    assert steps[-1] == c.where()
    exchange(c.p[2])
    c.g = [torch.ones_like(p).half() for p in c.p]
    c.opt.bind(c.g)
    c.opt.step(0.1)
    assert steps[-1] == c.where()
    c.opt.step(0.1, c.g)
    c.g[0].data = torch.ones(5).half()
    c.opt.m = torch.zeros_like(c.opt.m)   # (the last step's gradients do not matter here)
    with pytest.raises(ValueError, match="grads"):
        c.opt.step(0.1)


def test_what_no_longer_fits_is_refused(steps):
    c = Case(32)
    c.opt.step(0.1)
    for t, what in ((c.p[1], "params"), (c.copies[1], "copies"), (c.g[1], "grads")):
        whole = t.data
        for other in (torch.zeros(299, dtype=t.dtype), torch.zeros(600, dtype=t.dtype)[::2]):
            t.data = other
            with pytest.raises(ValueError, match=what):
                c.opt.step(0.1)
        t.data = whole
        c.opt.step(0.1)
        assert steps[-1] == c.where()
    assert c.opt.steps == 4
    c.opt.m.data = torch.zeros(5)
    for call in (lambda: c.opt.step(0.1), c.opt.moments):
        with pytest.raises(ValueError, match="state m"):
            call()


def test_a_refused_assignment_changes_nothing(steps):
    """The new moments are fine, another tensor is not: the step stays with the old ones."""
    c = Case(32)
    m, last = c.opt.m, c.p[2].data
    c.p[2].data = torch.zeros(5)
    with pytest.raises(ValueError, match="params"):
        c.opt.m = torch.ones_like(m)
    c.p[2].data = last
    c.opt.step(0.1)
    assert c.opt.m is m and steps[-1] == c.where()


def test_no_other_tensor_comes_to_lie_at_an_old_address(steps):
    """Memory that a step may still compare with is held, so that it cannot be given out again."""
    c = Case(32)
    old = c.p[0].data_ptr()
    for n in (1000, 1000, 500, 1000, 250):
        c.p[0].data = torch.zeros(n)
        gc.collect()
        assert c.p[0].data_ptr() != old
    with pytest.raises(ValueError, match="params"):
        c.opt.step(0.1)
