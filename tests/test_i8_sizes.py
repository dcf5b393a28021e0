"""Workspace sizes and kernel names of the 8-bit products are those of the call that is
made: its activation and its strides count.  Host logic alone; no kernel is launched."""
import ctypes
import random

import pytest

from convolution_nhwc_amd import api

# how these are divided depends on the activation
DIVIDED = [(22638, 18152, 264), (27242, 25984, 342), (3652, 49043, 550), (2622, 8316, 1685), (632, 7981, 6726)]


def need(rows, c, f, act, xt=api.BF16, unaligned=0):
    q = api.LinearI8Problem(rows, c, f, 0, -(-c // 16) * 16, 0, 0, act, xt, api.BF16, 0)
    b = ctypes.c_size_t()
    assert api.lib().cnhwc_linear_i8_workspace_size(ctypes.byref(q), unaligned, ctypes.byref(b)) == api.OK
    return b.value


class Rows:
    """What the names of kernels need of a tensor of rows."""

    def __init__(self, rows, c, stride=None):
        self.shape, self.strides = (rows, c), (stride or c, 1)

    def dim(self):
        return 2

    def numel(self):
        return self.shape[0] * self.shape[1]

    def is_contiguous(self):
        return self.strides[0] == self.shape[1]

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]


@pytest.fixture
def sized(monkeypatch):
    """linear_i8_workspace and linear_i8_plan of sizes alone."""
    pytest.importorskip("torch")

    def of(rows, c, f, xt=api.BF16, unaligned=0):
        monkeypatch.setattr(api, "_linear_operands", lambda x, w: (rows, c, f, c, -(-c // 16) * 16, xt))
        monkeypatch.setattr(api, "_off16", lambda *t: unaligned)
    return of


@pytest.mark.parametrize("rows,c,f", DIVIDED)
def test_a_workspace_without_an_act_does_for_each(rows, c, f, sized):
    sized(rows, c, f)
    sizes = {name: need(rows, c, f, a) for name, a in api.ACTS_OR_NONE.items()}
    assert len(set(sizes.values())) > 1
    assert api.linear_i8_workspace(None, None) == max(sizes.values())
    for name, size in sizes.items():
        assert api.linear_i8_workspace(None, None, act=name) == size


@pytest.mark.parametrize("xt", [api.F16, api.F32, api.I8])
def test_workspaces_of_many_sizes(xt, sized):
    rng = random.Random(3)
    for _ in range(1500):
        rows, c, f = (min(int(2 ** rng.uniform(0, top)), most) for top, most in ((16, 65536), (17, 131071), (13, 8192)))
        unaligned = rng.randrange(2)
        sized(rows, c, f, xt, unaligned)
        enough = api.linear_i8_workspace(None, None)
        assert all(enough >= need(rows, c, f, a, xt, unaligned) for a in api.ACTS_OR_NONE.values())


def test_an_unknown_act_is_refused(sized):
    sized(100, 64, 32)
    for call in (api.linear_i8_workspace, api.linear_i8_plan):
        with pytest.raises(ValueError, match="act"):
            call(None, None, act="tanh")


def test_names_follow_the_act_and_the_strides(sized):
    sized(27242, 25984, 342)
    assert "split" not in api.linear_i8_plan(None, None) and "split" in api.linear_i8_plan(None, None, act="gelu")
    # rows of results that are not whole vectors go to the small tiles
    sized(16384, 2048, 8192)
    assert "t256" in api.linear_i8_plan(None, None)
    assert "t128" in api.linear_i8_plan(None, None, y=Rows(16384, 8192, 8195))
    assert "t128" in api.linear_i8_plan(None, None, residual=Rows(16384, 8192, 8193))
    assert "t256" in api.linear_i8_plan(None, None, residual=Rows(16384, 8192, 8200), y=Rows(16384, 8192))


@pytest.mark.parametrize("rows,c,stride,copied", [(5000, 100, 112, True), (5000, 112, 112, False), (5000, 112, 120, True),
                                                  (5000, 112, 128, False), (40, 100, 112, False)])
def test_codes_that_are_copied(rows, c, stride, copied):
    """An x of 8-bit integers goes to the tiles as it is where c and its rows are whole 16-byte units."""
    q = api.LinearI8Problem(rows, c, 64, stride, 112, 0, 0, -1, api.I8, api.BF16, 0)
    buf = ctypes.create_string_buffer(200)
    assert api.lib().cnhwc_linear_i8_plan(ctypes.byref(q), buf, 200) == api.OK
    assert ("i8_pack" in buf.value.decode()) == copied
