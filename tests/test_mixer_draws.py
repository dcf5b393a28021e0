"""The residual block's two kinds of draws, the dropout's mask and the rounding of 8-bit
moments, have nothing to do with each other.  Nothing runs on a GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import adamw_oracle as ao  # noqa: E402
from convolution_nhwc_amd import api, mixer  # noqa: E402


@pytest.fixture
def keys(monkeypatch):
    """The seeds that optimizers are made with."""
    made = []
    monkeypatch.setattr(api, "AdamW", lambda params, seed=0, **kw: made.append(seed))
    return made


@pytest.mark.parametrize("seed", [0, 3, (1 << 63) - 1])
def test_moments_are_not_rounded_by_the_mask(seed, keys):
    block = mixer.ChannelMixer(1, 3, 3, 8, 16, seed=seed, device="cpu")
    block.adamw(8)
    block.adamw(8, seed=seed)
    block.adamw(8, seed=7)
    assert keys[0] == keys[1] and keys[2] not in (keys[0], 7)
    assert all(0 <= k < 1 << 64 and k != seed for k in keys)
    for step in (1, 2, 1000):
        # the mask of an element at this step is drawn from the first of these words
        mask, rounding = ao.draws(4096, 0, step, seed), ao.draws(4096, 0, step, keys[0])
        assert int((mask == rounding).sum()) == 0
        # 8192 pairs of 16 bits that agree by chance: an eighth of one is expected
        assert sum(int(np.sum((mask >> s) & 0xFFFF == (rounding >> s) & 0xFFFF)) for s in (np.uint64(0), np.uint64(16))) <= 5


def test_training_draws_from_its_seed(keys, monkeypatch):
    blocks = []

    class Stop(Exception):
        pass

    class Block(mixer.ChannelMixer):
        def __init__(self, *a, **kw):
            super().__init__(*a, device="cpu", **kw)
            blocks.append(self)

        def forward(self, *a):
            raise Stop
    monkeypatch.setattr(mixer, "ChannelMixer", Block)
    monkeypatch.setattr(torch.Tensor, "to", lambda self, *a: self)
    with pytest.raises(Stop):
        mixer.train(steps=1, seed=5, adamw=8)
    student = blocks[-1]
    assert student.seed == 5 and len(keys) == 1 and keys[0] != 5
