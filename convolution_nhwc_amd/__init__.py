"""MI355X (gfx950) NHWC convolution: forward, backward-data and weight gradient
over fp16/bf16, and the channel-mixing operators of a channels-last block (layer
norm, gated feed-forward, dropout; ``mixer`` is such a block).

The compute runs in the HIP library ``libcnhwc.so`` behind a C ABI
(``include/cnhwc.h``); ``convolution_nhwc_amd.api`` is its thin ctypes binding.
Importing this package loads nothing; the binding is loaded on first use and
raises if the library has not been built.
"""
import importlib

__all__ = ["api", "mixer", "synth"]


def __getattr__(name):
    if name in __all__:
        return importlib.import_module("." + name, __name__)
    raise AttributeError(name)
