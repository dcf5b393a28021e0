"""Every group norm kernel of the library is one that some size takes, and every size's is
there.  The plan is asked on the host; no kernel is launched."""
import ctypes
import re
import shutil
import subprocess

import pytest

from convolution_nhwc_amd import api

PLAIN, CUT = {1, 2, 4, 8, 12, 16, 20, 32}, {4, 12}     # vectors a thread


class Shape(ctypes.Structure):
    _fields_ = [("nv", ctypes.c_int), ("whole", ctypes.c_int), ("span", ctypes.c_int), ("spans", ctypes.c_int),
                ("per", ctypes.c_int), ("pieces", ctypes.c_int), ("vecs", ctypes.c_int), ("ty", ctypes.c_int),
                ("rest", ctypes.c_int * 64)]     # (more than the library's has)


def shape(dtype, n, pixels, c, groups, bwd):
    f = api.lib()._ZN5cnhwc8gn_shapeEillllb
    f.restype = Shape
    f.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 4 + [ctypes.c_bool]
    return f(dtype, n, pixels, c, groups, bwd)


def kernels(dtype, n, pixels, c, groups, bwd):
    """The kernels that launch_groupnorm_fwd and _bwd run, as they are named."""
    t = {api.F32: "F32", api.F16: "F16", api.BF16: "BF16"}[dtype]
    v, s = 4 if dtype == api.F32 else 8, shape(dtype, n, pixels, c, groups, bwd)
    whole = "true" if s.whole else "false"
    if s.nv == 0:
        return {"gn_%s_kernel<%s, %s>" % (k, t, whole) for k in (("sums", "dx") if bwd else ("stats", "apply"))}
    if c // groups >= v:
        assert s.whole, (dtype, n, pixels, c, groups, bwd)    # what the launchers take for granted
    assert s.nv in (PLAIN if s.whole and (bwd or c // groups >= v) else CUT)
    if bwd:
        return {"gn_bwd_kernel<%s, %d, %s>" % (t, s.nv, whole)}
    return {"gn_fwd_kernel<%s, %d, %d, %s>" % (t, s.nv, v if c // groups < v else 2, whole)}


def test_every_kernel_is_reached():
    nm = shutil.which("nm") or pytest.skip("needs nm")
    r = subprocess.run([nm, "-C", api.LIB_PATH], capture_output=True, text=True)
    built = {re.sub(r"cnhwc::", "", name) for name in re.findall(r"__device_stub__(gn_\w+<[^>]*>)\(", r.stdout)}
    if not built:
        pytest.skip("the library's local names were taken out")
    reached = set()
    for dtype in (api.F32, api.F16, api.BF16):
        for bwd in (False, True):
            for each in (1, 2, 3, 5, 6, 7, 8, 9, 12, 16, 37, 96):
                for groups in (1, 2, 3, 4, 8, 11, 32, 64):
                    for pixels in (1, 3, 9, 49, 100, 196, 400, 784, 1500, 3136, 3419, 3583, 5000, 12544):
                        for n in (1, 8, 64, 250, 257, 1000):
                            reached |= kernels(dtype, n, pixels, each * groups, groups, bwd)
    assert reached == built, (sorted(reached - built), sorted(built - reached))
