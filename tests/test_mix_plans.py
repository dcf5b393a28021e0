"""Which kernels the channel-mixing planner may choose, over ranges of sizes
(host only)."""
import ctypes

import pytest

from convolution_nhwc_amd import api


def plan(op, *fields):
    q = api.GatedProblem(*fields, 0)
    buf = ctypes.create_string_buffer(256)
    assert api.lib().cnhwc_gated_plan(ctypes.byref(q), op, buf, 256) == api.OK
    return buf.value.decode()


@pytest.mark.parametrize("dtype", [api.F16, api.BF16])
def test_few_rows_backward_only_where_a_kernel_exists(dtype):
    """More than 16 rows whose x does not stay in registers have no few-row kernel backward; forward they
    have one where the tiles would copy the weights first."""
    for rows in (1, 16, 17, 32, 33, 64, 65):
        for c in (1, 64, 1024, 1025, 2040, 2048, 2049, 2056, 4096, 4097, 4104, 9000):
            bwd = plan(api.OP_DGRAD, rows, c, 40, 0, 0, 0, dtype)
            assert ("gated_rows" in bwd) == (rows <= 16 or (rows <= 64 and c <= 2048)), (rows, c, bwd)
            fwd = plan(api.OP_FWD, rows, c, 40, 0, 0, 0, dtype)
            kept = rows <= 16 or c <= 2048
            assert ("gated_rows" in fwd) == (rows <= 64 and (kept or c % 8 != 0)), (rows, c, fwd)
