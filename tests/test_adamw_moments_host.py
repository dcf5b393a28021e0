"""How many moments one call reads back.  Nothing here launches a kernel."""
import pytest

from convolution_nhwc_amd import api


def moments(n, m=1 << 40):
    # (addresses far apart, never dereferenced; m may be one that an output covers)
    return api.lib().cnhwc_adamw_moments(n, m, 2 << 40, 3 << 40, 4 << 40, 5 << 40, 6 << 40, None)


@pytest.mark.parametrize("n", [-1, 1 << 35, 1 << 36, 1 << 39, 1 << 40])
def test_more_than_a_launch_has_threads_for_is_refused(n):
    # (an output over an input, so that no size gets past the checks)
    assert moments(n, m=5 << 40) == api.INVALID_ARG
    assert "n must be in [0, 2^35)" in api.last_error()


def test_the_largest_passes_the_check_of_sizes():
    assert moments((1 << 35) - 1, m=5 << 40) == api.INVALID_ARG
    assert "m_values overlaps m" in api.last_error()
