"""CPU-only: what the few-row kernel of one matrix reads of the weights, from the
arithmetic that the kernel shares with libep_probe.so."""
import ctypes

import pytest

import matmul_paths as P


def reach(groups, cols, units):
    P.matmul(0, 16, 2)                  # loads the library
    fn = P._lib.ep_probe_matmul_thin_reach
    fn.argtypes, fn.restype = [ctypes.c_int] * 3, ctypes.c_int64
    return fn(groups, cols, units)


@pytest.mark.parametrize("cols", [16, 48, 128, 144, 272, 2064, 4112, 7168, 131056])
@pytest.mark.parametrize("groups", [1, 2])
def test_thin_loads_stay_inside_the_weights(groups, cols):
    """All of them and nothing behind them, also where a block's second group of
    outputs is short or missing."""
    for units in (1, 15, 16, 17, 31, 32, 33, 48, 4090, 7169, 7170, 7184, 7185, 8177, 8191, 8192):
        assert reach(groups, cols, units) == cols * units, units
