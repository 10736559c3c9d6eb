"""Which kernel serves a product in 8-bit integers (libep_probe.so), for the
tests that have to reach each of them."""
import ctypes
import os

from combine_get_dispatch_layout_amd import ep

NONE, FEW, THIN, TILE64X64, TILE64X128, TILE128, TILE256 = range(7)
_lib = None


def matmul(rows, cols, rows_out, act=0, experts=0):
    """experts: 0 for one matrix; rows_out: of the weight matrix."""
    global _lib
    if _lib is None:
        _lib = ctypes.CDLL(os.path.join(os.path.dirname(ep.LIB_PATH), "libep_probe.so"))
        _lib.ep_probe_matmul_path.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 4
    return _lib.ep_probe_matmul_path(act, cols, rows_out // 2 if act else rows_out, experts, rows)


def splits(rows, cols, rows_out, act=0):
    """Blocks that the columns of a product with one matrix are split over, with
    a workspace."""
    matmul(0, 16, 2)                # loads the library
    _lib.ep_probe_matmul_splits.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3
    return _lib.ep_probe_matmul_splits(act, cols, rows_out // 2 if act else rows_out, rows)
