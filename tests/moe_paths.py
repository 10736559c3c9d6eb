"""Which kernel serves an expert product (libep_probe.so), for the tests that
have to reach each of them."""
import ctypes
import os

from combine_get_dispatch_layout_amd import ep

NONE, SMALL, ONE_TILE, MEMORY, TWO_TILES = range(5)
FMT = dict(bf16=0, mxfp4=1, int4=2)
_lib = None


def _probe():
    global _lib
    if _lib is None:
        _lib = ctypes.CDLL(os.path.join(os.path.dirname(ep.LIB_PATH), "libep_probe.so"))
        I, I64 = ctypes.c_int, ctypes.c_int64
        _lib.ep_probe_product_path.argtypes = [I, I, I, I, I64, I64, I64, I64, ctypes.POINTER(I64)]
        _lib.ep_probe_layer_in_two.argtypes = [I, I, I64, I64, I64]
    return _lib


def product(fmt, group, cols, rows_out, experts, rows, act=0, terms=1):
    """(path, rows multiplied at once); rows_out: of the weight matrix."""
    at_once = ctypes.c_int64()
    path = _probe().ep_probe_product_path(FMT[fmt], group, act, terms, cols, rows_out // 2 if act else rows_out,
                                          experts, rows, ctypes.byref(at_once))
    return path, at_once.value


def layer(fmt, group, tokens, topk, experts, hidden, inter):
    """Paths of the up and the down projection; the latter 0 where it adds up a
    handful of tokens' experts itself."""
    up = product(fmt, group, hidden, 2 * inter, experts, tokens * topk, act=1)[0]
    if _probe().ep_probe_layer_in_two(FMT[fmt], group, tokens, topk, inter):
        return up, 0
    return up, product(fmt, group, inter, hidden, experts, tokens * topk, terms=2)[0]
