"""Received int8 rows that the kernels of product.hpp serve, one case or more for
each kernel of theirs, with the choice that libep_probe.so tells."""
import ctypes
import os

import matmul_paths as P
import moe_paths
from combine_get_dispatch_layout_amd import ep, moe

# kernel, waves that share a tile's columns; tokens, experts, entries a token, columns,
# weight rows, gate, alignment, capacity, share of masked entries, skew
CASES = [
    (moe_paths.SMALL, 4, 20, 8, 2, 4112, 66, 0, 1, 0, 0.1, 1.0),
    (moe_paths.ONE_TILE, 1, 100, 64, 3, 272, 9000, 0, 1, 0, 0.1, 1.0),
    (moe_paths.ONE_TILE, 8, 32, 8, 2, 9216, 128, 0, 1, 0, 0.0, 0.5),
    (moe_paths.ONE_TILE, 8, 32, 8, 2, 9232, 258, 1, 16, 0, 0.1, 1.0),
    (moe_paths.MEMORY, 8, 32, 8, 2, 16400, 130, 0, 1, 0, 0.1, 1.0),
    (moe_paths.MEMORY, 8, 32, 8, 2, 16400, 130, 1, 1, 12, 0.0, 1.0),
    (moe_paths.MEMORY, 8, 8, 8, 1, 98192, 34, 0, 1, 0, 0.0, 0.5),
    (moe_paths.MEMORY, 1, 128, 32, 2, 16400, 4098, 0, 1, 0, 0.1, 1.0),
    (moe_paths.MEMORY, 1, 128, 32, 2, 16384, 8200, 1, 1, 0, 0.1, 0.5),
]


def kernel(N, E, K, C, M, act):
    """(kernel, waves that share a tile's columns), None for another family's."""
    if P.matmul(N * K, C, M, act, E) != P.FEW:
        return None
    lib = ctypes.CDLL(os.path.join(os.path.dirname(ep.LIB_PATH), "libep_probe.so"))
    sizes = [ctypes.c_int64(v) for v in (C, M // 2 if act else M, E, N * K)]
    args = [moe.EP_WEIGHT_INT8, 0, act, 1, *sizes]
    return lib.ep_probe_product_path(*args, None), lib.ep_probe_product_waves(*args)
