"""CPU-only: the workspace sizes that a Weights remembers."""
import ctypes

from combine_get_dispatch_layout_amd import moe
from test_matmul_abi import _FakeWeights, _w


def test_sizes_are_right_and_few():
    w = _FakeWeights(1, 4096, 7168)
    c = _w(rows=4096, cols=7168)
    w._ref, w._workspace = ctypes.byref(c), {}
    first = [moe.ep_matmul_workspace_size(w, n, act) for act in (0, 1) for n in range(1000)]
    assert len(w._workspace) <= 256 and any(first) and not all(first)
    w._workspace.clear()
    for i in (70, 64, 1999, 70, 0, 1064):
        assert moe.ep_matmul_workspace_size(w, i % 1000, i // 1000) == first[i]
