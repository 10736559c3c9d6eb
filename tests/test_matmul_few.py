"""CPU-only: which of product.hpp's kernels serves few int8 rows of many experts."""
import random

import pytest

import matmul_few as F
import moe_paths


@pytest.mark.parametrize("case", F.CASES)
def test_cases_reach_their_kernels(case):
    kernel, waves, N, E, K, C, M, act = case[:8]
    assert F.kernel(N, E, K, C, M, act) == (kernel, waves)


def test_never_two_tiles():
    """Which has no kernel for int8 rows."""
    rng = random.Random(6)
    for _ in range(2000):
        k = F.kernel(rng.randint(1, 3000), rng.choice([1, 2, 8, 64, 256, 1024]), rng.randint(1, 8),
                     16 * rng.randint(1, 8191), 2 * rng.randint(1, 10000), rng.randint(0, 1))
        assert k is None or moe_paths.SMALL <= k[0] <= moe_paths.MEMORY
