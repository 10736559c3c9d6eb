"""GPU tests of few int8 rows of many experts, in each kernel that serves them
(asserted), against sums in 64 bits: without an activation bit for bit."""
import pytest

import matmul_few as F
import matmul_paths as P
import test_gpu_matmul_paths as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", F.CASES)
def test_received_rows(case):
    kernel, waves, N, E, K, C, M, act, align, cap, mask, skew = case
    assert F.kernel(N, E, K, C, M, act) == (kernel, waves)
    T.test_received_rows(P.FEW, N, E, K, C, M, act, align, cap, mask, skew)
