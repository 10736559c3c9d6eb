"""CPU-only checks of the choice of kernels for products in 8-bit integers: the
limits the kernels have, and that the choice is total."""
import random

import pytest

import matmul_paths as P

# (path, stages): loads run stages - 1 steps of 128 columns ahead, and a tile's
# scales are loaded behind the last columns of the tile before, stages steps before
# its first.  They overwrite those of the tile `buffers` before, whose last step is
# (buffers - 1) * steps before that first one: not sooner than its end with
STAGES = {P.TILE64X64: 4, P.TILE64X128: 3, P.TILE128: 2, P.TILE256: 2}
BUFFERS = {P.TILE64X64: 2, P.TILE64X128: 2, P.TILE128: 3, P.TILE256: 3}


def test_nothing_and_little():
    assert P.matmul(0, 7168, 4096) == P.NONE and P.matmul(0, 7168, 4096, experts=8) == P.NONE
    for rows in (1, 16, 32):
        assert P.matmul(rows, 7168, 4096) == P.THIN
    assert P.matmul(33, 7168, 4096) == P.TILE64X64
    assert P.matmul(1, 7168, 28672) == P.TILE64X64
    assert P.matmul(1024, 7168, 4096, act=1, experts=256) == P.FEW
    assert P.matmul(65536, 7168, 4096, act=1, experts=256) == P.TILE256


def test_short_rows():
    """With one or two steps only tiles of two stages and three buffers of scales
    are right, with three also those of three stages."""
    rng = random.Random(3)
    for _ in range(3000):
        cols = 16 * rng.randint(1, 48)
        p = P.matmul(rng.randint(1, 20000), cols, 2 * rng.randint(1, 5000), rng.randint(0, 1), rng.choice([0, 1, 4, 64, 1024]))
        assert p != P.NONE and (p not in STAGES or (BUFFERS[p] - 1) * ((cols + 127) // 128) >= STAGES[p]), (cols, p)


def test_thin_is_for_one_matrix():
    rng = random.Random(4)
    for _ in range(2000):
        rows, out = rng.randint(1, 100), 2 * rng.randint(1, 20000)
        assert P.matmul(rows, 7168, out, rng.randint(0, 1), rng.randint(1, 64)) != P.THIN
        if P.matmul(rows, 2048, out) == P.THIN:
            assert rows <= 32 and (rows + 15) // 16 * ((out + 15) // 16) <= 640


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("experts", [0, 1, 8, 64, 256, 1024])
def test_every_size_has_a_kernel(experts, act):
    for rows in (1, 31, 32, 33, 1000, 1 << 20, (1 << 31) - 1):
        for cols in (16, 256, 272, 400, 528, 2048, 131056):
            for out in (2, 34, 4096, 1 << 20, 1 << 24):
                if rows * out < 1 << 35:
                    assert P.NONE < P.matmul(rows, cols, out, act, experts) <= P.TILE256
