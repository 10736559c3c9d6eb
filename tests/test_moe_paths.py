"""CPU tests of the choice among the product kernels (libep_probe.so)."""
import pytest

import moe_paths as P

KINDS = [("bf16", 0), ("mxfp4", 32), ("int4", 32), ("int4", 64), ("int4", 128)]


@pytest.mark.parametrize("fmt,group", KINDS)
def test_paths_of_ordinary_sizes(fmt, group):
    assert P.product(fmt, group, 2048, 2048, 1, 0)[0] == P.NONE
    # 64 KB, less 16 KB for the sums of four waves, hold 11 rows of 4112 bytes
    assert P.product(fmt, group, 2048, 2048, 1, 1) == (P.SMALL, 11)
    # a decode batch: 128 tokens, 256 experts, top-8
    assert P.product(fmt, group, 7168, 4096, 256, 1024, act=1)[0] == P.ONE_TILE
    assert P.product(fmt, group, 2048, 7168, 256, 1024, terms=2)[0] == P.ONE_TILE
    # x past LDS; more than 16 rows an expert
    assert P.product(fmt, group, 7168, 14336, 1, 13) == (P.MEMORY, 16)
    # 448 tiles leave four waves a tile, whose sums take 64 KB of the 128
    assert P.product(fmt, group, 1024, 14336, 1, 17) == (P.TWO_TILES, 31)
    assert P.product(fmt, group, 1024, 65536, 1, 17) == (P.TWO_TILES, 32)
    assert P.layer(fmt, group, 1, 8, 128, 2048, 768) == (P.SMALL, 0)
    assert P.layer(fmt, group, 128, 8, 256, 7168, 2048) == (P.ONE_TILE, P.ONE_TILE)


@pytest.mark.parametrize("fmt,group", KINDS)
def test_tiles_decide_between_small_and_big_blocks(fmt, group):
    """512 tiles of 32 outputs (16 with a gate)."""
    for act in (0, 1):
        assert P.product(fmt, group, 256, 32 * 31, 16, 16, act)[0] == P.SMALL
        assert P.product(fmt, group, 256, 32 * 31 + 2, 16, 16, act)[0] == P.ONE_TILE
    # or rows that the small blocks' LDS does not hold
    assert P.product(fmt, group, 32768, 32, 1, 1)[0] == P.ONE_TILE
    assert P.product(fmt, group, 65536, 32, 1, 1)[0] == P.MEMORY


@pytest.mark.parametrize("fmt,group", KINDS)
def test_rows_at_once_never_fall_below_the_mean(fmt, group):
    for cols in (128, 1024, 2048, 4096, 7168, 14336):
        for rows in (1, 2, 5, 16, 17, 64, 700):
            path, at_once = P.product(fmt, group, cols, 4096, 1, rows)
            assert at_once >= min(rows, 16)
            assert (path == P.TWO_TILES) <= (rows > 16)
            assert at_once <= (32 if path == P.TWO_TILES else 16)


def test_limits_of_a_handful():
    """64 KB hold the pairs' two terms in rows of whole lines and 16 bytes."""
    for fmt, group, line, most in (("bf16", 0, 64, 32), ("mxfp4", 32, 256, 32), ("int4", 128, 256, 32),
                                   ("int4", 64, 256, 8), ("int4", 32, 256, 8)):
        for I in (128, 256, 512, 1024, 2048):
            for N in range(1, 18):
                for K in range(1, 17):
                    row = 2 * (-(-I // line) * line) + 16
                    fits = N <= 16 and N * K <= most and 2 * N * K * row <= 65536
                    assert (P.layer(fmt, group, N, K, 64, 256, I)[1] == 0) == fits
