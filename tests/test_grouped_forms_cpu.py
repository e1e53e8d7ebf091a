"""The forms that the exact grouped products of the GPU tests take beside those of tests/moe_shapes.py: the selection
(csrc/mx_tiles.h) asked for each of their shapes."""
import pytest

from tests.test_moe_cpu import form_of, tiles  # noqa: F401


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("M,E,N,K,form", [
    (4096, 2, 8196, 1184, "256"), (4096, 7, 4100, 1184, "256"), (2500, 3, 8192, 1024, "256"),           # shares
    (500, 3, 333, 352, "few 16 x 2"), (61, 8, 4100, 2208, "32, 3 slots"), (900, 5, 1000, 416, "64"),     # offsets that
    (2000, 6, 2054, 800, "128"), (3000, 3, 8209, 800, "256"), (4096, 7, 8196, 1184, "256"),              # descend
    (100, 5, 131072, 16384, "128"), (1300, 5, 131072, 16384, "256"),                                     # past 4 GiB
    (1_100_000, 3, 17, 32, "few 16 x 2"), (2300, 3, 1_000_003, 32, "few 16 x 2"),                        # launches
])
def test_shape_takes_the_form_it_is_there_for(tiles, M, E, N, K, fmt, form):  # noqa: F811
    assert form_of(tiles, M, E, N, K, fmt) == form


def test_many_groups_take_every_tile(tiles):  # noqa: F811
    """The shapes of more groups than a wave has lanes."""
    got = {form_of(tiles, M, E, N, K, fmt).split(",")[0] for fmt in ("fp8", "fp4") for M, E, N, K in
           ((5000, 70, 1030, 544), (9000, 1024, 1030, 544), (20000, 130, 520, 544), (30000, 70, 1030, 512),
            (60000, 200, 1030, 544))}
    assert got == {"32", "64", "128", "256"}


def test_offsets_that_descend_fit(tiles):  # noqa: F811
    """The offsets that descend in the exact test have no more tiles than a launch has places for, whatever the tile."""
    for M, E in ((500, 3), (61, 8), (900, 5), (2000, 6), (3000, 3), (4096, 7)):
        h = M // 2
        for cuts in ([0, 40, 20] + [20] * E, [M] + [0] * E, [0, M, 0] + [5] * E, [h, M, 0, h] + [h] * E):
            for tile in (16, 32, 64, 128, 256):
                total = sum(-(-max(0, min(M, cuts[e + 1]) - cuts[e]) // tile) for e in range(E))
                assert total <= tiles.most(M, E, tile)
