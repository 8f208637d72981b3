"""Which tiles the sizes of linear_tiles.py take: all that are built, so that a change of the choice's model moves the tests'
sizes with it."""
import pytest

from linear_tiles import GRADIENTS, PRODUCTS, SHAPES, TYPES, compiler, plans


@pytest.fixture(scope="module")
def folder(tmp_path_factory):
    if compiler() is None:
        pytest.skip("g++ not available")
    return str(tmp_path_factory.mktemp("plan"))


def test_the_listed_sizes_take_the_listed_tiles(folder):
    got = plans(folder, [("p",) + c[:4] for c in PRODUCTS])
    assert got == [c[4:] for c in PRODUCTS]
    got = plans(folder, [("g",) + c[:4] for c in GRADIENTS])
    assert got == [(c[4], False, 1) for c in GRADIENTS]


def test_the_listed_sizes_reach_past_a_tile_and_a_step():
    for M, K, N, dtype, tile, _, splits in PRODUCTS:
        bm, bn = SHAPES[tile]
        size = {"f32": 4, "f16": 2, "bf16": 2, "int8": 1, "e4m3": 1}[dtype]
        assert M > bm and N > bn and M % bm and N % bn and K * size % 128
        assert K * size > 128 * splits * (4 if splits > 1 else 8)


def test_every_tile_that_is_built_is_listed():
    """By types: nine tiles (fp32 without the last, and 256 x 128 only for both gradients at once), three with loads of 4
    bytes."""
    products, joint = {c[3:6] for c in PRODUCTS}, {c[3:5] for c in GRADIENTS}
    split = {c[3:6] for c in PRODUCTS if c[6] > 1}
    for t in TYPES:
        assert {(t, k, True) for k in (5, 6, 7)} <= products & split
        tiles = set(range(9)) - ({4, 8} if t == "f32" else set())
        assert {(t, k, False) for k in tiles} <= products
        assert {(t, k, False) for k in tiles - ({2} if t == "f32" else set())} <= split
    for t in ("f32", "f16", "bf16"):
        assert {(t, k) for k in range(8 if t == "f32" else 9)} <= joint


def test_fp32_never_takes_the_tile_that_it_has_not(folder):
    sizes = [(what, M, K, N, "f32") for what in "pg" for M in (1, 20, 77, 130, 300, 700, 1500, 4000, 9000, 70000)
             for K in (1, 40, 333, 1110, 2560, 9000) for N in (1, 65, 200, 771, 2560, 10576, 40000)]
    assert all(tile != 8 for tile, _, _ in plans(folder, sizes))
