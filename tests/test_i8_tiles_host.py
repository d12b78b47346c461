"""Every tile of the 8-bit products is taken by some shape that a GPU test runs (no GPU here)."""
import i8_tiles
import test_gpu_i8
import test_gpu_i8_tiles


def test_the_shapes_of_each_dense_tile_take_it():
    names = [t[0] for t in i8_tiles.tiles()]
    assert list(test_gpu_i8_tiles.DENSE) == names
    for tile, rows, N, _ in test_gpu_i8_tiles.SHAPES:
        assert i8_tiles.tile_of(rows, N) == tile, (rows, N)
        assert rows > i8_tiles.FEW_ROWS      # (i8_linear runs the product too)


def test_every_routed_tile_is_taken():
    """mpad as csr() of the routed tests makes it, both forms of the projection."""
    marks = {m.args[0]: m.args[1] for m in test_gpu_i8.test_moe_gemm.pytestmark
             if m.name == "parametrize"}
    taken = set()
    for name in marks["name"]:
        counts, tile_m = test_gpu_i8.ROUTED[name]
        if not any(counts):
            continue
        mpad = sum(c + -c % tile_m for c in counts) + 21
        taken |= {i8_tiles.tile_of(mpad, 2 * F, len(counts), True) for F, _ in marks["F,D"]}
    assert taken == {t[0] for t in i8_tiles.tiles()} - {"I8Big"}
