"""The sizes of the GPU tests take the tile shapes that they are meant for: the launch geometry of each against the
shape's waves, LDS and tiles.  A change of the shapes or of their choice that leaves one untested fails here."""
import pytest

from tests.test_gpu_i8_ffn_rings import SIZES, TILES


@pytest.fixture(scope="module")
def loom():
    import int8_dequant_dot_amd as m
    return m


def shapes_of(loom, op, rows, k, tokens):
    """The tiles whose launch this would be."""
    c = loom.launch_config_invoke(loom.launch_config_lookup(op), [rows, k, tokens])
    gated = op != "i8_matmul"
    found = []
    for i, (channels, tile_tokens, waves, split, ring_w, ring_x) in enumerate(TILES):
        groups = -(-rows // (channels // 2 if gated else channels)) * -(-tokens // tile_tokens)
        lds = split * 128 * (ring_w * channels + ring_x * tile_tokens)
        if (c["workgroups"][0], c["workgroup_size"][0], c["workgroup_storage_bytes"]) == (groups, 64 * waves, lds):
            found.append(i)
    return found


@pytest.mark.parametrize("op", list(SIZES))
def test_every_tile_shape_is_tested(loom, op):
    assert sorted(SIZES[op]) == list(range(8 if op.endswith("backward") else 10))
    for tile, sizes in SIZES[op].items():
        channels, tokens, _, split, ring_w, _ = TILES[tile]
        out = channels // 2 if op != "i8_matmul" else channels
        # the first size tells its tile from all others; one token tile can look like another tile's
        assert shapes_of(loom, op, *sizes[0]) == [tile], sizes[0]
        for size in sizes:
            assert tile in shapes_of(loom, op, *size), size
            # rings that turn more than twice, a step that is partly filled, and edges inside the last tiles
            assert size[1] // 128 // split > 2 * ring_w and size[1] % 128 and size[0] % out and size[2] % tokens, size
