"""Every kernel of the 4-bit products is run by a size of test_gpu_experts_tiles.py: by the launch table, no GPU needed."""
import pytest

from tests.test_gpu_experts_tiles import DENSE, EXPERTS, GATED, K, ROUTED

# tokens and channels of a tile, waves, waves that split k, 128s of k in a step; gated waves have a block of either weight,
# so the last two shapes have half of the channels or half of the waves
TILES = {"plain": [(128, 256, 8, 1, 2), (64, 128, 4, 1, 2), (32, 128, 4, 1, 2), (32, 32, 8, 8, 1)],
         "gated": [(128, 128, 8, 1, 2), (64, 64, 4, 1, 2), (32, 64, 2, 1, 2), (32, 32, 8, 8, 1)]}


def groups_in_128(group):
    return max(1, 128 // group)


def kernel(loom, form, rows, tokens, group):
    """What the launch table chooses: ("stream", token slots) or ("tile", shape)."""
    name = {"dense": "i4_matmul", "routed": "i4_expert_matmul", "gated": "i4_expert_gated_projection"}[form]
    work = [rows, K, tokens, group] + ([] if form == "dense" else [EXPERTS])
    c = loom.launch_config_invoke(loom.launch_config_lookup(name), work)
    waves, lds, grid = c["workgroup_size"][0] // 64, c["workgroup_storage_bytes"], c["workgroups"][0]
    if lds <= 4096:
        return "stream", lds // 512
    found = []
    for i, (t, ch, w, split, half) in enumerate(TILES["gated" if form == "gated" else "plain"]):
        both = 2 * ch if form == "gated" else ch
        size = 2 * split * half * (t * 128 + both * (64 + 4 * groups_in_128(group)))
        tiles = -(-tokens // t) if form == "dense" else tokens // t + min(tokens, EXPERTS)
        if (waves, lds, grid) == (w, size, tiles * -(-rows // ch)):
            found.append(i)
    assert len(found) == 1, (form, rows, tokens, group, c)
    return "tile", found[0]


@pytest.mark.parametrize("form,sizes", [("dense", DENSE), ("routed", ROUTED), ("gated", GATED)])
def test_sizes_reach_every_kernel(form, sizes):
    import int8_dequant_dot_amd as loom
    seen = {(*kernel(loom, form, rows, tokens, group), groups_in_128(group)) for rows, tokens, group in sizes}
    want = {("tile", shape, subs) for shape in range(4) for subs in (1, 2, 4)}
    # slots of 4 hold a token in groups of 128, two of 64, four of 32; the routed stream has 4
    want |= {("stream", 4, 1), ("stream", 4, 2)} | ({("stream", 4, 4)} if form != "dense" else set())
    want |= {("stream", 8, subs) for subs in (1, 2, 4)} if form == "dense" else set()
    assert seen == want
