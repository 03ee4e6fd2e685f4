"""The tree attention's split of its work, on the GPU: sizes that the model of the scheduler says have tiles cut across two
groups of pairs and pairs in between without a part.  What the kernel hands to the joining kernel is compared with the model's,
and the values with 64 bits."""
import pytest
import torch

import sparse_mla_attention_fwd_gb300 as smla
from test_tree_schedule_cpu import GROUP, schedule, tiles_of
from test_tree_step_gpu import tree_case, tree_check

pytestmark = pytest.mark.gpu

MAX_PAIRS = 80


def expected(q_lens, k_lens, heads, pairs):
    """Each pair's entry for the joining kernel: first row, rows, last pair, pairs without a part; (0, 0, -1, 0) without one."""
    tiles = tiles_of([(n, k, k) for n, k in zip(q_lens, k_lens)], heads)
    per_tile, rows = max(128 // heads, 1), []
    first = [sum(q_lens[:b]) for b in range(len(q_lens))]
    joins = schedule(tiles, pairs)[1]
    for pair in range(pairs):
        if pair not in joins:
            rows.append((0, 0, -1, 0))
            continue
        i, last, none = joins[pair]
        b, k, g = tiles[i][0]
        tokens = min(per_tile, q_lens[b] - k * per_tile)
        rows.append(((first[b] + k * per_tile) * heads + 128 * g, min(128, heads - 128 * g) if heads > 128 else tokens * heads, last, none))
    return rows


@pytest.mark.parametrize("heads,requests", [
    (128, [(30, 55), (30, 731), (9, 278), (5, 2055), (17, 638), (5, 118), (5, 262), (5, 178)]),
    (129, [(2, 750), (1, 3222), (30, 565), (1, 99), (2, 155)]),
    (200, [(5, 1218), (30, 791), (1, 624)]),
    (64, [(9, 830), (30, 202), (5, 351), (9, 2793), (2, 929), (5, 265), (30, 601), (17, 635), (1, 59), (2, 130), (2, 2698), (9, 1821)]),
    (20, [(17, 3555), (17, 140), (1, 353), (17, 349), (5, 207), (2, 239), (17, 610), (9, 46), (30, 136), (1, 40), (2, 50), (5, 651),
          (17, 73), (30, 92), (9, 63), (1, 889), (5, 1522), (5, 1708), (30, 296), (9, 379), (9, 630), (2, 45), (1, 489), (2, 287),
          (1, 111), (30, 211), (17, 172), (17, 223), (17, 193), (30, 3215), (17, 404), (1, 36), (2, 826), (1, 709), (2, 240),
          (30, 96), (1, 120), (1, 153), (2, 179), (2, 691)]),
])
def test_cut_tiles_are_joined_as_the_model_says(heads, requests):
    pairs = min(torch.cuda.get_device_properties(0).multi_processor_count // 2, MAX_PAIRS)
    q_lens, k_lens = [n for n, _ in requests], [k for _, k in requests]
    want = expected(q_lens, k_lens, heads, pairs)
    if pairs == 76:       # a GB300: the sizes were chosen for its number of pairs
        assert any(none for _, _, _, none in want)
        assert any(last // GROUP != pair // GROUP for pair, (_, _, last, _) in enumerate(want) if last >= 0)
    size = smla.load_library().sparse_mla_chunk_workspace_size(sum(q_lens), heads)
    for kind in ("tree", "bits"):
        workspace = torch.full((size,), 0x7f, dtype=torch.uint8, device="cuda")
        tree_check(tree_case(len(requests), q_lens, k_lens, heads, kind=kind), workspace=workspace)
        # the entries lie behind everything else
        joins = workspace[size - 16 * MAX_PAIRS:].view(torch.int32).view(MAX_PAIRS, 4)[:pairs]
        assert [tuple(j) for j in joins.tolist()] == want
