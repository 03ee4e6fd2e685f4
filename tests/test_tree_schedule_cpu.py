"""The tree attention's split of its work, in a model of the scheduler of chunk_fwd.cu: over random requests every block of
keys of every tile is computed once, a tile's parts lie in slots of their own, and the joining kernel finds exactly the parts of
each cut tile, in order.  The constants are read from the source."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "sparse_mla_attention_fwd_gb300", "csrc", "chunk_fwd.cu")).read()


def constant(name):
    return int(re.search(r"constexpr int %s = (\d+);" % name, SOURCE).group(1))


COST, SHORTEST, KEYS, GROUP = (constant(n) for n in ("kTileCost", "kMinRange", "kKeys", "kTreeGroup"))


def up(a, b):
    return -(-a // b)


def tiles_of(requests, heads):
    """Tiles in the order of the axis: (request, token tile, group of heads), keys of the axis, readable keys."""
    per_tile, groups = (128 // heads, 1) if heads <= 128 else (1, up(heads, 128))
    return [((b, k, g), n_k, keys) for b, (n_q, n_k, keys) in enumerate(requests) for k in range(up(n_q, per_tile)) for g in range(groups)]


def schedule(tiles, pairs):
    """Each pair's (tile, first block, last block + 1, slot or -1), and its entry for the joining kernel."""
    starts, s = [], 0
    for _, n_k, _ in tiles:
        starts.append(s)
        s += n_k + COST
    span = max(up(s, pairs), SHORTEST)
    work, joins = {}, {}
    for pair in range(pairs):
        first = pair // GROUP * GROUP
        members = min(GROUP, pairs - first)
        v0, v1 = first * span, (first + members) * span
        load = [0 if g < members else span for g in range(GROUP)]
        a, e, pieces, done, join = v0, v1, False, [], None
        at = [i for i, begin in enumerate(starts) if begin <= v0]
        # the walk starts with all groups of heads of the token tile in which the range starts
        i = next(j for j, t in enumerate(tiles) if t[0][:2] == tiles[at[-1]][0][:2]) if v0 < s else len(tiles)
        while i < len(tiles):
            s0, (_, n_k, keys) = starts[i], tiles[i]
            size, blocks = n_k + COST, max(up(keys, KEYS), 1)
            if s0 >= e:
                break
            if not pieces:
                if s0 + size <= v0:
                    i += 1
                    continue
                begin = max(s0, v0)
                least = min(load)
                to = load.index(least)
                if s0 + size <= v1 and least + s0 + size - begin <= span:
                    load[to] += s0 + size - begin
                    if first + to != pair:
                        i += 1
                        continue
                else:
                    pieces, e = True, begin
                    for g in range(GROUP):
                        if first + g <= pair:
                            a, e = e, e + span - load[g]
                    if s0 >= e:
                        break
            j0 = 0 if s0 >= a else up(a - s0, KEYS)
            j1 = min(blocks, up(e - s0, KEYS))
            if j0 < j1:
                slot = -1
                if j0 > 0:
                    slot = 2 * pair
                elif j1 < blocks:
                    slot = 2 * pair + 1
                    assert join is None
                    join = i, s0, s0 + KEYS * (blocks - 1)
                done.append((i, j0, j1, slot))
            i += 1
        if join:
            i, s0, end_of = join
            z, none = end_of // span, 0
            if end_of < e:
                z = pair
            begin = e
            for g in range(1, GROUP):
                if first + g > pair and begin <= end_of:
                    end = begin + span - load[g]
                    if end_of < v1:
                        z = first + g
                    if up(begin - s0, KEYS) == up(end - s0, KEYS):
                        none |= 1 << (first + g - pair)
                    begin = end
            joins[pair] = i, z, none
        work[pair] = done
    return work, joins


@pytest.mark.parametrize("heads", [1, 20, 128, 129, 320, 1024])
@pytest.mark.parametrize("pairs", [76, 74, 9, 4, 3, 1])
def test_every_block_once_and_every_part_joined(heads, pairs):
    rng = random.Random(heads * 100 + pairs)
    for _ in range(60):
        requests = []
        for _ in range(rng.choice([1, 2, 5, 40])):
            n_k = int(10 ** rng.uniform(0, 4.3)) if rng.random() < 0.5 else rng.randint(0, 3000)
            requests.append((rng.choice([0, 1, 2, 9, 40]), n_k, n_k if rng.random() < 0.8 else rng.randint(0, n_k)))
        tiles = tiles_of(requests, heads)
        if not tiles:
            continue
        work, joins = schedule(tiles, pairs)
        seen, slots = {}, {}
        for done in work.values():
            for i, j0, j1, slot in done:
                for j in range(j0, j1):
                    assert (i, j) not in seen
                    seen[i, j] = slot
                if slot >= 0:
                    assert slot not in slots and slot < 2 * pairs
                    slots[slot] = i, j0, j1
        for i, (_, _, keys) in enumerate(tiles):
            slots_of = {seen[i, j] for j in range(max(up(keys, KEYS), 1))}      # KeyError: a block that nobody computes
            assert slots_of == {-1} or -1 not in slots_of
        joined = set()
        for w, (i, z, none) in joins.items():
            assert i not in joined and z < pairs
            joined.add(i)
            blocks = []
            for pair in range(w, z + 1):
                if pair - w < 32 and none >> (pair - w) & 1:
                    continue
                tile, j0, j1 = slots[2 * w + 1 if pair == w else 2 * pair]
                assert tile == i
                blocks += range(j0, j1)
            assert blocks == list(range(max(up(tiles[i][2], KEYS), 1)))
        assert joined == {i for (i, _), slot in seen.items() if slot >= 0}
