"""The chunk attention's named barriers when a wait gives up, checked on the CPU.

Waits on mbarriers give up after a time limit; named barriers (bar.sync) have none, so the order in which
the softmax and epilogue warps meet at them must end whatever waits gave up, and when.  This test explores
every interleaving of that protocol in a small model:

- two pairs of softmax warps, which look at the abort flag once a block and hand finished tiles to
- the epilogue, which sleeps on one named barrier per tile (256 threads: 64 + 64 + 128) until the end;
- an abort flag that may be set at any moment, after which every mbarrier wait returns at once.

The number of tile barriers and whether the pairs agree on leaving are read from the kernel's source."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "sparse_mla_attention_fwd_gb300", "csrc", "chunk_fwd.cu")
END = -1


def protocol():
    text = open(SOURCE).read()
    m = re.search(r"constexpr\s+uint32_t\s+kTileBars\s*=\s*(\d+)\s*;", text)
    # in the tile's hand-over, and on every other way out of the loop
    agree = len(re.findall(r"named_bar_or\(kAgreeBar, 128,", text)) == 2
    return (int(m.group(1)) if m else 2), agree


# A pair's state: (step, block, tiles handed over, result of the agreement).  Steps in program order:
CHECK, WAIT_PV, AGREE, AGREEING, ARRIVE, LEAVE, LEAVING, LAST_WAIT, LAST_ARRIVE, GONE = range(10)


def explore(tiles, bars, agree):
    """All reachable states for tiles of the given numbers of blocks; returns a stuck one, or None."""
    tile_of = [t for t, n in enumerate(tiles) for _ in range(n)]
    last = [i + 1 == len(tile_of) or tile_of[i + 1] != t for i, t in enumerate(tile_of)]
    n = len(tile_of)
    # abort, pairs, P written by each pair (blocks), tile barriers' arrivals, contribution to the agreement,
    # epilogue (step, tile, tiles whose O it has read), the tiles' descriptors
    start = (False, ((CHECK, 0, 0), (CHECK, 0, 0)), (0, 0), (0,) * bars, (), ("sync", 0, 0), (None,) * bars)
    todo, seen = [start], {start}
    while todo:
        s = todo.pop()
        abort, pairs, written, arrived, vote, (e_step, e_tile, e_read), slots = s

        def pv_done(b):   # both pairs' P, and the tile before read out of O
            return b < 0 or abort or (min(written) > b and e_read >= tile_of[b])

        def arrive(arrived, bar, threads):
            total = arrived[bar] + threads
            return arrived[:bar] + (0 if total == 256 else total,) + arrived[bar + 1:], total == 256

        nxt = []
        if not abort:
            nxt.append((True, *s[1:]))
        for i, (step, b, tile) in enumerate(pairs):
            def moved(new, written=written, arrived=arrived, vote=vote, e=(e_step, e_tile, e_read), slots=slots, other=None):
                p = list(pairs)
                p[i] = new
                if other is not None:
                    p[1 - i] = other
                return (abort, tuple(p), written, arrived, vote, e, slots)

            if step == CHECK:
                if b == n or abort:
                    nxt.append(moved((LEAVE if agree else LAST_WAIT, b, tile)))
                else:
                    nxt.append(moved((WAIT_PV, b, tile)))
            elif step == WAIT_PV and pv_done(b - 1):
                w = tuple(b + 1 if j == i else x for j, x in enumerate(written))
                after = (CHECK, b + 1, tile) if not last[b] else (AGREE if agree else ARRIVE, b, tile)
                nxt.append(moved(after, written=w))
            elif step in (AGREE, LEAVE):
                out = abort or step == LEAVE
                if not vote:
                    nxt.append(moved((AGREEING if step == AGREE else LEAVING, b, tile), vote=(out,)))
                else:           # the other pair has been waiting: both go on with the same answer
                    out = out or vote[0]
                    o_step, o_b, o_tile = pairs[1 - i]
                    other = (LAST_WAIT if o_step == LEAVING or out else ARRIVE, o_b, o_tile)
                    nxt.append(moved((LAST_WAIT if step == LEAVE or out else ARRIVE, b, tile), vote=(), other=other))
            elif step in (ARRIVE, LAST_ARRIVE):
                bar = tile % bars
                sl = slots[:bar] + (tile if step == ARRIVE else END,) + slots[bar + 1:] if i == 0 else slots
                a, full = arrive(arrived, bar, 64)
                e = ("awake", e_tile, e_read) if full and e_step == "waiting" and e_tile % bars == bar else (e_step, e_tile, e_read)
                nxt.append(moved((CHECK, b + 1, tile + 1) if step == ARRIVE else (GONE, b, tile), arrived=a, e=e, slots=sl))
            elif step == LAST_WAIT and pv_done(b - 1):
                nxt.append(moved((LAST_ARRIVE, b, tile)))
        rest = (abort, pairs, written)
        if e_step == "sync":
            a, full = arrive(arrived, e_tile % bars, 128)
            nxt.append((*rest, a, vote, ("awake" if full else "waiting", e_tile, e_read), slots))
        elif e_step == "awake":
            here = slots[e_tile % bars]
            nxt.append((*rest, arrived, vote, ("gone" if here == END else "read", e_tile, e_read), slots))
        elif e_step == "read" and (abort or pv_done(max(i for i, t in enumerate(tile_of) if t == e_tile))):
            nxt.append((*rest, arrived, vote, ("sync", e_tile + 1, e_tile + 1), slots))
        done = e_step == "gone" and all(p[0] == GONE for p in pairs)
        if not done and (not nxt or (len(nxt) == 1 and not abort and nxt[0][1:] == s[1:])):
            return s
        for x in nxt:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return None


TILES = [(), (1,), (3,), (1, 1), (2, 1), (1, 1, 1), (1, 2, 1), (1, 1, 1, 1, 1), (2, 1, 1, 3)]


@pytest.mark.parametrize("tiles", TILES)
def test_every_warp_leaves_whenever_a_wait_gives_up(tiles):
    bars, agree = protocol()
    assert explore(tiles, bars, agree) is None


def test_the_model_finds_protocols_that_sleep():
    # each pair leaving by itself; agreement, but the end's barrier still taken by the tile before the last
    assert any(explore(t, 2, False) for t in TILES)
    assert any(explore(t, 3, False) for t in TILES)
    assert any(explore(t, 2, True) for t in TILES)


def test_the_tiles_descriptors_have_a_slot_per_barrier():
    text = open(SOURCE).read()
    assert re.search(r"\}\s*done\[kTileBars\];", text)
