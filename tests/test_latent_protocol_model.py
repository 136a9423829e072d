"""A model check, on the CPU, of how the two score warps of the latent-attention kernel meet an item's queries.

The softmax threads load item i's queries (barrier `queries`, phase i) and the score warps, which take alternate
tiles, wait for them by parity.  The threads load item i + 1's when every score of item i is formed. With one tile to an
item only one of the two warps has formed it; the other may not have looked at phase i yet, and if phase i + 1
completes before it does, the parity it waits for is that of a phase to come: it stands still, and with it
the tile that it owns.  The safeguard: both warps arrive on a barrier (`seen`) when they have found an
item's queries, and the threads wait for that before they load the next item's.

Barriers and waits are those of an mbarrier with parity waits (test_protocol_model).  A run ends with every
tile scored from its own item's queries, or with the first violation.
"""
import numpy as np

from test_protocol_model import Barrier


def play(rng, tiles, handshake, slow):
    """One random interleaving over items of these numbers of tiles; what went wrong, or None."""
    first = np.concatenate([[0], np.cumsum(tiles)])
    queries, seen = Barrier(), Barrier(2)
    scores, free = [Barrier(), Barrier()], [Barrier(), Barrier()]
    loaded = -1                      # the item whose queries are in place
    # a score warp: its item, whether it has found the item's queries, its next tile within the item
    item, found, tile = [0, 0], [False, False], [0, 0]
    soft_item, soft_tile, load = 0, 0, 0
    while True:
        acts = []
        # the softmax threads: load item `load` (the first at once, others at the previous one's end), or take a tile
        if load == soft_item and load < len(tiles):
            if load == 0 or not handshake or seen.passes((load - 1) & 1):
                acts.append("load")
        elif soft_item < len(tiles):
            c = int(first[soft_item]) + soft_tile
            if scores[c & 1].passes((c >> 1) & 1):
                acts.append("take")
        for w in (0, 1):
            if item[w] == len(tiles):
                continue
            weight = 1 if w == slow else 6
            if not found[w]:
                if queries.passes(item[w] & 1):
                    acts += [("find", w)] * weight
                continue
            c = int(first[item[w]]) + tile[w]
            if (c & 1) != w or c < 2 or free[w].passes(((c >> 1) - 1) & 1):
                acts += [("tile", w)] * weight
        if not acts:
            done = soft_item == len(tiles) and item == [len(tiles)] * 2
            return None if done else "stands still"
        a = acts[rng.integers(len(acts))]
        if a == "load":
            loaded, load = load, load + 1
            queries.arrive()
        elif a == "take":
            c = int(first[soft_item]) + soft_tile
            free[c & 1].arrive()
            soft_tile += 1
            if soft_tile == tiles[soft_item]:
                soft_item, soft_tile = soft_item + 1, 0
        elif a[0] == "find":
            w = a[1]
            if loaded != item[w]:
                return "found another item's queries"
            found[w] = True
            if handshake:
                seen.arrive()
        else:
            w = a[1]
            c = int(first[item[w]]) + tile[w]
            if (c & 1) == w:
                if loaded != item[w]:
                    return "scored with another item's queries"
                scores[w].arrive()
            tile[w] += 1
            if tile[w] == tiles[item[w]]:
                item[w], found[w], tile[w] = item[w] + 1, False, 0


def outcomes(handshake, most, trials=400, seed=1):
    rng = np.random.default_rng(seed)
    return {play(rng, rng.integers(1, most + 1, size=int(rng.integers(2, 30))), handshake, t % 2) for t in range(trials)}


def test_every_item_is_scored_with_the_handshake():
    for most in (1, 2, 5):
        assert outcomes(True, most) == {None}


def test_without_it_the_model_stands_still():
    assert "stands still" in outcomes(False, 1)
    assert "stands still" in outcomes(False, 2)
