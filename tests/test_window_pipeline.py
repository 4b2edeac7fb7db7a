"""The waits of the window attention's chunk kernel, as a model on the CPU: the warps that load, zero and
multiply K and V tiles, and the barriers between them.

A barrier's wait names a parity: it passes while the phase of that parity is the last one completed, so
a warp that falls a whole turn of the ring behind waits for a phase that lies in the past, and for good
if the ring needs it to go on.  The model runs the warps in any order, each as far behind the others as
the barriers let it fall.  What arrives at ``kv_empty``, and how many arrivals it takes, is read from the
kernel's source."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_sparse_clsa_b200", "csrc",
                   "window_tc.cu")


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0   # phase: how many have completed

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0, "more arrivals than the phase takes"
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passes(self, parity):                                    # try_wait.parity
        return (self.phase - 1) & 1 == parity & 1                # the phase before the current one has it


def kernel():
    """(arrivals a phase of kv_empty takes, whether the warp that zeroes rows makes one for each tile)."""
    text = open(SRC).read()
    count = int(re.search(r"mbar_init\(kv_empty \+ i, (\d+)\)", text).group(1))
    zeroing = text[text.index("warp == kFixWarp"):text.index("warp == kMmaWarp")]
    return count, "mbar_arrive(kv_empty" in zeroing


def actors(tiles, slots, count, zeroing_arrives):
    """Generators that yield what they wait for: (barrier, parity).  tiles[j]: token tile j has rows to zero."""
    full = [Barrier(1) for _ in range(slots)]
    empty = [Barrier(count) for _ in range(slots)]
    fixed = [Barrier(1) for _ in range(4)]
    n = 2 * len(tiles)                                           # K, V, K, V, ...

    def load():
        for x in range(n):
            if x >= slots:
                yield empty[x % slots], x // slots - 1
            full[x % slots].arrive()

    def zero():
        nfix = 0
        for x in range(n):
            yield full[x % slots], x // slots
            if x % 2 and tiles[x // 2]:
                fixed[nfix & 3].arrive()
                nfix += 1
            if zeroing_arrives:
                empty[x % slots].arrive()

    def mma():
        nfix = 0
        yield full[0], 0
        empty[0].arrive()                                        # the first scores have read their K tile
        for j, fix in enumerate(tiles):
            v, k = 2 * j + 1, 2 * j + 2
            if fix:
                yield fixed[nfix & 3], nfix >> 2
                nfix += 1
            else:
                yield full[v % slots], v // slots
            if k < n:
                yield full[k % slots], k // slots
            empty[v % slots].arrive()
            if k < n:
                empty[k % slots].arrive()

    return {"load": load(), "zero": zero(), "mma": mma()}


def run(tiles, slots, count, zeroing_arrives, pick):
    """Who is stuck at the end: nobody, where every warp came through."""
    todo = actors(tiles, slots, count, zeroing_arrives)
    waits = {}
    for name in list(todo):
        try:
            waits[name] = next(todo[name])
        except StopIteration:
            del todo[name]
    while todo:
        ready = [a for a in todo if waits[a][0].passes(waits[a][1])]
        if not ready:
            return sorted(todo)
        a = pick(ready)
        try:
            waits[a] = next(todo[a])
        except StopIteration:
            del todo[a]
    return []


ORDERS = {"zeroing last": lambda r: min(r, key=("load", "mma", "zero").index), "zeroing first": lambda r: max(r, key=("load", "mma", "zero").index),
          "loads last": lambda r: max(r, key=("mma", "zero", "load").index), "products last": lambda r: max(r, key=("zero", "load", "mma").index)}


@pytest.mark.parametrize("slots", [5, 8])
def test_no_order_of_the_warps_stops_the_ring(slots):
    """Items whose last tiles have rows to zero, and long runs of tiles that have none, in every extreme order
    of the warps and in random ones."""
    count, arrives = kernel()
    cases = [[n == m - 1 for n in range(m)] for m in (1, 2, 3, 4, 9, 40)]
    cases += [[True] * 12, [False] * 12, [True] + [False] * 20 + [True], [False] * 5 + [True] * 3 + [False] * 7 + [True]]
    rng = random.Random(slots)
    cases += [[rng.random() < p for _ in range(rng.randint(1, 60))] for p in (0.1, 0.3, 0.7) for _ in range(20)]
    for tiles in cases:
        for name, pick in ORDERS.items():
            assert run(tiles, slots, count, arrives, pick) == [], (name, tiles)
        for _ in range(5):
            assert run(tiles, slots, count, arrives, rng.choice) == [], tiles


def test_the_model_shows_a_warp_that_fell_behind():
    """Without the zeroing warp's arrivals the ring runs on, a turn ahead of it, and stops."""
    assert run([False] * 20 + [True], 5, 1, False, ORDERS["zeroing last"]) == ["mma", "zero"]
    assert run([False] * 20 + [True], 5, 1, False, ORDERS["zeroing first"]) == []
    assert run([False] * 20 + [True], 5, 2, True, ORDERS["zeroing last"]) == []
