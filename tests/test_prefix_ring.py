"""The prefix kernel's ring of key and value tiles and its turns at the tensor core, as a
model of its barriers (no GPU): in whatever order loads and warps come, every product
reads the tile and the weights it is meant to read, and every wait ends."""
import os
import random
import re

import pytest

from tests import test_tree_attention_ring as tree

CSRC = os.path.dirname(tree.SRC)


class Bar:
    """An mbarrier: `count` arrivals make a phase."""

    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return self.phase & 1 != parity & 1


def prefix_model(slots, tiles, units, rng):
    """The prefix kernel's loader, product warps and softmax groups over `units` (key tiles of each), in a
    random order of steps.  Products run in the order of their issue, some time after it."""
    full, empty = [Bar(1) for _ in range(slots)], [Bar(tiles) for _ in range(slots)]
    s_full, p_full, o_full = ([Bar(1) for _ in range(tiles)] for _ in range(3))
    turn, q_full, q_free = [Bar(1) for _ in range(tiles)], Bar(1), Bar(tiles)
    held, queue, score, weight, query = [None] * slots, [], [None] * tiles, [None] * tiles, [None]

    def loader():
        use = 0
        for seg, cnt in enumerate(units):
            if seg:
                yield lambda: q_free.done(seg - 1)
            query[0] = seg
            q_full.arrive()
            for i in range(cnt):
                for kv in range(2):
                    s = use % slots
                    if use >= slots:
                        yield lambda: empty[s].done(use // slots - 1)
                    held[s] = (seg, i, kv)
                    full[s].arrive()
                    use += 1

    def products(t):
        j = turns = 0

        def mine():
            n = turns - 1
            return tiles == 1 or (t == 0 and n == 0) or turn[t].done(n - 1 if t == 0 else n)

        def landed(n):
            return full[n % slots].done(n // slots)

        def scores(seg, i, j, last):
            s = 2 * j % slots

            def run():
                assert held[s] == (seg, i, 0) and query[0] == seg
                assert weight[t] is None                 # the weights in the scores' place are read
                score[t] = (seg, i)
                s_full[t].arrive()
                empty[s].arrive()
                if last:
                    q_free.arrive()
            queue.append(run)

        def sums(seg, i, j, last):
            s = (2 * j + 1) % slots

            def run():
                assert held[s] == (seg, i, 1) and weight[t] == (seg, i)
                weight[t] = None
                empty[s].arrive()
                if last:
                    o_full[t].arrive()
            queue.append(run)

        def pass_on():
            if tiles == 2:
                turn[1 - t].arrive()

        for seg, cnt in enumerate(units):
            yield lambda: q_full.done(seg)
            yield lambda: landed(2 * j)
            turns += 1
            yield mine
            scores(seg, 0, j, cnt == 1)
            pass_on()
            for i in range(cnt):
                yield lambda: landed(2 * j + 1)
                if i + 1 < cnt:
                    yield lambda: landed(2 * j + 2)
                turns += 1
                yield mine
                yield lambda: p_full[t].done(j)
                sums(seg, i, j, i + 1 == cnt)
                if i + 1 < cnt:
                    scores(seg, i + 1, j + 1, i + 2 == cnt)
                pass_on()
                j += 1

    def softmax(t):
        j = 0
        for seg, cnt in enumerate(units):
            for i in range(cnt):
                yield lambda: s_full[t].done(j)
                assert score[t] == (seg, i)
                score[t], weight[t] = None, (seg, i)
                p_full[t].arrive()
                j += 1
            yield lambda: o_full[t].done(seg)

    def core():                                          # the tensor core
        while True:
            yield lambda: bool(queue)
            queue.pop(0)()

    actors = [loader()] + [products(t) for t in range(tiles)] + [softmax(t) for t in range(tiles)]
    waits = {}
    for a in actors:
        try:
            waits[a] = next(a)
        except StopIteration:
            pass
    engine = core()
    waits[engine] = next(engine)
    while len(waits) > 1:
        ready = [a for a, w in waits.items() if w()]
        assert ready, "every wait ends"
        a = rng.choice(ready)
        try:
            waits[a] = next(a)
        except StopIteration:
            del waits[a]
    while queue:
        queue.pop(0)()


@pytest.mark.parametrize("D,QT", [(64, 1), (64, 2), (128, 1), (128, 2)])
def test_the_ring_of_the_prefix_kernel(D, QT):
    text = open(os.path.join(CSRC, "kda_prefix_attention_tc.cu")).read()
    slots = tree.value(re.search(r"constexpr int SLOTS = ([^,;]+)[,;]", text).group(1), {"D": D, "QT": QT})
    rng = random.Random(D + QT)
    for n in range(300):
        prefix_model(slots, QT, [rng.choice([1, 1, 2, 3, 7]) for _ in range(rng.randint(1, 6))], rng)
