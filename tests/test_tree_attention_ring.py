"""The tensor-core tree attention's ring of key and value tiles, as a model of its
barriers (no GPU): whichever load or warp is late, every product reads the tile it
is meant to read, and every wait ends.

The numbers of slots, barriers and buffers, and what the value warp waits for, come
from the kernel's source.  An mbarrier wait with a parity returns when the current
phase has the other one, so a waiter must neither be two phases ahead nor behind.
"""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_03_gb300", "csrc",
                   "kda_tree_attention_tc.cu")


def value(expr, env):
    """A C expression of whole numbers with conditionals."""
    expr = expr.strip()
    depth, mark = 0, None
    for i, c in enumerate(expr):
        depth += (c == "(") - (c == ")")
        if c == "?" and depth == 0:
            mark = i
        elif c == ":" and depth == 0:
            return value(expr[mark + 1:i] if eval(expr[:mark], {}, env) else expr[i + 1:], env)
    if expr[0] == "(" and expr[-1] == ")":
        return value(expr[1:-1], env)
    return int(eval(expr.replace("/", "//"), {}, env))


def config(D, QT):
    text = open(SRC).read()
    env = {"D": D, "QT": QT}
    for name in ("SLOTS", "FULLS", "BUFS", "RING"):
        m = re.search(r"constexpr int " + name + r" = ([^,;]+)[,;]", text)
        # (without a number of its own: a barrier per slot)
        env[name] = env["SLOTS"] if m is None and name == "FULLS" else value(m.group(1), env)
    values = text[text.index("- values"):text.index("- softmax")]
    env["value_waits_for_keys"] = bool(re.search(r"wait\(full\(k_use", values))
    return env


class Bar:
    def __init__(self):
        self.phase = 0

    def done(self, parity):
        return self.phase & 1 != parity


def simulate(cfg, units, late):
    """units: per unit the steps (one or two of 64 keys) of its tiles; late: the (actor, number)s
    that go only when nothing else can, one at a time.  Returns None or what went wrong."""
    slots, fulls, bufs, ring = (cfg[x] for x in ("SLOTS", "FULLS", "BUFS", "RING"))
    tiles = [s for u in units for s in u]
    full, empty = [Bar() for _ in range(fulls)], [Bar() for _ in range(slots)]
    s_full, s_free = [Bar() for _ in range(bufs)], [Bar() for _ in range(bufs)]
    p_full, o_full, v_ready = [Bar() for _ in range(2)], [Bar() for _ in range(4)], [Bar() for _ in range(ring)]
    held = [None] * slots                          # the use whose bytes a slot holds
    wrong = []

    class Complete:                                # something asynchronous: goes when scheduled
        def __init__(self, name, act):
            self.name, self.act = name, act

    pending = []

    def loader():
        for u in range(2 * len(tiles)):
            s = u % slots
            if u >= slots:
                yield lambda: empty[s].done((u // slots - 1) & 1)
            held[s] = None

            def land(u=u, s=s):
                held[s] = u
                full[u % fulls].phase += 1
            pending.append(Complete(("load", u), land))
            yield lambda: True

    def arrive(bar):
        def go():
            bar.phase += 1
        return go

    def scores():
        j = 0
        for t, steps in enumerate(tiles):
            u = 2 * t
            yield lambda: full[u % fulls].done((u // fulls) & 1)
            for _ in range(steps):
                if j >= bufs:
                    yield lambda: s_free[j % bufs].done((j // bufs - 1) & 1)
                if held[u % slots] != u:
                    wrong.append(f"scores of tile {t} read slot {u % slots} holding {held[u % slots]}, not {u}")
                arrive(s_full[j % bufs])()
                j += 1
                yield lambda: True
            arrive(empty[u % slots])()

    def values():
        for t in range(len(tiles)):
            k, v = 2 * t, 2 * t + 1
            if cfg["value_waits_for_keys"]:
                yield lambda: full[k % fulls].done((k // fulls) & 1)
            yield lambda: full[v % fulls].done((v // fulls) & 1)
            if held[v % slots] != v:
                wrong.append(f"values of tile {t} prepared in slot {v % slots} holding {held[v % slots]}, not {v}")
            arrive(v_ready[t % ring])()

    def sums():
        j = 0
        for t, steps in enumerate(tiles):
            v = 2 * t + 1
            yield lambda: v_ready[t % ring].done((t // ring) & 1)
            for _ in range(steps):
                yield lambda: p_full[j & 1].done((j >> 1) & 1)
                if held[v % slots] != v:
                    wrong.append(f"sums of tile {t} read slot {v % slots} holding {held[v % slots]}, not {v}")
                arrive(o_full[j & 3])()
                j += 1
            arrive(empty[v % slots])()

    def softmax():
        j = 0
        for unit in units:
            done = 0
            for steps in unit:
                for _ in range(steps):
                    yield lambda: s_full[j % bufs].done((j // bufs) & 1)
                    arrive(s_free[j % bufs])()
                    if done >= 2:
                        yield lambda: o_full[(j - 2) & 3].done(((j - 2) >> 2) & 1)
                    arrive(p_full[j & 1])()
                    done, j = done + 1, j + 1
            yield lambda: o_full[(j - 1) & 3].done(((j - 1) >> 2) & 1)

    actors = {f.__name__: [f(), None, 0] for f in (loader, scores, values, sums, softmax)}
    for a in actors.values():
        a[1] = next(a[0], None)

    def step(name):
        a = actors[name]
        a[1] = next(a[0], None)
        a[2] += 1

    def ready(name):
        a = actors[name]
        return a[1] is not None and a[1]()

    while True:
        moved = False
        for name in actors:
            if ready(name) and (name, actors[name][2]) not in late:
                step(name)
                moved = True
        for c in list(pending):
            if c.name not in late:
                pending.remove(c)
                c.act()
                moved = True
        if not moved and pending:                  # now a late one
            pending.pop(0).act()
            moved = True
        for name in [n for n, _ in late if n in actors]:
            if not moved and ready(name):
                step(name)
                moved = True
        if wrong:
            return wrong[0]
        if not moved:
            stuck = [n for n, a in actors.items() if a[1] is not None]
            return f"{stuck} wait for ever" if stuck else None


# per unit the steps of its tiles: long caches, units of one and two tiles, ragged ones
PATTERNS = [[[2] * 12], [[1]] * 12, [[2, 1], [1]] * 6, [[1], [2, 1], [1]] * 4, [[2, 2, 1], [1], [2], [1], [1]] * 2,
            [[2, 1], [1], [1], [2, 2, 2], [1]] * 2, [[2]] * 8]


@pytest.mark.parametrize("D,QT", [(64, 1), (64, 2), (128, 1), (128, 2)])
@pytest.mark.parametrize("pattern", range(len(PATTERNS)))
def test_whatever_is_late(D, QT, pattern):
    cfg, units = config(D, QT), PATTERNS[pattern]
    tiles = sum(len(u) for u in units)
    assert cfg["SLOTS"] >= 4 and cfg["FULLS"] % cfg["SLOTS"] == 0
    late = [(("load", u),) for u in range(2 * tiles)]
    late += [((a, i),) for a in ("loader", "scores", "values", "sums", "softmax") for i in range(6 * tiles)]
    # two loads into one slot
    late += [(("load", u), ("load", u + cfg["SLOTS"])) for u in range(2 * tiles - cfg["SLOTS"])]
    for these in late:
        found = simulate(cfg, units, these)
        assert found is None, (cfg, these, found)


@pytest.mark.parametrize("D,QT", [(64, 1), (64, 2), (128, 1), (128, 2)])
def test_lines_of_the_units_under_way_fit_their_ring(D, QT):
    """A unit's end may still be read while the value warp prepares all tiles behind it in the
    ring: of SLOTS uses in a row up to half, rounded up, are values."""
    cfg = config(D, QT)
    assert cfg["RING"] > (cfg["SLOTS"] + 1) // 2
