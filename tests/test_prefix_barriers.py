"""The prefix kernel's barriers, product by product (no GPU): arrival counts and the parities of all waits are
the source's own text.  Loads land some time after they are asked for, products are done some time after they
are issued, each row tile's in the order of their issue, the two tiles' in any; the turn is passed before a
tile's last products of the scores.  Modelled beside the ring and the weights: the tail of a cut value tile,
zeroed for both tiles by one of them, and the sums, read by four warps before the next unit overwrites them."""
import os
import random
import re

import pytest

from tests import test_tree_attention_ring as tree
from tests.test_prefix_ring import CSRC, Bar

TEXT = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "kda_prefix_attention_tc.cu")).read())
NAMES = ("full", "empty", "s_full", "p_full", "o_full", "turn", "q_full", "q_free", "v_ready")


def arguments(call):
    """The arguments of every `call(` in the source, as texts."""
    for m in re.finditer(r"(?<![\w.])" + call + r"\(", TEXT):
        depth, args, start = 1, [], m.end()
        for at in range(m.end(), len(TEXT)):
            depth += (TEXT[at] in "([{") - (TEXT[at] in ")]}")
            if depth == 0 or (depth == 1 and TEXT[at] == ","):
                args.append(" ".join(TEXT[start:at].split()))
                start = at + 1
            if depth == 0:
                break
        yield args


def counts():
    return {re.match(r"\w+", bar).group(): count for bar, count in arguments("mbar_init")}


def parities():
    """Barrier -> what its waits compute, as Python."""
    found = {}
    for bar, parity in arguments("wait"):
        parity = parity.replace("C::SLOTS", "SLOTS").replace("/", "//")
        parity = re.sub(r"\(([^()?]+) \? ([^:]+) : ([^()]+)\)", r"(\2 if \1 else \3)", parity)
        assert found.setdefault(re.match(r"\w+", bar).group(), parity) == parity
    return found


def test_every_barrier_is_modelled():
    assert set(counts()) == set(NAMES) == set(parities())
    # the order in which a step's products, commits and the turn are issued
    scores = TEXT[TEXT.index("auto scores = "):TEXT.index("for (; run.left > 0 && ok;", TEXT.index("auto scores = "))]
    order = [scores.index(x) for x in ("mma_bf16_w(", "if (ks == D / 16 - 3) your_turn();", "mma_commit_w(s_full(t))",
                                       "mma_commit_w(empty(s))", "if (last) mma_commit_w(q_free)")]
    assert order == sorted(order)
    step = TEXT[TEXT.index("if (!landed(j, 1)) break;"):TEXT.index("} else if (warp >= 4)")]
    order = [step.index(x) for x in ("mbar_arrive(v_ready)", "wait(v_ready", "!landed(j + 1, 0)", "!my_turn() || !wait(p_full(t)",
                                     "mma_tmem_a_w(", "mma_commit_w(empty(s))", "scores(j + 1, i + 2 == cnt)",
                                     "mma_commit_w(o_full(t))", "your_turn();")]
    assert order == sorted(order)
    assert "mbar_arrive(turn(1 - t))" in TEXT and "mbar_arrive(p_full(t))" in TEXT


def model(SLOTS, QT, units, rng, bars=None):
    """`units`: their key tiles, the last of which may be cut: (tiles, cut)."""
    n_of, parity = bars or (counts(), parities())
    count = {b: eval(n_of[b], {}, {"QT": QT}) for b in NAMES}
    code = {b: compile(parity[b], b, "eval") for b in NAMES}
    one = {b: Bar(count[b]) for b in ("q_full", "q_free", "v_ready")}
    many = {b: [Bar(count[b]) for _ in range(SLOTS)] for b in ("full", "empty")}
    tile = {b: [Bar(count[b]) for _ in range(QT)] for b in ("s_full", "p_full", "o_full", "turn")}
    held, query, landing = [None] * SLOTS, [None], []
    queues = [[] for _ in range(QT)]
    score, weight = [None] * QT, [[None] * 4 for _ in range(QT)]
    sums, unread = [None] * QT, [set() for _ in range(QT)]

    def wait(name, bar, **names):
        p = eval(code[name], {}, {"SLOTS": SLOTS, **names})
        return lambda: bar.done(p)

    def loader():
        use = 0
        yield lambda: True
        for seg, (cnt, cut) in enumerate(units):
            if seg > 0:
                yield wait("q_free", one["q_free"], seg=seg)

            def queries(seg=seg):
                query[0] = seg
                one["q_full"].arrive()
            query[0] = None
            landing.append(queries)
            for i in range(cnt):
                for kv in range(2):
                    s = use % SLOTS
                    if use >= SLOTS:
                        yield wait("empty", many["empty"][s], use=use)

                    def lands(s=s, what=(seg, i, kv)):
                        held[s] = [what, False]
                        many["full"][s].arrive()
                    held[s] = None
                    landing.append(lands)
                    use += 1

    def products(t):
        j = cuts = turns = 0
        issue = queues[t].append

        def landed(i, kv):
            return wait("full", many["full"][(2 * i + kv) % SLOTS], i=i, kv=kv)

        def my_turn():
            nonlocal turns
            n = turns
            turns += 1
            return (lambda: True) if QT == 1 or (t == 0 and n == 0) else wait("turn", tile["turn"][t], t=t, n=n)

        def your_turn():
            if QT == 2:
                tile["turn"][1 - t].arrive()

        def scores(seg, i, j, last):
            s = 2 * j % SLOTS

            def product(end):
                assert held[s][0] == (seg, i, 0) and query[0] == seg
                assert weight[t] == [None] * 4           # the weights in the scores' place are read
                score[t] = (seg, i) if end else None

            def commit():
                tile["s_full"][t].arrive()
                many["empty"][s].arrive()
                if last:
                    one["q_free"].arrive()
            issue(lambda: product(False))
            your_turn()
            yield                                        # (the other tile may go on from here)
            issue(lambda: product(False))
            issue(lambda: product(True))
            issue(commit)

        def values(seg, i, j, last, cut):
            s = (2 * j + 1) % SLOTS

            def product():
                assert held[s] == [(seg, i, 1), cut]     # a cut tile's tail is zeros
                assert weight[t] == [(seg, i)] * 4
                assert i > 0 or not unread[t]            # the last unit's sums are read
                sums[t] = seg

            def commit():
                weight[t][:] = [None] * 4
                many["empty"][s].arrive()
                if last:
                    unread[t].update(range(4))
                    tile["o_full"][t].arrive()
            issue(product)
            issue(commit)

        for seg, (cnt, cut) in enumerate(units):
            yield wait("q_full", one["q_full"], seg=seg)
            yield landed(j, 0)
            yield my_turn()
            for _ in scores(seg, 0, j, cnt == 1):
                yield lambda: True
            for i in range(cnt):
                last = i + 1 == cnt
                yield landed(j, 1)
                if last and cut:
                    if t == 0:
                        held[(2 * j + 1) % SLOTS][1] = True
                        one["v_ready"].arrive()
                    else:
                        yield wait("v_ready", one["v_ready"], cuts=cuts)
                    cuts += 1
                if not last:
                    yield landed(j + 1, 0)
                yield my_turn()
                yield wait("p_full", tile["p_full"][t], j=j)
                values(seg, i, j, last, last and cut)
                if not last:
                    for _ in scores(seg, i + 1, j + 1, i + 2 == cnt):
                        yield lambda: True
                else:
                    your_turn()
                j += 1

    def softmax(t, warp):
        j = 0
        for seg, (cnt, _) in enumerate(units):
            for i in range(cnt):
                yield wait("s_full", tile["s_full"][t], j=j)
                assert score[t] == (seg, i) and weight[t][warp] is None
                assert i == 0 or sums[t] == seg          # (the sums that it may rescale)
                weight[t][warp] = (seg, i)
                tile["p_full"][t].arrive()
                j += 1
            yield wait("o_full", tile["o_full"][t], seg=seg)
            yield lambda: True
            assert sums[t] == seg
            unread[t].discard(warp)

    def engine(queue, first_in_first_out):
        while True:
            yield lambda: bool(queue)
            queue.pop(0 if first_in_first_out else rng.randrange(len(queue)))()

    actors = [loader()] + [products(t) for t in range(QT)] + [softmax(t, w) for t in range(QT) for w in range(4)]
    machines = [engine(q, True) for q in queues] + [engine(landing, False)]
    waits = {a: next(a) for a in actors + machines}
    left, pace = set(actors), {a: rng.choice([1, 1, 1, 20]) for a in actors + machines}
    while left or any(queues) or landing:
        ready = [a for a, w in waits.items() if w()]
        assert ready, "every wait ends"
        a = rng.choices(ready, [1 / pace[x] for x in ready])[0]
        try:
            waits[a] = next(a)
        except StopIteration:
            del waits[a]
            left.discard(a)


def some_units(rng):
    return [(rng.choice([1, 1, 2, 3, 7]), rng.random() < 0.5) for _ in range(rng.randint(1, 6))]


@pytest.mark.parametrize("D,QT", [(64, 1), (64, 2), (128, 1), (128, 2)])
def test_the_barriers_of_the_prefix_kernel(D, QT):
    slots = tree.value(re.search(r"constexpr int SLOTS = ([^,;]+)[,;]", TEXT).group(1), {"D": D, "QT": QT})
    rng = random.Random(D + QT)
    for _ in range(250):
        model(slots, QT, some_units(rng), rng)


@pytest.mark.parametrize("bar,count,parity", [
    ("p_full", "3", None), ("empty", "1", None), ("q_free", "1", None), ("v_ready", None, "0"), ("o_full", None, "1"),
    ("turn", None, "n & 1"), ("s_full", None, "(j + 1) & 1")])
def test_the_model_sees_a_wrong_barrier(bar, count, parity):
    n_of, p_of = counts(), parities()
    if count:
        n_of[bar] = count
    if parity:
        p_of[bar] = parity
    rng = random.Random(1)
    with pytest.raises((AssertionError, TypeError)):
        for _ in range(300):
            model(5, 2, some_units(rng), rng, (n_of, p_of))
