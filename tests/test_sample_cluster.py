"""The sampling kernel's histograms, which the CTAs of a cluster read from each other: a model
of the way by a large k to top-p (no GPU).  Whichever CTA runs ahead, every read finds the
counts that it is meant to find, and all CTAs meet at the same barriers."""
import itertools
import os
import re

import pytest

from tests import test_tree_sources as sources


def narrow():
    """The source of the border's search, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(sources.CSRC, "kda_sample.cu")).read())
    return sources.block(text, text.index("auto narrow = "))


def meets_before_it_leaves():
    """Whether the CTAs come together between a histogram's reads and every way out that follows its border."""
    text, found = narrow(), []
    for m in re.finditer(r"if \(!border\(", text):
        line_end = text.index("\n", m.start())
        brace = text[m.start():line_end].rstrip().endswith("{")
        way_out = sources.block(text, line_end - 1) if brace else text[m.start():line_end]
        assert "return;" in way_out
        found.append("cluster.sync();" in way_out[:way_out.index("return;")])
    assert len(found) == 2
    return all(found)


def cta(me, ctas, memory, meets, log):
    """One CTA of a row with fewer logits than k: yields at each step, "meet" at a cluster barrier."""
    memory[me] = "cleared"
    yield
    memory[me] = "counts"
    yield "meet"
    for r in range(ctas):                               # what every rank has of this histogram
        log.append(memory[r])
        yield
    if meets:
        yield "meet"
    memory[me] = "cleared"                              # top-p's first histogram
    yield
    memory[me] = "sums"
    yield "meet"


def run(order, ctas, meets):
    """The CTAs' steps in the order given (a CTA at a barrier waits for all); what was read."""
    memory, log = [None] * ctas, []
    actors = [cta(c, ctas, memory, meets, log) for c in range(ctas)]
    waiting = [False] * ctas
    left = set(range(ctas))
    for c in itertools.chain(order, itertools.cycle(range(ctas))):
        if not left:
            return log
        if c in left and not waiting[c]:
            try:
                waiting[c] = next(actors[c]) == "meet"
            except StopIteration:
                left.discard(c)
        if left and all(waiting[x] for x in left):
            waiting = [False] * ctas


@pytest.mark.parametrize("ctas", [2, 3])
def test_bins_are_read_before_they_are_cleared(ctas):
    meets = meets_before_it_leaves()
    steps = 10 if ctas == 2 else 8
    for order in itertools.product(range(ctas), repeat=steps):
        assert set(run(order, ctas, meets)) == {"counts"}, order


def test_the_model_sees_a_missing_barrier():
    assert any("sums" in run(order, 2, False) for order in itertools.product(range(2), repeat=12))
