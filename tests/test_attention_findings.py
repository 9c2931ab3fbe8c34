"""The attention kernels' findings, in their source (no GPU: no wait is made to run out)."""
import os
import re

import pytest

from tests.test_tree_sources import CSRC


@pytest.mark.parametrize("name", ["kda_tree_attention_tc.cu", "kda_prefix_attention_tc.cu"])
def test_a_finding_takes_no_others_place(name):
    """A word for each finding: a bad length that every CTA has found hides no wait that ran out later."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert "atomicCAS(" not in text
    assert re.findall(r"words\[W_STATUS\] = ([^;]+);", text) == ["place.status"]
    leaves = re.findall(r"left->status = ([^;]+);", text)
    assert len(leaves) == 1
    for word in ("words[W_STATUS]", "words[W_ABORT] != 0 ? KDA_DEVICE_TIMEOUT", "words[W_PAGE] != 0 ? KDA_DEVICE_BAD_PAGE"):
        assert word in leaves[0]
    assert len(re.findall(r"words\[W_PAGE\] = 1;", text)) == 1


def test_a_finding_takes_no_others_place_in_the_other_form():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "kda_tree_attention.cu")).read())
    assert re.findall(r"s_status = ([^;]+);", text) == ["status"] and "atomicOr(&s_status" in text


def test_the_sets_are_joined_as_sets():
    for name in ("kda_tree_cut.cuh", "kda_prefix_cut.cuh"):
        text = open(os.path.join(CSRC, name)).read()
        assert "places[i].status" in text
        assert not re.search(r"max\([^;]*(status|load)", text) and not re.search(r"status = KDA_DEVICE", text)
