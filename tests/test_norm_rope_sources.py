"""What the head norm's source has to hold where no run shows its absence (no GPU)."""
import os
import re

from tests import test_tree_sources as sources


def test_rows_are_not_read_through_the_read_only_path():
    """q_out may be q and k_out may be k: what a kernel writes it must not read by __ldg."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(sources.CSRC, "kda_norm_rope.cu")).read())
    load = sources.block(text, text.index("auto load = "))
    assert "raw[" in load and "__ldg(" not in load
    for m in re.finditer(r"__ldg\(([^;]*);", text):
        assert re.search(r"\bw\b", m.group(1)) and "source(" not in m.group(1)
