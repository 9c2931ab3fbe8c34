"""What a kernel's source has to hold where no run shows its absence (no GPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_03_gb300", "csrc")
REMOTE = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))) if "map_shared_rank" in open(p).read()]


def block(text, start):
    """The text from the brace at or after `start` to the one that closes it."""
    start = text.index("{", start)
    depth = 0
    for end in range(start, len(text)):
        depth += (text[end] == "{") - (text[end] == "}")
        if depth == 0:
            return text[start:end + 1]
    raise ValueError("unbalanced braces")


def kernels(path):
    """The bodies of the __global__ functions, without comments and lambdas (whose returns leave no kernel)."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer("__global__", text):
        body = block(text, text.index(") {", m.end()))
        for at in [x.start() for x in re.finditer(r"= \[&\]\(", body)][::-1]:
            body = body.replace(block(body, at), "", 1)
        yield body


@pytest.mark.parametrize("path", REMOTE, ids=os.path.basename)
def test_a_cluster_has_started_before_its_shared_memory_is_touched(path):
    """Shared memory of another CTA exists once that CTA runs: the kernel arrives at a cluster
    barrier in front of all branches, and waits before the first access to another's
    memory and before every way out that comes earlier."""
    bodies = [b for b in kernels(path) if "map_shared_rank" in b]
    assert bodies
    for body in bodies:
        remote = body.index("map_shared_rank")
        arrive = body.find("cluster.barrier_arrive(")
        assert 0 <= arrive < min(body.index("if ("), body.index("return;"))
        waits = [m.start() for m in re.finditer(r"cluster\.barrier_wait\(", body)]
        at = arrive
        for way in [m.start() for m in re.finditer("return;", body) if m.start() < remote] + [remote]:
            assert any(at < w < way for w in waits)
            at = way


@pytest.mark.parametrize("name,branch,aligned", [
    # lanes without a row skip the stores, and lanes add different numbers of values
    ("kda_tree_attention_tc.cu", "if (!real) continue;", "tmem_ld32(o_col + x, o);"),
    # the solve's loops are as long as a group's lines
    ("kda_tree.cu", "wlo[m * C::WLD + j] =", "ldsm4(abase"),
    # values that are not finite are added where a lane's node sees them
    ("kda_tree.cu", "seen[o][x >> 1][x & 1] +=", "yh[i][t] = transpose8x8(hi);")])
def test_a_warp_is_together_for_its_aligned_instructions(name, branch, aligned):
    """Instructions that a whole warp issues as one stand behind a __syncwarp where lanes took different
    ways before them: in a loop, at the iteration's start."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    at, branched = text.index(aligned), text.index(branch)
    if branched < at:
        assert "__syncwarp();" in text[branched:at]
    else:
        loop = max(m.start() for m in re.finditer(r"\n +for \(", text[:at]))
        assert "__syncwarp();" in text[loop:at]
