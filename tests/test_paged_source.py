"""Rules of the paged kernels' source that no run can show: a warp-wide instruction
whose lanes arrive apart is undefined, and may work for as long as the compiler
happens to bring them together."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "io_aware_exact_12_gb300", "csrc")
FILES = ["attn_paged_append.cu", "attn_paged_decode.cu", "attn_paged_select.cu"]


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", FILES)
def test_block_and_cluster_barriers_bring_the_warp_together_first(name):
    """`.aligned` (and bar.sync, which implies it) wants all lanes of a warp at once.  Their callers come out of spins and
    loops whose lanes leave at different times, so the barrier's own function has to gather them."""
    src = _source(name)
    for at in (m.start() for m in re.finditer(r'"(?:barrier\.cluster\.arrive|barrier\.sync|bar\.sync)\b', src)):
        body = src[src.rindex("__forceinline__", 0, at):at]
        body = body[body.index("{") + 1:]
        assert body.split("asm")[0].strip() == "__syncwarp();", body


@pytest.mark.parametrize("name", FILES)
def test_matrix_steps_follow_a_warp_barrier(name):
    """ldmatrix, movmatrix and mma want the warp together too: between the last branch on a lane's own data (a spin on a
    barrier, a page that is not there) and a loop of them stands a warp barrier."""
    src = _source(name)
    for m in re.finditer(r"for \([^;]*;[^;]*;[^)]*\) \{", src):
        if m.group(0) not in ("for (; tiles > 0; --tiles, ++turn) {", "for (int i = 0; i < groups; ++i) {"):
            continue
        body = src[m.end():]
        first = min(body.index(x) for x in ("ldsm4(", "mma16<") if x in body)
        here = [x.start() for x in re.finditer(r"__syncwarp\(\);", body[:first])]
        here = [x for x in here if body.count("{", 0, x) == body.count("}", 0, x)]  # of the loop itself, not of a branch
        assert here, "no warp barrier before the first matrix step"
        last = here[-1]
        between = body[last:first]
        assert "if (" not in between and "mbar_wait" not in between and "look_up" not in between, between
