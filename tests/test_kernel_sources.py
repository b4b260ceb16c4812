"""What the kernels' sources have to hold throughout, read from the text:
rules whose breach a run would show by chance only."""

import glob
import os
import re

import pytest

import mla_decode_paged_gb300 as mla

CSRC = os.path.join(os.path.dirname(os.path.abspath(mla.__file__)), "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _text(path):
    with open(path) as f:
        return f.read()


def _bodies(text, pattern):
    """The text of every function whose body matches, from its opening line."""
    for m in re.finditer(r"^[^\s/#].*\)\s*\{\n(?:.*\n)*?\}", text, re.M):
        if re.search(pattern, m.group(0)):
            yield m.group(0)
    for m in re.finditer(r"^[^\s/#].*\)\s*\{.*\}$", text, re.M):      # on one line
        if re.search(pattern, m.group(0)):
            yield m.group(0)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_warps_meet_before_a_cluster_barrier(path):
    # barrier.cluster.*.aligned is for whole warps: its wrapper brings lanes that took a branch together first
    text = _text(path)
    uses = len(re.findall(r"barrier\.cluster\.arrive\S*aligned", text))
    found = list(_bodies(text, r"barrier\.cluster\.\w+\S*aligned"))
    assert sum(len(re.findall(r"barrier\.cluster\.arrive\S*aligned", b)) for b in found) == uses
    for body in found:
        assert re.search(r"__sync(warp|threads)\(\)", body[:body.index("barrier.cluster")]), body
