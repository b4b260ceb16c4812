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


@pytest.mark.parametrize("name", ["token_weights.cu", "value_lora.cu"])
def test_a_wait_that_runs_out_does_so_for_the_whole_warp(name):
    # where a wait's result decides what follows, it is joined over the warp (or the block) first: a lane that left
    # alone would be waited for by the others at their next warp-wide step
    lines = _text(os.path.join(CSRC, name)).splitlines()
    for i, line in enumerate(lines):
        for m in re.finditer(r"(mbar_wait\w*|wait_pair<PAIR>)\(", line):
            if line.lstrip().startswith(("mbar_wait", "__device__", "//", "return PAIR ?")) or re.match(
                    r"\s*(for|if) \(.*\) mbar_wait\(", line) and "ok" not in line:
                continue        # a definition, or a wait whose result is not used
            statement = " ".join(lines[i:i + 5])
            joined = "__all_sync" in line[:m.start()] or re.match(r".*?;\s+(ok = __syncthreads_and\(|if \(!warp_agrees\()",
                                                                  statement)
            assert joined, "%s:%d %s" % (name, i + 1, line.strip())


def test_both_blocks_of_a_pair_wait_for_its_last_commit():
    # commit<PAIR> arrives in both CTAs: neither may end before the last one (`fin`) has landed in it
    text = _text(os.path.join(CSRC, "token_weights.cu"))
    waits = re.findall(r"^.*mbar_wait\(&ms\.fin, 0\);", text, re.M)
    assert len(waits) == 2 and any("rank > 0" in w for w in waits)
    end = text[text.index("Neither CTA of a pair ends"):]
    assert end.index("sync_all<PAIR>()") < end.index("mbar_wait(&ms.fin, 0)") < end.rindex("sync_all<PAIR>()", 0, end.index("tmem_free"))


def test_a_wait_for_a_whole_request_goes_by_its_tiles():
    # q_free completes with the last tile of a request, which at the sizes accepted may take longer than the limit of
    # one step's wait: 2^30 tokens of 2,048 rows are 2^22 tiles of a pair, each about 4,700 cycles
    common, text = (_text(os.path.join(CSRC, n)) for n in ("common.cuh", "token_weights.cu"))
    limit = int(re.search(r"kWaitCycles = (\d+)LL", common).group(1))
    tile = 1 << int(re.search(r"kTileCycles = 1 << (\d+);", text).group(1))
    tiles, cycles = 2**22, 4700
    assert tiles * cycles > limit               # one step's limit would not do
    assert limit + tiles * tile > 2 * tiles * cycles
    (wait,) = re.findall(r"warp_wait\w*\(&ms\.q_free.*\)", text)
    assert "kWaitCycles + tiles * kTileCycles" in wait
    # a role that gives up meanwhile ends it at once
    (body,) = _bodies(common, r"bool warp_wait_long\(")
    assert re.search(r"while \(!ok && !aborted\(abort_flag\)\)", body)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_every_status_word_is_read(path):
    # each source has a status word of its own; what a kernel may set there, device_status has to see
    text = re.sub(r"//.*", "", _text(path))
    sets = re.search(r"\b(flag|mbar_wait|warp_wait|warp_wait_long|kv_row|kv_row_of_page|request_len)\(|\bTileIter<|\bUnitCursor<", text)
    readers = re.findall(r"cudaError_t (\w+_status)\(unsigned int \*flags, bool clear\) \{ return read_status", text)
    if not sets or os.path.basename(path) == "api.cu":
        return
    assert len(readers) == 1, "no reader of this source's status word"
    table = re.search(r"\(\*readers\[\]\).*?\};", _text(os.path.join(CSRC, "api.cu")), re.S).group(0)
    assert "mla::" + readers[0] in table
