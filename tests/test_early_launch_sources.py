"""Rules of the kernels that start early, share a cluster or walk tiles, read
from their sources: a breach would show in a run by chance only."""

import os
import re

import pytest

import mla_decode_paged_gb300 as mla

CSRC = os.path.join(os.path.dirname(os.path.abspath(mla.__file__)), "csrc")


def _text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def _function(text, head):
    """From the first match of `head` to the line that closes it."""
    m = re.search(head, text)
    assert m, head
    return text[m.start():text.index("\n}", m.start())]


def test_warps_meet_before_the_shared_cluster_barriers():
    # barrier.cluster.*.aligned is for whole warps
    text = _text("cluster.cuh")
    for name in ("cluster_arrive", "cluster_wait"):
        body = _function(text, r"void %s\(\)" % name)
        assert body.index("__syncwarp()") < body.index("barrier.cluster")
    assert len(re.findall(r"barrier\.cluster", text)) == 2


@pytest.mark.parametrize("name", ["absorb.cu", "index_scores.cu", "norm_rope.cu", "select.cu"])
def test_a_kernel_that_starts_early_waits_for_the_one_before(name):
    # launched while the kernel before still runs, it may touch no global memory before grid_wait()
    text = _text(name)
    early = set(re.findall(r"launch_early\((\w+)", text)) | set(re.findall(r"cudaLaunchKernelEx\(&cfg, (\w+)", text))
    assert early
    for kernel in early:
        body = _function(text, r"\b%s\(" % kernel)
        assert body.count("grid_wait();") == 1, kernel
        before = body[body.index("{"):body.index("grid_wait();")]
        before = re.sub(r"const auto fetch = .*?\n    \};", "", before, flags=re.S)       # called after it
        assert not re.search(r"__ldg|\brow_of\(|\bfind_start|\bfetch\(|\breturn\b", before), kernel


@pytest.mark.parametrize("name", ["absorb.cu", "index_scores.cu"])
def test_a_wait_that_decides_is_joined_over_the_warp(name):
    # mbar_wait alone: only where its result is not used
    for line in _text(name).splitlines():
        if re.search(r"\bmbar_wait\(", line):
            assert re.match(r"\s*((for|if) \(.*\) )?mbar_wait\(&ms\.\w+(\[.*\])?, .*\);\s*$", line), line
            assert "ok" not in line and "=" not in re.sub(r"[<>!=]=|int k = .*?;|int u = .*?;", "", line.split("mbar_wait")[0]), line


@pytest.mark.parametrize("name", ["absorb.cu", "index_scores.cu"])
def test_every_issued_product_ends_before_its_memory_is_given_back(name):
    body = _function(_text(name), r"void mma_issuer\(")
    assert body.index("tc::commit(&ms.fin)") < body.index("mbar_wait(&ms.fin, 0)")
    assert body.rstrip().endswith("mbar_wait(&ms.fin, 0);")


def test_the_scores_wait_for_a_request_goes_by_its_tiles():
    # q_free completes with a request's last tile: 2^31 tokens are 2^24 tiles, about 1,300 cycles each
    text = _text("index_scores.cu")
    limit = int(re.search(r"kWaitCycles = (\d+)LL", _text("common.cuh")).group(1))
    tile = 1 << int(re.search(r"kTileCycles = 1 << (\d+);", text).group(1))
    tiles, cycles = 2**24, 1300
    assert tiles * cycles > limit and limit + tiles * tile > 2 * tiles * cycles
    (wait,) = re.findall(r"warp_wait_long\(&ms\.q_free.*?\)\)", text, re.S)
    assert "kWaitCycles + pending * kTileCycles" in wait


def test_no_block_of_a_cluster_ends_while_its_memory_is_read():
    body = _function(_text("select.cu"), r"\bselect_kernel\(")
    assert body.rstrip().endswith("if (!one) cluster_wait();")
    assert body.rindex("remote(") < body.rindex("cluster_arrive();") < body.rindex("cluster_wait();")
    assert body.count("cluster_arrive();") == 2 and body.count("cluster_wait();") == 3       # the first's on either path


@pytest.mark.parametrize("name", ["absorb.cu", "index_scores.cu", "norm_rope.cu", "select.cu", "cluster.cuh", "tile_walk.cuh",
                                  "vec8.cuh", "tc.cuh"])
def test_a_kernel_that_starts_early_reads_by_plain_loads(name):
    # a read-only load says that its data does not change while the kernel runs, and may be moved before grid_wait()
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", _text(name))


def test_the_requests_lengths_are_read_by_plain_loads():
    body = _function(_text("common.cuh"), r"int request_len\(")
    assert "indptr[r]" in body and "__ldg(indptr" not in body


@pytest.mark.parametrize("name", ["absorb.cu", "index_scores.cu", "norm_rope.cu", "select.cu"])
def test_no_argument_is_dereferenced_before_the_wait(name):
    text = _text(name)
    early = set(re.findall(r"launch_early\((\w+)", text)) | set(re.findall(r"cudaLaunchKernelEx\(&cfg, (\w+)", text))
    for kernel in early:
        body = _function(text, r"\b%s\(" % kernel)
        before = body[body.index("{"):body.index("grid_wait();")]
        before = re.sub(r"const auto (fetch|copy) = .*?\n    \};", "", before, flags=re.S)       # called after it
        assert not re.search(r"\ba\.\w+ ?\[|\*a\.|\ba\.(x|weight|positions|slots|cos_sin|q|weights|q_scales|pages|indptr|scores)\b", before)


@pytest.mark.parametrize("name", ["value_gate.cu", "merge_row.cuh"])
def test_the_value_kernel_reads_by_plain_loads(name):
    # launched while attend or merge still run; its gate and lengths may be written by whatever kernel comes before
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", _text(name))
