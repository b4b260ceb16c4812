"""index_select: host-side refusals (CPU), then every row's page list against
a plain selection on the GPU: ties, NaN and infinite scores, blocks cut short,
rows that see nothing, rows of all lengths."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

DEV = "cuda"
A = 1 << 20
B, C, D, E = (A + (i << 34) for i in range(1, 5))


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.library()


def _call(lib, **kw):
    a = dict(s=A, pages=B, n=100, indptr=C, R=3, qlen=2, topk=4, block=2, recent=1, sinks=1, flags=0, po=D, cap=48, io=E)
    a.update(kw)
    return lib.mla_index_select(a["s"], a["pages"], a["n"], a["indptr"], a["R"], a["qlen"], a["topk"], a["block"],
                                a["recent"], a["sinks"], a["flags"], a["po"], a["cap"], a["io"], None)


@pytest.mark.parametrize("kw,msg", [
    (dict(flags=2), b"flag"),
    (dict(R=-1), b"negative"),
    (dict(n=-1), b"negative"),
    (dict(qlen=0), b"qlen"),
    (dict(qlen=17), b"qlen"),
    (dict(topk=-1), b"topk"),
    (dict(block=0), b"block"),
    (dict(block=3), b"block"),
    (dict(block=512), b"block"),
    (dict(recent=-1), b"negative"),
    (dict(sinks=-1), b"negative"),
    (dict(recent=0), b"recent"),
    (dict(cap=47), b"too small"),
    (dict(s=None), b"null"),
    (dict(pages=None), b"null"),
    (dict(indptr=None), b"null"),
    (dict(po=None), b"null"),
    (dict(io=None), b"null"),
    (dict(s=A + 2), b"misaligned"),
    (dict(io=E + 1), b"misaligned"),
    (dict(po=A + 796), b"overlaps"),
    (dict(po=B + 396), b"overlaps"),
    (dict(io=C + 12), b"overlaps"),
    (dict(io=D + 188), b"two outputs"),
])
def test_refusals(lib, kw, msg):
    assert _call(lib, **kw) == mla.MLA_ERR_INVALID
    assert msg in lib.mla_last_error()


@pytest.mark.parametrize("kw", [dict(n=1 << 31), dict(R=(1 << 24) + 1, qlen=1, cap=1 << 30), dict(cap=1 << 31)])
def test_too_large(lib, kw):
    assert _call(lib, **kw) == mla.MLA_ERR_UNSUPPORTED


def test_capacity(lib):
    assert mla.index_select_capacity(3, 2, 100, 4, 2) == 48
    assert mla.index_select_capacity(3, 2, 100, 40, 2) == 200
    assert mla.index_select_capacity(1, 16, 1000, (1 << 31) - 1, 256) == 16000
    assert mla.index_select_capacity(0, 1, 0, 5) == 0
    with pytest.raises(mla.MlaError, match="block"):
        mla.index_select_capacity(1, 1, 10, 1, 5)


def test_binding_refusals():
    mla.build()
    s, p, i = torch.zeros(2, 9), torch.zeros(9, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for args, kw, msg in [
        ((s[0], p, i, 2), {}, "scores"), ((s.double(), p, i, 2), {}, "scores"), ((s[:, :8], p, i, 2), {}, "scores"),
        ((s.repeat(9, 1), p, i, 2), {}, "scores"), ((s, p.long(), i, 2), {}, "pages"), ((s, p, i[:0], 2), {}, "indptr"),
        ((s, p, i, 1.5), {}, "topk"), ((s, p, i, 2), {}, "CUDA"),
    ]:
        with pytest.raises(ValueError, match=msg):
            mla.index_select(*args, **kw)


# ------------------------------------------------------------------- GPU


def _plain(scores, pages, lengths, topk, block, recent, sinks, causal, start=0):
    """Every row's list by the definition, on the host."""
    lists, qlen, at = [], scores.shape[0], start
    for n in lengths:
        for tq in range(qlen):
            seen = max(0, n - qlen + tq + 1) if causal else n
            count = -(-seen // block)
            keep = min(count, topk)
            rec = min(recent, keep)
            snk = min(sinks, keep - rec)
            x = scores[tq, at:at + seen]
            x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
            x = torch.cat([x, torch.full((count * block - seen,), -math.inf)])
            top = x.view(count, block).amax(1) if count else x
            mid = torch.arange(snk, count - rec)
            best = mid[torch.sort(top[mid], descending=True, stable=True).indices[:keep - rec - snk]]
            mark = torch.zeros(count, dtype=torch.bool)
            mark[:snk] = True
            mark[count - rec:] = True
            mark[best] = True
            tok = (mark.nonzero() * block + torch.arange(block)).view(-1)
            lists.append(pages[at:at + seen][tok[tok < seen]])
        at += n
    return lists


def _run(scores, lengths, topk, block=1, recent=0, sinks=0, causal=False, **kw):
    total = sum(lengths)
    pages = torch.randperm(total + 3, generator=torch.Generator().manual_seed(total))[:total].to(torch.int32)
    indptr = torch.tensor([0] + list(torch.tensor(lengths, dtype=torch.int64).cumsum(0)), dtype=torch.int32)
    po, io = mla.index_select(scores.to(DEV), pages.to(DEV), indptr.to(DEV), topk, block=block, recent=recent, sinks=sinks,
                              causal=causal, **kw)
    lists = _plain(scores, pages, lengths, topk, block, recent, sinks, causal)
    counts = torch.tensor([0] + [x.numel() for x in lists], dtype=torch.int64).cumsum(0)
    assert torch.equal(io.cpu().long(), counts)
    want = torch.full((po.numel(),), -1, dtype=torch.int32)
    if lists:
        want[:counts[-1]] = torch.cat(lists)
    assert torch.equal(po.cpu(), want)
    assert mla.device_status() == 0
    return po, io


def _rand(qlen, total, seed=0):
    """As index_scores leaves them: many zeros."""
    return torch.randn(qlen, total, generator=torch.Generator().manual_seed(seed + total)).sub(0.3).clamp(min=0)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lengths,qlen,topk,block,recent,sinks", [
    ([1], 1, 1, 1, 0, 0),
    ([1], 4, 1, 1, 0, 0),
    ([5, 0, 3], 2, 0, 1, 0, 0),
    ([0, 0], 3, 4, 4, 1, 0),
    ([31, 32, 33, 100], 2, 16, 1, 3, 2),
    ([31, 32, 33, 100], 2, 1000, 1, 3, 2),
    ([300, 2, 513, 64], 4, 7, 2, 2, 1),
    ([300, 2, 513, 64], 4, 7, 16, 1, 0),
    ([300, 2, 513, 64], 16, 3, 32, 1, 1),
    ([3000, 20, 5130, 640], 3, 5, 64, 2, 9),
    ([3000, 20, 5130, 640], 1, 5, 256, 1, 1),
    ([8191, 8192, 8193], 1, 2000, 1, 10, 4),
    ([20000], 1, 700, 1, 0, 0),
    ([131072], 1, 2048, 1, 0, 0),
    ([131072], 2, 32, 64, 2, 1),
    ([131072], 1, 100, 8, 1, 0),
    ([131072], 1, 9000, 2, 4096, 4000),
    ([100000, 1, 2], 2, 300, 4, 1, 1),
    ([700] * 40, 8, 100, 1, 16, 0),
    ([700] * 40, 16, 10, 16, 1, 1),             # more rows than a block's threads
    ([9, 0, 2, 40] * 300, 1, 8, 1, 1, 0),
    ([9, 0, 2, 40] * 300, 2, 3, 8, 1, 1),
    ([40000] * 3 + [50] * 100, 1, 512, 1, 0, 0),
    ([50] * 300 + [20000, 9000, 4097, 4096] + [700] * 100, 1, 512, 1, 3, 1),
    ([300] * 160 + [70000, 33000], 2, 600, 8, 1, 0),
])
def test_lists(lengths, qlen, topk, block, recent, sinks, causal):
    _run(_rand(qlen, sum(lengths)), lengths, topk, block, recent, sinks, causal)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,topk,block,recent,sinks", [
    ([12000] * 170 + [16384, 16385, 40000, 1, 0], 700, 1, 2, 1),        # more rows than SMs, of a block's round and longer
    ([20000] * 170 + [100000, 33000, 5], 700, 1, 0, 0),                 # in clusters, and longer than these hold
    ([70000] * 160 + [131072, 3, 0, 300], 2048, 2, 1, 1),
    ([140000] * 154 + [9], 2048, 1, 0, 0),                              # in the largest clusters
    ([12000] * 10 + [50000, 16384, 16385, 0, 7], 700, 1, 2, 1),         # fewer
    ([30000] * 10 + [90000, 32768, 32770, 0, 7], 700, 2, 1, 0),
])
@pytest.mark.parametrize("ties", [False, True])
def test_many_long_rows(lengths, topk, block, recent, sinks, ties):
    scores = _rand(1, sum(lengths))
    _run((4 * scores).round() if ties else scores, lengths, topk, block, recent, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("requests", [1, 90])
@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64, 128, 256])
def test_every_block_size_below_zero(block, requests):
    # scores below 0 throughout: what no token filled must not count
    lengths = [(17 * block + 3 + 577 * i) % 5000 + 1 for i in range(requests)]
    scores = -torch.rand(2, sum(lengths), generator=torch.Generator().manual_seed(block)) - 0.5
    _run(scores, lengths, 7, block, 1, 1, True)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 4, 64])
def test_ties_nan_and_infinities(block):
    n = 6000
    g = torch.Generator().manual_seed(block)
    for scores in (torch.zeros(2, n), torch.full((2, n), -math.inf), torch.full((2, n), math.nan),
                   torch.randint(0, 3, (2, n), generator=g).float(),
                   torch.where(torch.rand(2, n, generator=g) < 0.3, torch.full((2, n), math.nan), torch.randn(2, n, generator=g)),
                   torch.where(torch.rand(2, n, generator=g) < 0.1, torch.full((2, n), math.inf), -torch.rand(2, n, generator=g)),
                   torch.where(torch.rand(2, n, generator=g) < 0.5, torch.tensor(0.0), torch.tensor(-0.0)).expand(2, n).contiguous(),
                   torch.randint(-2**31, 2**31 - 1, (2, n), generator=g).to(torch.int32).view(torch.float32)):
        _run(scores, [n // 3, n - n // 3], 900 // block, block, 1, 1, True)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 16])
def test_scores_that_a_row_does_not_see_do_not_matter(block):
    lengths, qlen = [200, 5000, 3], 4
    scores = _rand(qlen, sum(lengths))
    a = _run(scores, lengths, 64 // block, block, 1, 0, True)
    at = 0
    for n in lengths:
        for tq in range(qlen):
            scores[tq, at + max(0, n - qlen + tq + 1):at + n] = math.inf
        at += n
    b = _run(scores, lengths, 64 // block, block, 1, 0, True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_given_outputs_and_a_list_that_starts_past_its_first_entries():
    scores, pages = _rand(2, 255), torch.arange(1000, 1255, dtype=torch.int32)
    indptr = torch.tensor([5, 205, 225], dtype=torch.int32)
    po = torch.full((500,), 7, dtype=torch.int32, device=DEV)
    io = torch.full((5,), 7, dtype=torch.int32, device=DEV)
    a, b = mla.index_select(scores.to(DEV), pages.to(DEV), indptr.to(DEV), 30, recent=2, pages_out=po, indptr_out=io)
    assert a.data_ptr() == po.data_ptr() and b.data_ptr() == io.data_ptr()
    lists = _plain(scores, pages, [200, 20], 30, 1, 2, 0, False, start=5)
    assert io.tolist() == [0, 30, 60, 80, 100]
    assert po.tolist() == torch.cat(lists).tolist() + [-1] * 400
    with pytest.raises(mla.MlaError, match="too small"):
        mla.index_select(scores.to(DEV), pages.to(DEV), indptr.to(DEV), 30, pages_out=po[:119])


@pytest.mark.gpu
def test_no_requests():
    po, io = mla.index_select(torch.zeros(2, 0, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV),
                              torch.zeros(1, dtype=torch.int32, device=DEV), 4,
                              pages_out=torch.zeros(300, dtype=torch.int32, device=DEV))
    assert io.tolist() == [0] and po.eq(-1).all()


@pytest.mark.gpu
def test_bad_indptr_is_flagged():
    scores, pages = _rand(1, 300).to(DEV), torch.arange(300, dtype=torch.int32, device=DEV)
    po, io = mla.index_select(scores, pages, torch.tensor([0, 100, 50, 400], dtype=torch.int32, device=DEV), 20)
    assert mla.device_status() == mla.DEV_BAD_INDPTR
    assert io.tolist() == [0, 20, 20, 20]
    assert po.tolist() == _plain(scores.cpu(), pages.cpu(), [100], 20, 1, 0, 0, False)[0].tolist() + [-1] * 40
    # requests that share entries keep more than the list has: what does not fit is dropped
    po, io = mla.index_select(scores, pages, torch.tensor([0, 300, 0, 300], dtype=torch.int32, device=DEV), 300)
    assert mla.device_status() == mla.DEV_BAD_INDPTR
    assert po.tolist() == pages.tolist()


@pytest.mark.gpu
def test_other_stream_and_graph():
    lengths = [5000, 3, 700]
    scores, total = _rand(2, sum(lengths)), sum(lengths)
    po, io = _run(scores, lengths, 256)
    pages = torch.randperm(total + 3, generator=torch.Generator().manual_seed(total))[:total].to(torch.int32).to(DEV)
    indptr = torch.tensor([0, 5000, 5003, 5703], dtype=torch.int32, device=DEV)
    s = scores.to(DEV)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(3)]
    for side in sides:
        a = mla.index_select(s, pages, indptr, 256, stream=side)
        side.synchronize()
        assert torch.equal(a[0], po) and torch.equal(a[1], io)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = mla.index_select(s, pages, indptr, 256)
    s.copy_(s.roll(1, 0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[0][256:512], po[:256]) and torch.equal(a[0][:256], po[256:512])


@pytest.mark.gpu
@pytest.mark.parametrize("block,recent", [(1, 0), (32, 1)])
def test_past_32_bits(block, recent):
    # 16 rows of scores past 2^32 bytes, one request at their end
    n, total = 100000, (1 << 27) + 12345
    g = torch.Generator().manual_seed(1)
    mine = torch.randn(16, n, generator=g).clamp(min=0)
    scores = torch.zeros(16, total, device=DEV)
    scores[:, -n:] = mine.to(DEV)
    pages = torch.zeros(total, dtype=torch.int32, device=DEV)
    rows = torch.randperm(n, generator=g).to(torch.int32)
    pages[-n:] = rows.to(DEV)
    po, io = mla.index_select(scores, pages, torch.tensor([total - n, total], dtype=torch.int32, device=DEV), 64, block=block,
                              recent=recent, causal=True)
    lists = _plain(mine, rows, [n], 64, block, recent, 0, True)
    assert io.tolist() == [0] + torch.tensor([x.numel() for x in lists]).cumsum(0).tolist()
    assert po[:io[-1]].tolist() == torch.cat(lists).tolist()
    assert mla.device_status() == 0


@pytest.mark.gpu
def test_many_rows():
    # 2^17 rows of a few tokens: the indptr comes from the scan
    R, qlen = 1 << 13, 16
    lengths = torch.randint(0, 12, (R,), generator=torch.Generator().manual_seed(2)).tolist()
    _run(_rand(qlen, sum(lengths)), lengths, 4, 1, 1, 0, True)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("block", [1, 2, 4, 64, 256])
@pytest.mark.parametrize("lengths,qlen", [
    ([5], 1),
    ([10, 0, 63, 64, 65, 3], 3),
    ([3, 700, 1, 66] * 64, 4),          # 1,024 rows: each cluster counts the rows before its own
    ([3, 700, 1, 66, 9] * 205, 1),      # 1,025: a kernel of its own does
    ([20001], 1),                       # a cluster
    ([9001, 20001, 1] * 60, 1),
])
def test_no_block_stays(lengths, qlen, block, causal):
    # every list is empty, whatever the last block's length; a caller's larger output is -1 throughout
    po = torch.full((777,), 7, dtype=torch.int32, device=DEV)
    po, io = _run(_rand(qlen, sum(lengths)), lengths, 0, block, 1, 2, causal, pages_out=po)
    assert not io.any() and po.eq(-1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 8])
@pytest.mark.parametrize("lengths,qlen", [([9, 0, 2, 40] * 256, 1), ([9, 0, 2, 40, 5] * 205, 1), ([33, 4, 0, 8] * 64, 4)])
def test_rows_around_those_that_every_cluster_counts(lengths, qlen, block):
    # 1,024 rows and 1,025
    _run(_rand(qlen, sum(lengths)), lengths, 3, block, 1, 1, True, pages_out=torch.full((30000,), 7, dtype=torch.int32, device=DEV))


@pytest.mark.gpu
@pytest.mark.parametrize("block,topk", [(1, 700), (64, 12)])
@pytest.mark.parametrize("requests,most", [(256, 20000), (24, 40000), (160, 40000)])
def test_eight_causal_rows_of_a_ragged_batch(requests, most, block, topk):
    # lengths over their logarithm: requests far beyond what the mean gives a block or a cluster, others empty
    u = torch.rand(requests, generator=torch.Generator().manual_seed(requests))
    lengths = torch.exp(u * math.log(most)).long()
    lengths[::31] = 0
    lengths[5] = most
    _run(_rand(8, int(lengths.sum())), lengths.tolist(), topk, block, 2, 1, True)
