"""index_scores: host-side refusals (CPU), then every token's score against
the formula in 64 bits on the GPU: head and row counts around a group of
columns, lengths around a tile, masks, empty requests, bad pages."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

DEV = "cuda"
A = 1 << 20
B, C, D, E, F, G = (A + (i << 34) for i in range(1, 7))
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.library()


def _call(lib, **kw):
    a = dict(q=A, w=B, qs=None, k=C, pool=50, pages=D, n=100, indptr=E, R=3, qlen=2, heads=4, scale=1.0, out=F, flags=0)
    a.update(kw)
    return lib.mla_index_scores(a["q"], a["w"], a["qs"], a["k"], a["pool"], a["pages"], a["n"], a["indptr"], a["R"],
                                a["qlen"], a["heads"], a["scale"], a["out"], a["flags"], None)


@pytest.mark.parametrize("kw,msg", [
    (dict(flags=2), b"flag"),
    (dict(R=-1), b"negative"),
    (dict(n=-1), b"negative"),
    (dict(pool=-1), b"negative"),
    (dict(qlen=0), b"qlen"),
    (dict(qlen=17), b"qlen"),
    (dict(heads=0), b"heads"),
    (dict(heads=129), b"heads"),
    (dict(scale=math.inf), b"scale"),
    (dict(q=None), b"null"),
    (dict(w=None), b"null"),
    (dict(k=None), b"null"),
    (dict(pages=None), b"null"),
    (dict(indptr=None), b"null"),
    (dict(out=None), b"null"),
    (dict(q=A + 8), b"misaligned"),
    (dict(k=C + 8), b"misaligned"),
    (dict(qs=G + 2), b"misaligned"),
    (dict(pool=0), b"empty"),
    (dict(out=A + 3068), b"overlaps"),
    (dict(out=B + 92), b"overlaps"),
    (dict(out=C - 796), b"overlaps"),
    (dict(out=D), b"overlaps"),
    (dict(out=E + 12), b"overlaps"),
    (dict(qs=G, out=G), b"overlaps"),
])
def test_refusals(lib, kw, msg):
    assert _call(lib, **kw) == mla.MLA_ERR_INVALID
    assert msg in lib.mla_last_error()


@pytest.mark.parametrize("kw", [dict(pool=1 << 31), dict(n=1 << 31), dict(R=(1 << 24) + 1, qlen=1),
                                dict(R=1 << 24, qlen=1, heads=128)])
def test_too_large(lib, kw):
    assert _call(lib, **kw) == mla.MLA_ERR_UNSUPPORTED


def test_empty(lib):
    assert _call(lib, R=0, q=None, out=None) == mla.MLA_OK
    assert _call(lib, n=0, q=None, out=None) == mla.MLA_OK


def test_binding_refusals():
    mla.build()
    q, w = torch.zeros(4, 2, 128, dtype=torch.uint8), torch.zeros(4, 2)
    k, p, i = torch.zeros(9, 128, dtype=torch.uint8), torch.zeros(5, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    for args, kw, msg in [
        ((q.float(), w, k, p, i), {}, "e4m3"), ((q[:, 0], w, k, p, i), {}, "e4m3"), ((q[..., :64], w, k, p, i), {}, "q must"),
        ((q, w[:2], k, p, i), {}, "weights"), ((q, w.half(), k, p, i), {}, "weights"), ((q, w, k.float(), p, i), {}, "k must"),
        ((q, w, k[:, :64], p, i), {}, "k must"), ((q, w, k, p.long(), i), {}, "pages"), ((q, w, k, p, i), dict(qlen=2), "indptr"),
        ((q, w, k, p, i), dict(q_scales=w[0]), "q_scales"), ((q, w, k, p, i), {}, "CUDA"),
    ]:
        with pytest.raises(ValueError, match=msg):
            mla.index_scores(*args, **kw)


# ------------------------------------------------------------------- GPU


def _indptr(lengths):
    return torch.tensor([0] + list(torch.tensor(lengths, dtype=torch.int64).cumsum(0)), dtype=torch.int32).to(DEV)


def _inputs(lengths, qlen, heads, seed=0, scales=True):
    total, S = sum(lengths), len(lengths) * qlen
    g = torch.Generator().manual_seed(seed + total + heads)
    q = torch.randn(S, heads, 128, generator=g).mul(60).clamp(-448, 448).to(E4M3).to(DEV)
    k = torch.randn(total + 9, 128, generator=g).mul(5).to(E4M3).to(DEV)
    w = torch.randn(S, heads, generator=g).to(DEV)
    qs = torch.rand(S, heads, generator=g).add(0.1).to(DEV) if scales else None
    pages = torch.randperm(total + 9, generator=g)[:total].to(torch.int32).to(DEV)
    return q, w, qs, k, pages, _indptr(lengths)


def _plain(q, w, qs, k, pages, lengths, qlen, scale, causal):
    """Scores in 64 bits, and the sums of the terms' magnitudes."""
    out = torch.full((qlen, pages.numel()), math.nan, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(out)
    at = 0
    w = w.double() if qs is None else w.double() * qs.double()
    kd = k.view(E4M3).double()
    for r, n in enumerate(lengths):
        rows = kd[pages[at:at + n].long()]
        for tq in range(qlen):
            t = r * qlen + tq
            qt = q.view(E4M3)[t].double()
            out[tq, at:at + n] = scale * (torch.relu(rows @ qt.T) @ w[t])
            mag[tq, at:at + n] = abs(scale) * ((rows.abs() @ qt.abs().T) @ w[t].abs())
            if causal:
                out[tq, at + max(0, n - qlen + tq + 1):at + n] = -math.inf
        at += n
    return out, mag


def _check(got, want, mag):
    """Off by less than 2^-16 of the magnitudes' sum: the products are exact, their sums of 128 and then of up to 128
    heads in float32 add (128 + 128) x 2^-24 of it, the weights' two products 2^-22."""
    got = got.double()
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got.isnan(), want.isnan())
    fine = want.isfinite()
    assert torch.all((got - want).abs()[fine] <= mag[fine] * 2.0 ** -16)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,qlen,heads,causal", [
    ([1], 1, 1, False),
    ([1], 16, 128, True),
    ([127, 128, 129], 1, 64, False),
    ([0, 0, 5, 0, 300, 0], 1, 32, False),
    ([0], 2, 8, False),
    ([3, 1000, 2], 4, 16, True),
    ([3, 1000, 2], 4, 17, True),
    ([400] * 30, 2, 48, True),
    ([257, 511], 8, 12, True),
    ([257, 511], 3, 96, False),
    ([257, 511], 5, 127, True),
    ([2000], 16, 15, True),
    ([2000], 16, 33, True),
    ([1] * 500, 1, 64, False),
    ([7, 0] * 400, 2, 24, True),
    ([20000, 3, 9000], 1, 64, False),
    (list(range(0, 700, 3)), 1, 128, False),
    ([130] * 700, 1, 4, False),
])
def test_scores(lengths, qlen, heads, causal):
    q, w, qs, k, pages, indptr = _inputs(lengths, qlen, heads, scales=heads % 2 == 0)
    got = mla.index_scores(q, w, k, pages, indptr, q_scales=qs, scale=0.3, qlen=qlen, causal=causal)
    assert got.shape == (qlen, sum(lengths)) and got.dtype == torch.float32
    _check(got, *_plain(q, w, qs, k, pages, lengths, qlen, 0.3, causal))
    assert mla.device_status() == 0
    again = mla.index_scores(q.view(torch.uint8), w, k.view(torch.uint8), pages, indptr, q_scales=qs, scale=0.3, qlen=qlen,
                             causal=causal)
    assert torch.equal(got.view(torch.int32), again.view(torch.int32))


@pytest.mark.gpu
def test_largest_and_special_values():
    # the largest codes: 128 x 448^2 and every head's weight; negative and zero weights
    q, w, _, k, pages, indptr = _inputs([300, 10], 1, 64)
    q.view(torch.uint8)[0] = 0x7E
    k.view(torch.uint8)[pages[3].item()] = 0x7E
    k.view(torch.uint8)[pages[4].item()] = 0xFE
    w[1] = -w[1].abs()
    w[0, :9] = 0
    got = mla.index_scores(q, w, k, pages, indptr)
    _check(got, *_plain(q, w, None, k, pages, [300, 10], 1, 1.0, False))
    assert got[0, 4] == 0
    # NaN codes reach their own token's score (of a key) or their own row's scores (of a query)
    k.view(torch.uint8)[pages[7].item(), 5] = 0x7F
    q.view(torch.uint8)[1, 3, 0] = 0xFF
    bad = mla.index_scores(q, w, k, pages, indptr)
    assert bad[0, 7].isnan() and bad[0, 300:].isnan().all()
    keep = torch.arange(300, device=DEV) != 7
    assert torch.equal(bad[0, :300][keep], got[0, :300][keep])


@pytest.mark.gpu
def test_padding_columns_hold_no_garbage():
    # 5 heads of 16 columns and 3 rows of 4: the rest of the operand must not keep NaN codes of an earlier call
    q, w, qs, k, pages, indptr = _inputs([500, 60], 4, 128)
    q.view(torch.uint8)[:] = 0x7F
    mla.index_scores(q, w, k, pages, indptr, qlen=4)
    q, w, qs, k, pages, indptr = _inputs([500, 60], 3, 5)
    got = mla.index_scores(q, w, k, pages, indptr, q_scales=qs, qlen=3)
    _check(got, *_plain(q, w, qs, k, pages, [500, 60], 3, 1.0, False))


@pytest.mark.gpu
def test_entries_of_no_request_are_left():
    q, w, qs, k, pages, indptr = _inputs([5, 200, 20, 30], 2, 64)
    out = torch.full((2, 255), 7.0, device=DEV)
    mla.index_scores(q[2:6], w[2:6], k, pages, indptr[1:4].contiguous(), qlen=2, out=out)
    want, mag = _plain(q[2:6], w[2:6], None, k, pages[5:225], [200, 20], 2, 1.0, False)
    _check(out[:, 5:225], want, mag)
    assert out[:, :5].eq(7).all() and out[:, 225:].eq(7).all()


@pytest.mark.gpu
def test_bad_pages_and_indptr_are_flagged():
    q, w, qs, k, pages, indptr = _inputs([200, 100], 1, 32)
    pages[10], pages[250] = -3, k.shape[0]
    got = mla.index_scores(q, w, k, pages, indptr)
    assert mla.device_status() == mla.DEV_BAD_PAGE
    pages[10] = pages[250] = 0
    _check(got, *_plain(q, w, None, k, pages, [200, 100], 1, 1.0, False))
    bad = indptr.clone()
    bad[1] = 400                        # past the list, and past the next request's end
    out = torch.full((1, 300), 7.0, device=DEV)
    mla.index_scores(q, w, k, pages, bad, out=out)
    assert mla.device_status() == mla.DEV_BAD_INDPTR
    assert out.eq(7).all()


@pytest.mark.gpu
def test_other_stream_graph_and_two_at_once():
    q, w, qs, k, pages, indptr = _inputs([3000, 50, 700], 2, 64)
    want = mla.index_scores(q, w, k, pages, indptr, qlen=2, causal=True)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(3)]
    got = [mla.index_scores(q, w, k, pages, indptr, qlen=2, causal=True, stream=s) for s in sides]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = mla.index_scores(q, w, k, pages, indptr, qlen=2, causal=True)
    w.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b, want * 2)


@pytest.mark.gpu
def test_past_32_bits():
    # rows of the index cache and of the output past 2^32 bytes
    n, pool = 1 << 16, (1 << 25) + 5000
    k = torch.zeros(pool, 128, dtype=torch.uint8, device=DEV)
    g = torch.Generator(DEV).manual_seed(1)
    k[-4000:] = torch.randn(4000, 128, device=DEV, generator=g).mul(5).to(E4M3).view(torch.uint8)
    q = torch.randn(16, 8, 128, device=DEV, generator=g).mul(60).clamp(-448, 448).to(E4M3)
    w = torch.randn(16, 8, device=DEV, generator=g)
    total = (1 << 26) + n + 3                           # x 16 rows x 4 bytes: past 2^32
    pages = torch.zeros(total, dtype=torch.int32, device=DEV)
    pages[-n:] = torch.randint(pool - 4000, pool, (n,), device=DEV, generator=g).to(torch.int32)
    indptr = torch.tensor([total - n, total], dtype=torch.int32, device=DEV)
    out = mla.index_scores(q, w, k, pages, indptr, qlen=16, causal=True)
    some = torch.randint(0, n, (2000,), generator=torch.Generator().manual_seed(4)).to(DEV)
    some[:40] = torch.arange(n - 40, n, device=DEV)
    rows = k[pages[-n:][some].long()].view(E4M3).double()
    for tq in (0, 7, 15):
        want = torch.relu(rows @ q[tq].double().T) @ w[tq].double()
        mag = (rows.abs() @ q[tq].double().abs().T) @ w[tq].double().abs()
        want[some >= n - 16 + tq + 1] = -math.inf
        _check(out[tq, -n:][some], want, mag)
    assert mla.device_status() == 0


def _spread(requests, most, seed):
    """Lengths spread over the logarithm of 1 to `most`, some requests empty."""
    u = torch.rand(requests, generator=torch.Generator().manual_seed(seed))
    n = torch.exp(u * math.log(most)).long()
    n[::31] = 0
    return n.tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [12, 64])
def test_eight_causal_rows_of_a_ragged_batch(heads):
    # 512 columns a request with 64 heads: two groups of rows
    lengths = _spread(256, 6000, heads)
    q, w, qs, k, pages, indptr = _inputs(lengths, 8, heads)
    got = mla.index_scores(q, w, k, pages, indptr, q_scales=qs, scale=0.3, qlen=8, causal=True)
    _check(got, *_plain(q, w, qs, k, pages, lengths, 8, 0.3, True))
    assert mla.device_status() == 0
