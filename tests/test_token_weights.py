"""token_weights: host-side refusals (CPU), then the weight each cached token
received against the formula in 64 bits on the GPU: head layouts, causal
rows, fp8 queries, empty and one-token requests, rows that see nothing,
a pool past 2^31 bytes, bad pages and page lists."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

DEV = "cuda"
A = 1 << 20
B, C, D, E, F, G, H = (A + (i << 28) for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.library()


def _call(lib, **kw):
    a = dict(q=A, qs=12 * 576, kv=B, pool=100, pages=C, n=50, indptr=D, R=2, qlen=1, heads=12, scale=0.1,
             kv_scale=1.0, q_scale=1.0, lse=E, decay=1.0, w=F, out=G, flags=0, ws=None, wsn=0)
    a.update(kw)
    return lib.mla_token_weights(a["q"], a["qs"], a["kv"], a["pool"], a["pages"], a["n"], a["indptr"], a["R"],
                                 a["qlen"], a["heads"], a["scale"], a["kv_scale"], a["q_scale"], a["lse"], a["decay"],
                                 a["w"], a["out"], a["flags"], a["ws"], a["wsn"], None)


@pytest.mark.parametrize("kw,msg", [
    (dict(flags=4), b"flag"),
    (dict(R=-1), b"num_requests"),
    (dict(qlen=0), b"qlen"),
    (dict(qlen=17), b"qlen"),
    (dict(heads=0), b"heads"),
    (dict(heads=129, qs=129 * 576), b"heads"),
    (dict(qs=12 * 576 - 8), b"q_row_stride"),
    (dict(qs=12 * 576 + 4), b"q_row_stride"),
    (dict(qs=12 * 576 + 8, flags=2), b"q_row_stride"),
    (dict(pool=-1), b"negative"),
    (dict(n=-1), b"negative"),
    (dict(scale=float("nan")), b"scale"),
    (dict(kv_scale=float("inf")), b"scale"),
    (dict(q_scale=float("inf")), b"scale"),
    (dict(decay=float("nan")), b"decay"),
    (dict(q=None), b"null"),
    (dict(lse=None), b"null"),
    (dict(w=None), b"null"),
    (dict(out=None), b"null"),
    (dict(q=A + 8), b"misaligned"),
    (dict(kv=B + 4), b"misaligned"),
    (dict(out=G + 2), b"misaligned"),
    (dict(pool=0), b"empty"),
    (dict(out=F + 4), b"overlaps"),
    (dict(scale=1e30, kv_scale=1e30), b"too large"),
    (dict(qlen=16), b"workspace"),
    (dict(qlen=16, ws=H, wsn=100), b"workspace"),
    (dict(qlen=16, ws=H + 8, wsn=1 << 20), b"misaligned workspace"),
    (dict(qlen=16, ws=G, wsn=1 << 20), b"workspace overlaps"),
    (dict(qlen=16, ws=F, wsn=1 << 20), b"workspace overlaps"),
    (dict(qlen=16, ws=B, wsn=1 << 20), b"workspace overlaps"),
    (dict(qs=1 << 61), b"q_row_stride"),
    (dict(out=A + 12 * 576 * 4 - 4), b"out overlaps"),
    (dict(out=B + 99 * 576), b"out overlaps"),
    (dict(out=C), b"out overlaps"),
    (dict(out=D + 8), b"out overlaps"),
    (dict(out=E + 2 * 12 * 4 - 4), b"out overlaps"),
])
def test_refusals(lib, kw, msg):
    assert _call(lib, **kw) == mla.MLA_ERR_INVALID
    assert msg in lib.mla_last_error()


def test_unsupported_sizes_and_nothing_to_do(lib):
    assert _call(lib, pool=1 << 31) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, n=1 << 31) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, R=0) == mla.MLA_OK
    assert _call(lib, n=0, pages=None) == mla.MLA_OK


def test_workspace(lib):
    assert mla.token_weights_workspace(1, 12, 1000) == 0
    assert mla.token_weights_workspace(1, 128, 1000, True) == 0
    assert mla.token_weights_workspace(1, 128, 1000) == 0
    assert mla.token_weights_workspace(2, 96, 1000) > 0
    with pytest.raises(mla.MlaError, match="qlen"):
        mla.token_weights_workspace(17, 12, 1000)


def test_binding_refusals():
    q = torch.zeros(2, 4, 576, dtype=torch.bfloat16)
    kv = torch.zeros(8, 576, dtype=torch.uint8)
    p, i = torch.zeros(5, dtype=torch.int32), torch.tensor([0, 2, 5], dtype=torch.int32)
    lse = torch.zeros(2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        mla.token_weights(q, kv, p, i, 0.1, 1.0, lse)
    with pytest.raises(ValueError, match="lse"):
        mla.token_weights(q, kv, p, i, 0.1, 1.0, lse[:, :3])


# ------------------------------------------------------------------- GPU


def _make(lengths, qlen, heads, pad, seed, q8=False, std=0.5, qstd=1.0, extra=5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    total, R = sum(lengths), len(lengths)
    pool = total + extra
    pages = torch.randperm(pool, generator=g, device=DEV)[:total].to(torch.int32)
    kv = torch.randn(pool, 576, generator=g, device=DEV).mul_(std).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn(R * qlen, pad, 576, generator=g, device=DEV).mul_(qstd)
    q = q.to(torch.float8_e4m3fn) if q8 else q.to(torch.bfloat16)
    if pad > heads:
        q[:, heads:] = float("nan")
    indptr = torch.zeros(R + 1, dtype=torch.int32)
    indptr[1:] = torch.tensor(lengths, dtype=torch.int32).cumsum(0)
    return q, kv, pages, indptr.to(DEV)


def _formula(q, kv, pages, lengths, heads, qlen, sc, causal, lse=None):
    """New weights per token in 64 bits, a bound of the kernel's error, and the LSE (made here if not given).

    A score is a float32 accumulation of 18 tensor-core steps of 32 products for each of the query's two 8-bit
    terms: under 64 roundings of the sum of magnitudes.  The two terms hold q to 2^-21 of the row's largest element
    (exactly where it is not that small).  Scale, LSE and exponential add 8 roundings of their magnitudes; the sum over
    rows has one rounding a row."""
    out, bound, at, lses = [], [], 0, []
    for r, n in enumerate(lengths):
        k = kv[pages[at:at + n].long()].view(torch.float8_e4m3fn).double()
        qq = q[r * qlen:(r + 1) * qlen, :heads].double().reshape(-1, 576)
        s = qq @ k.T * sc
        if causal:
            t = torch.arange(qlen, device=DEV).repeat_interleave(heads)[:, None]
            s = s.masked_fill(torch.arange(n, device=DEV)[None] >= n - qlen + t + 1, -math.inf)
        if lse is None:
            ls = torch.logsumexp(s, 1).float() if n else torch.full((qlen * heads,), -math.inf, device=DEV)
            lses.append(ls)
        else:
            ls = lse.view(-1, qlen * heads)[r]
        l64 = ls.double()[:, None]
        p = torch.where(l64 == -math.inf, torch.zeros_like(s), torch.exp(s - l64))
        mag = abs(sc) * (qq.abs() @ k.abs().T)
        split = abs(sc) * qq.abs().amax(1, keepdim=True) * k.abs().sum(1)[None] * 2.0**-21
        x = torch.where(p > 0, s - l64, torch.zeros_like(s))
        big = torch.where(p > 0, s.abs() + l64.abs(), torch.zeros_like(s))
        delta = 64 * 2.0**-24 * mag + split + 8 * 2.0**-24 * (x.abs() + big + 1)
        out.append(p.sum(0))
        bound.append((p * (torch.expm1(delta) + p.shape[0] * 2.0**-24)).sum(0))
        at += n
    z = torch.zeros(0, dtype=torch.float64, device=DEV)
    return torch.cat(out + [z]), torch.cat(bound + [z]), torch.cat(lses).view(-1, heads) if lses else lse


def _check(got, want, bound, what=""):
    assert got.isfinite().all()
    bad = (got.double() - want).abs() > bound + 2.0**-24 * want.abs() + 2.0**-149
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        what, int(bad.sum()), bad.numel(), float(((got.double() - want).abs() / (bound + 1e-300)).max()))


SHAPES = [
    # lengths, qlen, heads, padded heads
    ([64, 100], 1, 12, 12),
    ([1], 1, 1, 1),
    ([1, 0, 2, 127, 128, 129, 0], 1, 12, 12),
    ([300, 5, 1000], 4, 12, 12),
    ([257], 8, 12, 16),
    ([513, 31], 1, 96, 128),
    ([200, 140], 2, 128, 128),
    ([150], 16, 128, 128),
    ([77, 300], 3, 5, 8),
    ([4000, 4], 1, 24, 24),
    ([1500], 1, 40, 40),
]


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lengths,qlen,heads,pad", SHAPES)
def test_against_the_formula(lengths, qlen, heads, pad, q8, causal):
    q, kv, pages, indptr = _make(lengths, qlen, heads, pad, 17 * heads + qlen, q8)
    scale, kv_scale, q_scale = 0.0721, 0.8, 0.9 if q8 else 1.0
    want, bound, lse = _formula(q, kv, pages, lengths, heads, qlen, scale * kv_scale * q_scale, causal)
    lse = lse.contiguous()
    args = (q, kv, pages, indptr, scale, kv_scale, lse)
    kw = dict(heads=heads, qlen=qlen, causal=causal, q_scale=q_scale)
    got = mla.token_weights(*args, **kw)
    _check(got, want, bound, "new weights")
    # a request's new weights sum to its rows that see a token
    old = torch.rand(got.numel(), device=DEV)
    out = mla.token_weights(*args, weights=old, decay=0.75, **kw)
    _check(out, want + 0.75 * old.double(), bound + 2.0**-23 * (want + old.double()), "accumulated")
    keep = old.clone()
    assert mla.token_weights(*args, weights=keep, decay=0.75, out=keep, **kw) is keep
    assert torch.equal(keep, out)
    nan = torch.full_like(old, float("nan"))
    assert torch.equal(mla.token_weights(*args, weights=nan, decay=0.0, **kw), got)
    assert mla.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("qstd,std", [(6.0, 2.0), (1.0, 20.0), (1e-3, 0.5)])
def test_peaked_and_flat_scores(qstd, std):
    lengths = [700, 40]
    q, kv, pages, indptr = _make(lengths, 2, 12, 12, 5, qstd=qstd, std=std)
    want, bound, lse = _formula(q, kv, pages, lengths, 12, 2, 0.05, False)
    got = mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse.contiguous(), qlen=2)
    _check(got, want, bound)


@pytest.mark.gpu
def test_outlier_channels_and_row_magnitudes():
    lengths = [400, 3]
    q, kv, pages, indptr = _make(lengths, 1, 24, 24, 6)
    q[:, ::2] *= 1e-6
    q[:, 1::4] *= 30000
    q[:, :, 7] *= 64
    q[:, 3] = 0
    sc = 1e-5
    want, bound, lse = _formula(q, kv, pages, lengths, 24, 1, sc, False)
    got = mla.token_weights(q, kv, pages, indptr, sc, 1.0, lse.contiguous())
    _check(got, want, bound)


@pytest.mark.gpu
def test_rows_without_lse_and_foreign_lse():
    lengths = [130, 9]
    q, kv, pages, indptr = _make(lengths, 2, 12, 12, 7)
    _, _, lse = _formula(q, kv, pages, lengths, 12, 2, 0.05, False)
    lse = lse.clone()
    lse[0, 3] = -math.inf            # an empty row gives nothing
    lse[1, :] = -math.inf
    lse[2] += 3.0                    # the LSE of a longer context (other ranks' tokens)
    lse[3, 0] = math.inf
    want, bound, _ = _formula(q, kv, pages, lengths, 12, 2, 0.05, False, lse)
    got = mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse, qlen=2)
    _check(got, want, bound)


@pytest.mark.gpu
def test_query_rows_in_a_wider_buffer_and_negative_scale():
    lengths = [90, 200]
    q, kv, pages, indptr = _make(lengths, 1, 12, 12, 8)
    wide = torch.full((2, 20, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:20] = q
    view = wide[:, 8:20]
    want, bound, lse = _formula(q, kv, pages, lengths, 12, 1, -0.05, False)
    got = mla.token_weights(view, kv, pages, indptr, -0.05, 1.0, lse.contiguous())
    _check(got, want, bound)


@pytest.mark.gpu
def test_entries_past_the_last_request_stay():
    q, kv, pages, indptr = _make([60, 70], 1, 12, 12, 9)
    _, _, lse = _formula(q, kv, pages, [60, 70], 12, 1, 0.05, False)
    more = torch.cat([pages, torch.full((9,), -1, dtype=torch.int32, device=DEV)])
    out = torch.full((139,), -7.0, device=DEV)
    mla.token_weights(q, kv, more, indptr, 0.05, 1.0, lse.contiguous(), out=out)
    assert (out[130:] == -7).all() and (out[:130] > 0).all()
    assert mla.device_status() == 0


@pytest.mark.gpu
def test_pool_past_2_31_bytes():
    rows = 4_000_000                 # 2.3 GB
    kv = torch.zeros(rows, 576, dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    pages = torch.cat([torch.arange(rows - 150, rows, device=DEV), torch.arange(0, 100, device=DEV)]).to(torch.int32)
    kv[pages.long()] = torch.randn(250, 576, generator=g, device=DEV).mul_(0.5).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn(2, 12, 576, generator=g, device=DEV).to(torch.bfloat16)
    indptr = torch.tensor([0, 149, 250], dtype=torch.int32, device=DEV)
    want, bound, lse = _formula(q, kv, pages, [149, 101], 12, 1, 0.05, False)
    _check(mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse.contiguous()), want, bound)


@pytest.mark.gpu
def test_bad_pages_and_bad_page_lists_are_flagged():
    lengths = [200, 100, 50]
    q, kv, pages, indptr = _make(lengths, 1, 12, 12, 10)
    want, bound, lse = _formula(q, kv, pages, lengths, 12, 1, 0.05, False)
    lse = lse.contiguous()
    bad = pages.clone()
    bad[3], bad[130], bad[220], bad[221] = -1, kv.shape[0], 2**31 - 1, -2**31
    fixed = pages.clone()
    fixed[3] = fixed[130] = fixed[220] = fixed[221] = 0
    got = mla.token_weights(q, kv, bad, indptr, 0.05, 1.0, lse)
    assert mla.device_status() == mla.DEV_BAD_PAGE
    assert torch.equal(got, mla.token_weights(q, kv, fixed, indptr, 0.05, 1.0, lse))     # read as row 0
    for ind in ([0, 200, 100, 350], [0, 200, 900, 350], [0, -4, 300, 350]):
        out = torch.full((350 + 64,), -7.0, device=DEV)
        mla.token_weights(q, kv, pages, torch.tensor(ind, dtype=torch.int32, device=DEV), 0.05, 1.0, lse,
                          out=out[:350])
        assert mla.device_status() == mla.DEV_BAD_INDPTR
        assert (out[350:] == -7).all()


@pytest.mark.gpu
def test_page_list_named_again_and_again():
    # every other entry of indptr goes back to 0: the requests in between are bad, the others all tokens each,
    # thousands of times the list's tiles
    q, kv, pages, indptr = _make([300], 1, 12, 12, 10)
    _, _, lse = _formula(q, kv, pages, [300], 12, 1, 0.05, False)
    R = 3001
    ind = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
    ind[1::2] = 300
    out = torch.full((300 + 64,), -7.0, device=DEV)
    mla.token_weights(q.expand(R, -1, -1).contiguous(), kv, pages, ind, 0.05, 1.0, lse.expand(R, -1).contiguous(),
                      out=out[:300])
    assert mla.device_status() == mla.DEV_BAD_INDPTR
    assert (out[300:] == -7).all()


@pytest.mark.gpu
def test_many_requests_of_all_lengths():
    # more requests than threads of a CTA, most of one tile or none: every CTA changes requests at every tile
    lengths = [(i * 37) % 150 if i % 5 else 0 for i in range(1500)] + [0] * 700 + [260]
    for heads in (4, 70):
        q, kv, pages, indptr = _make(lengths, 1, heads, heads, 12)
        want, bound, lse = _formula(q, kv, pages, lengths, heads, 1, 0.05, False)
        _check(mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse.contiguous()), want, bound)
    assert mla.device_status() == 0


@pytest.mark.gpu
def test_given_workspace_and_overlapping_calls():
    lengths = [900, 300]
    q, kv, pages, indptr = _make(lengths, 2, 96, 96, 13)
    _, _, lse = _formula(q, kv, pages, lengths, 96, 2, 0.05, False)
    args, kw = (q, kv, pages, indptr, 0.05, 1.0, lse.contiguous()), dict(qlen=2)
    want = mla.token_weights(*args, **kw)
    ws = torch.empty(mla.token_weights_workspace(2, 96, 1200), dtype=torch.uint8, device=DEV)
    assert torch.equal(mla.token_weights(*args, workspace=ws, **kw), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [mla.token_weights(*args, stream=s, **kw) for s in (side, None, side, None)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.gpu
def test_same_bits_again_on_a_stream_and_in_a_graph():
    lengths = [3000, 1, 777, 0, 5000]
    q, kv, pages, indptr = _make(lengths, 2, 12, 12, 11)
    _, _, lse = _formula(q, kv, pages, lengths, 12, 2, 0.05, True)
    lse = lse.contiguous()
    kw = dict(qlen=2, causal=True)
    first = mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse, stream=side, **kw)
    side.synchronize()
    assert torch.equal(first, again)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse, **kw)
    g.replay()
    assert torch.equal(out, first)
    q.mul_(0.5)
    g.replay()
    assert torch.equal(out, mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("qlen,heads,q8", [(1, 12, False), (3, 43, False), (3, 43, True)])
def test_the_longest_page_list(qlen, heads, q8):
    # one request of as many tokens as are accepted, over and over the same 64 rows: in one pass (12 query rows) and as
    # groups' partial sums joined by a second kernel (129).  Every token's sum is its own, so equal rows give equal bits.
    n = 2**31 - 65536
    need = 4 * n * 2 + mla.token_weights_workspace(qlen, heads, n, q8) + (8 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("%d GB of device memory free" % (need >> 30))
    q, kv, _, _ = _make([64], qlen, heads, heads, 21, q8)
    head = torch.arange(64, dtype=torch.int32, device=DEV)
    want, bound, lse = _formula(q, kv, head, [64], heads, qlen, 0.05, False)
    pages = head.repeat(n // 64)
    indptr = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out = mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse.contiguous(), heads=heads, qlen=qlen)
    assert mla.device_status() == 0
    del pages
    _check(out[:64], want, bound)
    rows = out.view(-1, 64).view(torch.int32)
    for part in rows.split(1 << 22):
        assert bool((part == rows[0]).all())
    with pytest.raises(mla.MlaError, match="2\\^31 - 65536"):
        mla.token_weights_workspace(qlen, heads, n + 1, q8)
    del out, rows, part
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [12, 70])
@pytest.mark.parametrize("qlen", [1, 3])
def test_a_list_that_starts_past_its_first_entries(qlen, heads):
    lengths, skip = [60, 0, 170], 37
    q, kv, pages, indptr = _make(lengths, qlen, heads, heads, 9)
    want, bound, lse = _formula(q, kv, pages, lengths, heads, qlen, 0.05, False)
    more = torch.cat([torch.full((skip,), -1, dtype=torch.int32, device=DEV), pages,
                      torch.full((9,), -1, dtype=torch.int32, device=DEV)])
    out = torch.full((more.numel(),), -7.0, device=DEV)
    mla.token_weights(q, kv, more, indptr + skip, 0.05, 1.0, lse.contiguous(), qlen=qlen, out=out)
    assert (out[:skip] == -7).all() and (out[skip + 230:] == -7).all()
    _check(out[skip:skip + 230], want, bound)
    assert mla.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("R,heads", [(1 << 22, 1), (20001, 80)])
def test_many_empty_requests_between_two_tiles_of_a_block(R, heads):
    # the tiles of the first and of the last request meet inside one CTA (or pair), whose roles each pass over all the
    # empty requests between them; none may give up on another meanwhile
    first, last = 128 * 151, 128 * 153
    g = torch.Generator(device=DEV).manual_seed(R)
    kv = torch.randn(64, 576, generator=g, device=DEV).mul_(0.5).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.zeros(R, heads, 576, dtype=torch.bfloat16, device=DEV)
    q[0], q[-1] = (torch.randn(heads, 576, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    indptr = torch.full((R + 1,), first, dtype=torch.int32, device=DEV)
    indptr[0], indptr[-1] = 0, first + last
    pages = torch.arange(64, dtype=torch.int32, device=DEV).repeat((first + last) // 64)
    lse = torch.zeros(R, heads, device=DEV)
    out = mla.token_weights(q, kv, pages, indptr, 0.05, 1.0, lse)
    assert mla.device_status() == 0
    want, bound, _ = _formula(q[[0, -1]], kv, pages[:128], [64, 64], heads, 1, 0.05, False, lse[:2])
    _check(out, torch.cat([want[:64].repeat(first // 64), want[64:].repeat(last // 64)]),
           torch.cat([bound[:64].repeat(first // 64), bound[64:].repeat(last // 64)]))


@pytest.mark.gpu
def test_the_longest_list_named_again_and_again():
    # 150 requests that each name nearly all of the longest list, a bad one between any two: 2.5e9 tiles claimed.
    # Flagged, ended by what the list could hold, and nothing outside it written.
    n = 2**31 - 65536
    if torch.cuda.mem_get_info()[0] < 4 * n * 2 + (8 << 30):
        pytest.skip("%d GB of device memory free" % ((4 * n * 2 >> 30) + 8))
    R = 299
    ind = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
    ind[1::2] = n
    q, kv, _, _ = _make([64], 1, 1, 1, 22)
    pages = torch.arange(64, dtype=torch.int32, device=DEV).repeat(n // 64)
    buf = torch.full((n + 64,), -7.0, device=DEV)
    mla.token_weights(q.expand(R, -1, -1).contiguous(), kv, pages, ind, 0.05, 1.0, torch.zeros(R, 1, device=DEV), out=buf[:n])
    assert mla.device_status() == mla.DEV_BAD_INDPTR
    assert bool((buf[n:] == -7).all())
    del pages, buf
    torch.cuda.empty_cache()
