"""kv_evict: host-side refusals (CPU), then the kept and freed tokens of
every request against a plain selection on the GPU: ties, NaN and infinite
weights, empty and one-token requests, budgets of every kind."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

DEV = "cuda"
A = 1 << 20
B, C, D, E, F = (A + (i << 28) for i in range(1, 6))


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.library()


def _call(lib, **kw):
    a = dict(pages=A, n=100, indptr=B, R=3, w=C, budgets=None, budget=10, recent=1, sinks=1, po=D, io=E, wo=F)
    a.update(kw)
    return lib.mla_kv_evict(a["pages"], a["n"], a["indptr"], a["R"], a["w"], a["budgets"], a["budget"], a["recent"],
                            a["sinks"], a["po"], a["io"], a["wo"], None)


@pytest.mark.parametrize("kw,msg", [
    (dict(R=-1), b"negative"),
    (dict(n=-1), b"negative"),
    (dict(recent=-1), b"negative"),
    (dict(sinks=-1), b"negative"),
    (dict(indptr=None), b"null"),
    (dict(io=None), b"null"),
    (dict(pages=None), b"null"),
    (dict(w=None), b"null"),
    (dict(po=None), b"null"),
    (dict(wo=None), b"null"),
    (dict(w=C + 2), b"misaligned"),
    (dict(budgets=C + 401), b"misaligned"),
    (dict(po=A), b"overlaps"),
    (dict(wo=C + 396), b"overlaps"),
    (dict(io=B + 4), b"overlaps"),
    (dict(budgets=D + 396), b"overlaps"),
    (dict(wo=D + 100), b"two outputs"),
])
def test_refusals(lib, kw, msg):
    assert _call(lib, **kw) == mla.MLA_ERR_INVALID
    assert msg in lib.mla_last_error()


def test_too_many_pages(lib):
    assert _call(lib, n=1 << 31) == mla.MLA_ERR_UNSUPPORTED


def test_binding_refusals():
    p, i = torch.zeros(4, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    w = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        mla.kv_evict(p, i, w, 2)
    with pytest.raises(ValueError, match="weights"):
        mla.kv_evict(p, i, w[:3], 2)
    with pytest.raises(ValueError, match="budget"):
        mla.kv_evict(p, i, w, torch.tensor([1, 2], dtype=torch.int32))


# ------------------------------------------------------------------- GPU


def _plain(pages, lengths, weights, budgets, recent, sinks):
    """Kept rows, freed rows, kept counts and kept weights by the definition, on the host."""
    at, kept, freed, counts, kw = 0, [], [], [], []
    for n, b in zip(lengths, budgets):
        p, w = pages[at:at + n], weights[at:at + n]
        at += n
        keep = min(n, max(b, 0))
        rec = min(recent, keep)
        snk = min(sinks, keep - rec)
        mid = list(range(snk, n - rec))
        key = [(-math.inf if math.isnan(w[i]) else w[i]) for i in mid]
        best = sorted(range(len(mid)), key=lambda j: (-key[j], mid[j]))[:keep - rec - snk]
        chosen = set(range(snk)) | set(range(n - rec, n)) | {mid[j] for j in best}
        kept += [p[i] for i in range(n) if i in chosen]
        kw += [w[i] for i in range(n) if i in chosen]
        freed += [p[i] for i in range(n) if i not in chosen]
        counts.append(keep)
    return kept, freed, counts, kw


def _run(lengths, weights, budget, recent=0, sinks=0, tail=0, **kw):
    total = sum(lengths)
    g = torch.Generator().manual_seed(total + recent)
    pages = torch.randperm(total + tail + 3, generator=g)[:total + tail].to(torch.int32)
    indptr = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32) if lengths else \
        torch.zeros(1, dtype=torch.int32)
    budgets = budget.tolist() if isinstance(budget, torch.Tensor) else [budget] * len(lengths)
    dev = budget.to(DEV) if isinstance(budget, torch.Tensor) else budget
    po = torch.full((total + tail,), -7, dtype=torch.int32, device=DEV)
    wo = torch.full((total + tail,), -7.0, device=DEV)
    w = torch.cat([weights, torch.full((tail,), 9.0)])
    _, io, _ = mla.kv_evict(pages.to(DEV), indptr.to(DEV), w.to(DEV), dev, recent=recent, sinks=sinks, pages_out=po,
                            weights_out=wo, **kw)
    kept, freed, counts, kw_ = _plain(pages.tolist(), lengths, weights.tolist(), budgets, recent, sinks)
    assert io.tolist() == [0] + torch.tensor(counts, dtype=torch.int64).cumsum(0).tolist()
    assert po.tolist() == kept + freed + [-7] * tail
    got = wo.cpu()
    want = torch.cat([torch.tensor(kw_, dtype=torch.float32), torch.zeros(len(freed)), torch.full((tail,), -7.0)])
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    assert mla.device_status() == 0


def _rand(n, seed):
    return torch.randn(n, generator=torch.Generator().manual_seed(seed)).mul(2).exp()


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,budget,recent,sinks", [
    ([1], 0, 0, 0),
    ([1], 1, 0, 0),
    ([1], 5, 3, 2),
    ([2, 0, 3], 2, 1, 1),
    ([10, 20], -3, 4, 4),
    ([100], 7, 0, 0),
    ([100], 7, 20, 0),          # recent above the budget
    ([100], 7, 3, 20),          # sinks take the rest
    ([1023, 1024, 1025], 1024, 10, 2),
    ([5000, 31, 0, 0, 2049, 4097], 700, 64, 4),
    ([5000, 31, 2049], 5000, 64, 4),
    ([40000], 39999, 1, 1),     # one token goes
    ([40000], 1, 0, 0),
    ([70001, 3, 131072], 8192, 512, 4),
    ([300000], 1000, 100, 4),
    ([8192, 8193, 8191, 0, 16385, 9000], 4000, 100, 4),
    ([9000] * 12 + [100] * 300 + [50000, 20000], 4096, 64, 2),      # long requests with a part to select and without
    ([9000] * 30, 9000, 0, 0),
    ([9000, 40000], 0, 0, 0),
    ([1500000, 10, 700000], 300000, 1000, 4),                       # several rounds a block
    ([100] * 900 + [100000], 50, 5, 1),                             # one long request among many short
    ([7] * 700, 3, 1, 1),
    ([2500] * 40, 333, 10, 0),
    ([3000] * 60 + [30000, 0, 1], 700, 16, 4),                      # a block a request, one of them in rounds
    ([200] * 152, 50, 3, 1),
    ([200] * 153, 50, 3, 1),
    ([9000, 20000, 500] * 20, 3000, 64, 4),                         # two blocks a request
])
def test_against_the_definition(lengths, budget, recent, sinks):
    _run(lengths, _rand(sum(lengths), 3), budget, recent, sinks, tail=5)


@pytest.mark.gpu
def test_budget_per_request():
    lengths = [500, 500, 0, 500, 1200]
    _run(lengths, _rand(sum(lengths), 5), torch.tensor([10, 600, 3, 0, 1199], dtype=torch.int32), 4, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [33, 3000, 50000])
def test_ties_zeros_and_non_finite(n):
    w = torch.randint(0, 4, (n,), generator=torch.Generator().manual_seed(n)).float()
    _run([n], w, n // 3, 2, 1)
    _run([n], torch.zeros(n), n // 2)
    z = torch.zeros(n)
    z[::2] = -0.0
    _run([n], z, n // 2)                                   # -0 and +0 are equal
    w = _rand(n, 1)
    w[::5] = float("nan")
    w[::7] = float("-inf")
    w[::11] = float("inf")
    w[1::3] *= -1
    w[2::13] = 1e-42                                       # subnormal
    for b in (1, n // 20, n // 2, n - 2):
        _run([n], w, b, 1, 1)
    _run([n], torch.full((n,), float("nan")), n // 2)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[700] * 50, [700] * 200, [12000, 5] * 40])
def test_ties_in_many_requests(lengths):
    n = sum(lengths)
    w = torch.randint(0, 4, (n,), generator=torch.Generator().manual_seed(n)).float()
    for budget in (1, 200, 650):
        _run(lengths, w, budget, 2, 1)


@pytest.mark.gpu
def test_keys_that_differ_in_the_last_bits_only():
    n = 20000
    base = torch.full((n,), 1.0).view(torch.int32)
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(0)).to(torch.int32)
    for mod in (n, 64, 1024):
        _run([n], (base + perm % mod).view(torch.float32), 777)


@pytest.mark.gpu
def test_no_requests_and_no_tokens():
    _run([], torch.zeros(0), 5, tail=3)
    _run([0, 0], torch.zeros(0), 5)


@pytest.mark.gpu
def test_bad_indptr_is_flagged_and_stays_in_bounds():
    n = 64
    pages = torch.arange(n, dtype=torch.int32, device=DEV)
    w = torch.rand(n, device=DEV)
    for ind in ([0, 40, 20, 64], [0, 30, 100, 64], [0, -5, 10, 64], [0, 64, 0, 64]):
        guard = torch.full((n + 64,), -7, dtype=torch.int32, device=DEV)
        wg = torch.full((n + 64,), -7.0, device=DEV)
        mla.kv_evict(pages, torch.tensor(ind, dtype=torch.int32, device=DEV), w, 8, recent=2, pages_out=guard[:n],
                     weights_out=wg[:n])
        torch.cuda.synchronize()
        assert mla.device_status() == mla.DEV_BAD_INDPTR
        assert (guard[n:] == -7).all() and (wg[n:] == -7).all()


@pytest.mark.gpu
def test_calls_on_two_streams():
    lengths = [30000, 9000, 12]
    total = sum(lengths)
    pages = torch.randperm(total, device=DEV).to(torch.int32)
    indptr = torch.tensor([0, 30000, 39000, 39012], dtype=torch.int32, device=DEV)
    w = torch.rand(total, device=DEV)
    want = mla.kv_evict(pages, indptr, w, 1000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [mla.kv_evict(pages, indptr, w, 1000, stream=s) for s in (side, None, side, None)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
    assert mla.device_status() == 0


@pytest.mark.gpu
def test_repeated_streamed_and_captured():
    lengths = [9000, 12, 3000]
    total = sum(lengths)
    pages = torch.randperm(total, device=DEV).to(torch.int32)
    indptr = torch.tensor([0, 9000, 9012, 12012], dtype=torch.int32, device=DEV)
    w = torch.rand(total, device=DEV)
    first = mla.kv_evict(pages, indptr, w, 1000, recent=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = mla.kv_evict(pages, indptr, w, 1000, recent=10, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mla.kv_evict(pages, indptr, w, 1000, recent=10)
    w.copy_(w.flip(0))
    g.replay()
    now = mla.kv_evict(pages, indptr, w, 1000, recent=10)
    assert all(torch.equal(a, b) for a, b in zip(out, now))


@pytest.mark.gpu
def test_the_longest_page_list():
    # one request of as many tokens as are accepted, all of one weight but a few: the first ones stay, and those
    n = 2**31 - 65536
    if torch.cuda.mem_get_info()[0] < 4 * n * 5:
        pytest.skip("%d GB of device memory free" % (4 * n * 5 >> 30))
    pages = torch.arange(n, dtype=torch.int32, device=DEV)
    indptr = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    w = torch.ones(n, device=DEV)
    heavy = [2**30 + 20000, 2**31 - 70000]
    w[heavy] = 2.0
    budget, recent = 2**30 + 12345, 7
    po, io, wo = mla.kv_evict(pages, indptr, w, budget, recent=recent)
    assert io.tolist() == [0, budget] and mla.device_status() == 0
    first = budget - recent - len(heavy)
    assert torch.equal(po[:first], pages[:first])
    assert po[first:budget].tolist() == heavy + list(range(n - recent, n))
    assert wo[first:budget].tolist() == [2.0, 2.0] + [1.0] * recent
    assert bool((wo[:first] == 1).all()) and bool((wo[budget:] == 0).all())
    # freed: what is left, in order
    at = budget
    for a, b in ((first, heavy[0]), (heavy[0] + 1, heavy[1]), (heavy[1] + 1, n - recent)):
        assert torch.equal(po[at:at + b - a], pages[a:b])
        at += b - a
    assert at == n
    del pages, w, po, wo
    torch.cuda.empty_cache()


def test_too_many_requests(lib):
    assert _call(lib, R=65537) == mla.MLA_ERR_UNSUPPORTED
    assert b"num_requests above 2^16" in lib.mla_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("R", [1025, 5000, 65536])
def test_more_requests_than_a_block_has_threads(R):
    # every block sums over all requests before its own; one long request among empty and short ones
    lengths = [(i * 7) % 5 for i in range(R)]
    lengths[R // 3] = 20000
    lengths[-1] = 9
    budgets = torch.tensor([(i * 11) % 4 for i in range(R)], dtype=torch.int32)
    budgets[R // 3] = 777
    _run(lengths, _rand(sum(lengths), R), budgets, 1, 1, tail=5)


@pytest.mark.gpu
@pytest.mark.parametrize("R", [3, 900])
def test_a_list_that_starts_past_its_first_entries(R):
    # a batch's later requests, with the whole batch's page list: what belongs to none of them is in neither part
    lengths, skip, tail = [(i * 13) % 40 + 1 for i in range(R)], 17, 6
    total = sum(lengths)
    g = torch.Generator().manual_seed(R)
    pages = torch.randperm(skip + total + tail, generator=g).to(torch.int32)
    w = _rand(skip + total + tail, R)
    indptr = torch.tensor([skip] + (skip + torch.tensor(lengths).cumsum(0)).tolist(), dtype=torch.int32)
    po = torch.full((skip + total + tail,), -7, dtype=torch.int32, device=DEV)
    wo = torch.full((skip + total + tail,), -7.0, device=DEV)
    _, io, _ = mla.kv_evict(pages.to(DEV), indptr.to(DEV), w.to(DEV), 11, recent=2, sinks=1, pages_out=po, weights_out=wo)
    kept, freed, counts, kw = _plain(pages[skip:].tolist(), lengths, w[skip:].tolist(), [11] * R, 2, 1)
    assert io.tolist() == [0] + torch.tensor(counts).cumsum(0).tolist()
    assert po.tolist() == kept + freed + [-7] * (skip + tail)
    assert wo.tolist() == kw + [0.0] * len(freed) + [-7.0] * (skip + tail)
    assert mla.device_status() == 0
