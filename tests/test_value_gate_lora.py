"""value_gate_lora: host-side refusals (CPU), then the projection, the
adapters and the gate against the formula in 64 bits on the GPU: ranks,
head counts, rows per request, requests without an adapter or without
tokens, shared and bad adapter indices."""

import pytest
import torch

import mla_decode_paged_gb300 as mla

DEV = "cuda"
A = 1 << 20
B, C, D, E, F, G, H, I, J = (A + (i << 28) for i in range(1, 10))


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.library()


def _call(lib, **kw):
    a = dict(latent=A, w=B, gate=C, lengths=D, la=E, lb=F, ad=G, sc=H, n=3, rank=16, R=4, qlen=2, heads=12, out=I,
             ws=J, wsn=1 << 27)
    a.update(kw)
    return lib.mla_value_gate_lora(a["latent"], a["w"], a["gate"], a["lengths"], a["la"], a["lb"], a["ad"], a["sc"],
                                   a["n"], a["rank"], a["R"], a["qlen"], a["heads"], a["out"], a["ws"], a["wsn"], None)


@pytest.mark.parametrize("kw,msg", [
    (dict(R=-1), b"num_requests"),
    (dict(qlen=0), b"qlen"),
    (dict(qlen=17), b"qlen"),
    (dict(heads=0), b"heads"),
    (dict(heads=129), b"heads"),
    (dict(rank=0), b"rank"),
    (dict(rank=12), b"rank"),
    (dict(rank=136), b"rank"),
    (dict(n=0), b"num_adapters"),
    (dict(latent=None), b"null"),
    (dict(lb=None), b"null"),
    (dict(ad=None), b"null"),
    (dict(out=None), b"null"),
    (dict(latent=A + 8), b"misaligned"),
    (dict(la=E + 8), b"misaligned"),
    (dict(ws=J + 8), b"misaligned"),
    (dict(gate=C + 2), b"misaligned"),
    (dict(out=C), b"out overlaps"),
    (dict(out=A + 8 * 12 * 1024 - 4), b"out overlaps"),
    (dict(out=H + 8), b"out overlaps"),
    (dict(ws=I), b"workspace overlaps"),
    (dict(ws=B + 12 * 128 * 1024 - 16), b"workspace overlaps"),
    (dict(ws=G), b"workspace overlaps"),
])
def test_refusals(lib, kw, msg):
    assert _call(lib, **kw) == mla.MLA_ERR_INVALID
    assert msg in lib.mla_last_error()


def test_unsupported_and_nothing_to_do(lib):
    assert _call(lib, n=1 << 30) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, R=1 << 30, qlen=4, wsn=1 << 62) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, R=0) == mla.MLA_OK


def test_workspace(lib):
    n = mla.value_gate_lora_workspace(4, 2, 12, 16)
    assert n >= 0
    if n:
        assert _call(lib, wsn=n - 1) == mla.MLA_ERR_INVALID and b"workspace" in lib.mla_last_error()
        assert _call(lib, ws=None) == mla.MLA_ERR_INVALID and b"workspace" in lib.mla_last_error()
    with pytest.raises(mla.MlaError, match="rank"):
        mla.value_gate_lora_workspace(4, 2, 12, 7)


def test_binding_refusals():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = torch.zeros(2, dtype=torch.int32)
    good = [z(2, 3, 512), z(3, 128, 512), z(2, 384), i, z(2, 8, 512), z(2, 384, 8), i, torch.zeros(2)]
    with pytest.raises(ValueError, match="CUDA"):
        mla.value_gate_lora(*good)
    for k, bad in ((0, z(2, 3, 511)), (4, z(2, 8, 500)), (5, z(2, 384, 16)), (6, i.long()), (7, torch.zeros(3))):
        with pytest.raises(ValueError):
            mla.value_gate_lora(*[bad if j == k else t for j, t in enumerate(good)])


# ------------------------------------------------------------------- GPU


def _make(R, qlen, heads, rank, n, seed, astd=0.04, bstd=0.2):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(torch.bfloat16)

    S = R * qlen
    return dict(latent=normal(S, heads, 512, std=0.05), w_uv=normal(heads, 128, 512, std=0.044),
                gate=normal(S, heads * 128), lengths=torch.randint(1, 99, (R,), generator=g, device=DEV).to(torch.int32),
                lora_a=normal(n, rank, 512, std=astd), lora_b=normal(n, heads * 128, rank, std=bstd),
                adapters=torch.randint(-1, n, (R,), generator=g, device=DEV).to(torch.int32),
                lora_scale=torch.rand(n, generator=g, device=DEV) * 4 - 2, qlen=qlen)


def _formula(s):
    """The result in 64 bits, and a bound of the kernel's error before the last rounding: 512 products and their
    float32 sum (under 64 roundings of the sum of magnitudes in the tensor core's steps of 16), the low-rank product
    as two bf16 terms (2^-16) with the scale, the sigmoid (under 2^-19)."""
    S, H, _ = s["latent"].shape
    x = s["latent"].double().transpose(0, 1)
    w = s["w_uv"].double()
    val = (x @ w.transpose(1, 2)).transpose(0, 1).reshape(S, -1)
    mag = (x.abs() @ w.abs().transpose(1, 2)).transpose(0, 1).reshape(S, -1) * 64 * 2.0**-24
    q = s["qlen"]
    for r, a in enumerate(s["adapters"].tolist()):
        if 0 <= a < s["lora_a"].shape[0]:
            xa = x[:, r * q:(r + 1) * q]
            A, Bm = s["lora_a"][a].double(), s["lora_b"][a].double().view(H, 128, -1)
            f = float(s["lora_scale"][a])
            val[r * q:(r + 1) * q] += f * ((xa @ A.T) @ Bm.transpose(1, 2)).transpose(0, 1).reshape(q, -1)
            m = ((xa.abs() @ A.T.abs()) * 64 * 2.0**-24 + (xa @ A.T).abs() * 2.0**-16) @ Bm.abs().transpose(1, 2)
            mag[r * q:(r + 1) * q] += abs(f) * m.transpose(0, 1).reshape(q, -1)
    sig = 1 / (1 + torch.exp(-s["gate"].double()))
    live = (s["lengths"] > 0).repeat_interleave(q)[:, None]
    out = torch.where(live, val * sig, torch.zeros_like(val))
    return out, torch.where(live, mag * sig + 2.0**-19 * out.abs(), torch.zeros_like(val))


def _check(out, s):
    want, bound = _formula(s)
    assert out.isfinite().all()
    bad = (out.double() - want).abs() > bound + 2.0**-8 * (want.abs() + bound) + 1e-40
    assert not bad.any(), "%d of %d off" % (int(bad.sum()), bad.numel())


@pytest.mark.gpu
@pytest.mark.parametrize("R,qlen,heads,rank,n", [
    (1, 1, 1, 8, 1),
    (2, 1, 12, 16, 2),
    (64, 1, 12, 16, 64),
    (17, 1, 12, 40, 3),
    (33, 3, 5, 24, 7),
    (20, 8, 12, 64, 20),
    (5, 16, 3, 128, 2),
    (7, 5, 16, 72, 4),
    (32, 1, 96, 32, 8),
    (300, 1, 4, 8, 300),
    (256, 8, 12, 64, 32),
    (40, 2, 128, 104, 5),
    (300, 3, 12, 16, 5),         # several tiles a block, requests across tiles
    (130, 16, 7, 128, 9),
    (3, 16, 128, 64, 3),
    (90, 9, 20, 48, 90),
])
def test_against_the_formula(R, qlen, heads, rank, n):
    s = _make(R, qlen, heads, rank, n, R + rank)
    _check(mla.value_gate_lora(**s), s)
    assert mla.device_status() == 0


@pytest.mark.gpu
def test_adapters_that_dominate():
    s = _make(19, 2, 12, 32, 5, 3, astd=0.5, bstd=3.0)
    _check(mla.value_gate_lora(**s), s)


@pytest.mark.gpu
@pytest.mark.parametrize("adapters", [[-1] * 18, [2] * 18, [0, 0, 1, 1, -1, -1] * 3])
def test_no_adapter_and_shared_adapters(adapters):
    s = _make(18, 4, 12, 16, 3, 4)
    s["adapters"] = torch.tensor(adapters, dtype=torch.int32, device=DEV)
    if all(a < 0 for a in adapters):     # adapters nobody uses are not read into any result
        s["lora_a"].fill_(float("nan"))
        s["lora_b"].fill_(float("nan"))
        s["lora_scale"].fill_(float("nan"))
    _check(mla.value_gate_lora(**s), s)


@pytest.mark.gpu
def test_nan_stays_with_its_adapter():
    s = _make(24, 1, 12, 16, 4, 5)
    s["adapters"] = (torch.arange(24, device=DEV) % 4 - 1).to(torch.int32)       # -1, 0, 1, 2
    clean = mla.value_gate_lora(**s)
    s["lora_a"][1] = float("nan")
    s["lora_b"][3] = float("inf")                                                # nobody's
    out = mla.value_gate_lora(**s)
    hit = s["adapters"] == 1
    assert out[hit].isnan().all() and torch.equal(out[~hit], clean[~hit])
    s["lora_a"][1] = 0.01
    s["lora_b"][1] = float("inf")
    out = mla.value_gate_lora(**s)
    assert not out[hit].isfinite().any() and torch.equal(out[~hit], clean[~hit])


@pytest.mark.gpu
def test_empty_requests_are_zero_whatever_they_hold():
    s = _make(21, 3, 12, 24, 4, 6)
    s["lengths"][::3] = 0
    s["lengths"][1] = -2
    dead = (s["lengths"] <= 0).repeat_interleave(3)
    s["gate"][dead] = float("nan")
    out = mla.value_gate_lora(**s)
    assert (out[dead] == 0).all()
    s["gate"][dead] = 0
    _check(out, s)
    s["latent"][dead] = float("nan")
    again = mla.value_gate_lora(**s)
    assert torch.equal(again, out)


@pytest.mark.gpu
def test_bad_adapter_indices_are_flagged_and_skipped():
    s = _make(6, 2, 12, 16, 3, 7)
    s["adapters"] = torch.tensor([0, 3, -2, 2, 2**31 - 1, -(2**31)], dtype=torch.int32, device=DEV)
    out = mla.value_gate_lora(**s)
    assert mla.device_status() == mla.DEV_BAD_ADAPTER
    s["adapters"] = torch.tensor([0, -1, -1, 2, -1, -1], dtype=torch.int32, device=DEV)
    assert torch.equal(out, mla.value_gate_lora(**s))
    assert mla.device_status() == 0


@pytest.mark.gpu
def test_given_buffers_streams_and_graphs():
    s = _make(48, 2, 12, 32, 9, 8)
    want = mla.value_gate_lora(**s)
    n = mla.value_gate_lora_workspace(48, 2, 12, 32)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    assert mla.value_gate_lora(**s, out=out, workspace=ws) is out and torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [mla.value_gate_lora(**s, stream=st) for st in (side, None, side, None)]      # overlapping calls
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = mla.value_gate_lora(**s)
        graphs.append((g, o))
    s["latent"].mul_(2)
    for g, _ in graphs:
        g.replay()
    now = mla.value_gate_lora(**s)
    assert all(torch.equal(o, now) for _, o in graphs)


@pytest.mark.gpu
def test_without_adapters_it_is_value_gate_up_to_one_rounding():
    s = _make(30, 2, 12, 16, 2, 9)
    s["adapters"].fill_(-1)
    out = mla.value_gate_lora(**s).double()
    ref = mla.value_gate(s["latent"], s["w_uv"], s["gate"], s["lengths"], 2).double()
    # value_gate rounds the value and the product (2^-8 each), this one the product: 3 half steps apart at most
    assert ((out - ref).abs() <= 3.02 * 2.0**-8 * out.abs() + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("R,heads,rank", [(40, 12, 24), (150, 5, 16), (70, 3, 128)])
def test_rows_that_share_adapters_in_no_order(R, heads, rank):
    # an adapter of more rows than a product holds, some of a few, some of one, and none
    s = _make(R, 1, heads, rank, 6, 31)
    ad = [0 if i % 3 else (i * 7) % 9 - 1 for i in range(R)]
    s["adapters"] = torch.tensor([a if a < 6 else -1 for a in ad], dtype=torch.int32, device=DEV)
    want = mla.value_gate_lora(**s)
    _check(want, s)
    s["latent"][4] = float("nan")       # a row's own only, whoever shares its adapter
    got = mla.value_gate_lora(**s)
    others = torch.arange(R, device=DEV) != 4
    assert torch.equal(got[others], want[others])
    assert got[4].isnan().any()


@pytest.mark.gpu
@pytest.mark.parametrize("R,heads,rank,n", [
    (100, 96, 32, 8),           # one block a head, four tiles each
    (33, 96, 16, 33),           # the second tile holds one row
    (385, 12, 64, 5),           # 13 tiles over 12 blocks of a head: one of them has two
    (1000, 12, 16, 40),         # three tiles a block or two, the last of eight rows
    (1000, 12, 128, 1000),      # and an adapter a row
    (700, 40, 8, 3),            # eight tiles a block or seven
])
def test_single_rows_over_several_tiles_a_block(R, heads, rank, n):
    s = _make(R, 1, heads, rank, n, R + rank)
    s["lengths"][5::37] = 0
    out = mla.value_gate_lora(**s)
    _check(out, s)
    assert torch.equal(mla.value_gate_lora(**s), out)
    for r in (2, R // 2, R - 1):        # a row's own NaN stays in its row, in every tile of a block
        s["latent"][r] = float("nan")
    got = mla.value_gate_lora(**s)
    others = torch.ones(R, dtype=torch.bool, device=DEV)
    others[[2, R // 2, R - 1]] = False
    assert torch.equal(got[others], out[others])
    for r in (2, R // 2, R - 1):
        assert got[r].isnan().all() if s["lengths"][r] > 0 else (got[r] == 0).all()
    assert mla.device_status() == 0


@pytest.mark.gpu
def test_a_padded_row_of_a_batch_does_not_depend_on_the_others():
    # the same requests alone (tiles of few rows) and in a batch that takes several tiles a block
    s = _make(600, 1, 24, 40, 9, 21)
    out = mla.value_gate_lora(**s)
    few = {k: (v[:7] if k in ("latent", "gate", "lengths", "adapters") else v) for k, v in s.items()}
    want, bound = _formula(few)
    got = mla.value_gate_lora(**{k: (v.contiguous() if isinstance(v, torch.Tensor) else v) for k, v in few.items()})
    for o in (out[:7], got):
        assert ((o.double() - want).abs() <= bound + 2.0**-8 * (want.abs() + bound) + 1e-40).all()


@pytest.mark.gpu
@pytest.mark.parametrize("R,qlen,heads,rank", [(43800, 1, 96, 8), (21900, 2, 96, 8)])
def test_offsets_past_31_bits(R, qlen, heads, rank):
    # more than 2^31 latent elements; the first, a middle and the last requests against the formula
    S = R * qlen
    assert S * heads * 512 > 2**31
    s = dict(_make(96, qlen, heads, rank, 5, 77))
    picks = torch.cat([torch.arange(32), torch.arange(2**31 // (heads * 512 * qlen) - 16, 2**31 // (heads * 512 * qlen) + 16),
                       torch.arange(R - 32, R)]).to(DEV)
    rows = (picks[:, None] * qlen + torch.arange(qlen, device=DEV)).view(-1)
    big = dict(s, latent=torch.zeros(S, heads, 512, dtype=torch.bfloat16, device=DEV),
               gate=torch.zeros(S, heads * 128, dtype=torch.bfloat16, device=DEV),
               lengths=torch.ones(R, dtype=torch.int32, device=DEV),
               adapters=torch.zeros(R, dtype=torch.int32, device=DEV))
    for k, at in (("latent", rows), ("gate", rows), ("lengths", picks), ("adapters", picks)):
        big[k][at] = s[k]
    out = mla.value_gate_lora(**big)
    assert mla.device_status() == 0
    _check(out[rows], s)
    assert bool((out[100 * qlen:200 * qlen] == 0).all())
    del big, out
    torch.cuda.empty_cache()
