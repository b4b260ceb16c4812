"""query_absorb: host-side refusals (CPU), then its product and rotation
against the formula in 64 bits on the GPU: head counts, row counts around a
tile, layouts, both outputs."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

DEV = "cuda"
A = 1 << 20
B, C, D, E = (A + (i << 32) for i in range(1, 5))
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.library()


def _call(lib, **kw):
    a = dict(q=A, qr=384, qh=192, w=B, pos=C, cs=D, np=100, flags=0, T=10, H=2, scale=1.0, out=E, outr=1152)
    a.update(kw)
    return lib.mla_query_absorb(a["q"], a["qr"], a["qh"], a["w"], a["pos"], a["cs"], a["np"], a["flags"], a["T"], a["H"],
                                a["scale"], a["out"], a["outr"], None)


@pytest.mark.parametrize("kw,msg", [
    (dict(flags=4), b"flag"),
    (dict(T=-1), b"negative"),
    (dict(H=0), b"heads"),
    (dict(H=129), b"heads"),
    (dict(pos=None), b"together"),
    (dict(cs=None), b"together"),
    (dict(np=0), b"num_positions"),
    (dict(flags=2, scale=0.0, outr=1152), b"q_scale"),
    (dict(flags=2, scale=math.nan, outr=1152), b"q_scale"),
    (dict(qr=184), b"strides"),
    (dict(qh=196), b"strides"),
    (dict(qr=1 << 31), b"strides"),
    (dict(outr=576), b"out_row_stride"),
    (dict(outr=1156), b"out_row_stride"),
    (dict(flags=2, outr=1160), b"out_row_stride"),
    (dict(q=None), b"null"),
    (dict(w=None), b"null"),
    (dict(out=None), b"null"),
    (dict(q=A + 8), b"misaligned"),
    (dict(out=E + 8), b"misaligned"),
    (dict(cs=D + 8), b"misaligned"),
    (dict(pos=C + 4), b"misaligned"),
    (dict(out=A + 16 * 479), b"overlaps"),
    (dict(out=B), b"overlaps"),
    (dict(out=D + 25584), b"overlaps"),
    (dict(out=C), b"overlaps"),
])
def test_refusals(lib, kw, msg):
    assert _call(lib, **kw) == mla.MLA_ERR_INVALID
    assert msg in lib.mla_last_error()


def test_sizes(lib):
    assert _call(lib, T=1 << 31) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, T=0, q=None, w=None, out=None) == mla.MLA_OK
    assert _call(lib, T=0, q=None, pos=None, out=None) == mla.MLA_OK      # an empty tensor's pointer is null


def test_binding_refusals():
    mla.build()
    q, w = torch.zeros(4, 2, 192, dtype=BF), torch.zeros(2, 128, 512, dtype=BF)
    pos, cs = torch.zeros(4, dtype=torch.int64), torch.zeros(8, 64)
    for args, kw, msg in [
        ((q.half(), w), {}, "bf16"), ((q[:, 0], w), {}, "bf16"), ((q[..., :128], w), {}, "192"), ((q, w[:1]), {}, "w_uk"),
        ((q, w.float()), {}, "w_uk"), ((q, w), dict(positions=pos), "together"),
        ((q, w), dict(positions=pos, cos_sin=cs[:, :32]), "cos_sin"), ((q, w), dict(positions=pos[1:], cos_sin=cs), "positions"),
        ((q, w), {}, "CUDA"), ((q.expand(4, 2, 192).repeat(1, 65, 1), w.repeat(65, 1, 1)), {}, "128 heads"),
    ]:
        with pytest.raises(ValueError, match=msg):
            mla.query_absorb(*args, **kw)


# ------------------------------------------------------------------- GPU


def _inputs(T, H, seed=0, far=4000):
    g = torch.Generator().manual_seed(seed + 31 * T + H)
    q = torch.randn(T, H, 192, generator=g).to(BF).to(DEV)
    w = (torch.randn(H, 128, 512, generator=g) / 16).to(BF).to(DEV)
    pos = torch.randint(0, far, (T,), generator=g).to(DEV)
    freq = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    a = torch.arange(far, dtype=torch.float64)[:, None] * freq
    return q, w, pos, torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


def _plain(q, w, pos, cs, pairs):
    """The result in 64 bits, and what its float32 sums may be off by: 128 products' (exact in float32) sum in any
    order, 2^-24 x 128 of their magnitudes' sum; a rotation's two products and their sum 2^-22 of theirs."""
    q, w = q.double(), w.double()
    lat = torch.einsum("thn,hnc->thc", q[..., :128], w)
    off = torch.einsum("thn,hnc->thc", q[..., :128].abs(), w.abs()) * 2.0 ** -17
    r = q[..., 128:]
    mag = torch.zeros_like(r)
    if pos is not None:
        t = cs.double()[pos][:, None]
        c, s = t[..., :32], t[..., 32:]
        u, v = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :32], r[..., 32:])
        a, b = u * c - v * s, v * c + u * s
        r = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
        m = (u.abs() + v.abs()) * 2.0 ** -22
        mag = torch.stack([m, m], -1).flatten(-2) if pairs else torch.cat([m, m], -1)
    return torch.cat([lat, r], 2), torch.cat([off, mag], 2)


def _check(out, y, off, q_scale=None):
    if q_scale is None:
        assert out.dtype == BF
        assert torch.all((out.double() - y).abs() <= y.abs() * 2.0 ** -8 + off * 1.01)
        return
    z = (y / q_scale).clamp(-448, 448)
    # the reciprocal's and the product's roundings: 2^-23 of the quotient
    assert torch.all((out.view(E4M3).double() - z).abs() <=
                     z.abs() * 2.0 ** -4 + 2.0 ** -10 + (off / q_scale + z.abs() * 2.0 ** -22) * 1.07)


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale", [None, 0.03])
@pytest.mark.parametrize("T,H,rope", [
    (1, 1, "halves"), (1, 128, "pairs"), (2, 3, None), (64, 12, "halves"), (127, 12, "pairs"), (128, 5, "halves"),
    (129, 12, "halves"), (130, 96, "pairs"), (300, 1, "halves"), (513, 40, "pairs"), (2048, 12, "halves"),
    (5000, 16, "halves"), (1100, 96, None), (700, 128, "pairs"),
])
def test_product_and_rotation(T, H, rope, q_scale):
    q, w, pos, cs = _inputs(T, H)
    if rope is None:
        pos = cs = None
    out = mla.query_absorb(q, w, positions=pos, cos_sin=cs, interleaved=rope == "pairs", q_scale=q_scale)
    assert out.shape == (T, H, 576)
    y, off = _plain(q, w, pos, cs, rope == "pairs")
    _check(out, y, off, q_scale)
    assert mla.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("q_scale", [None, 0.03])
@pytest.mark.parametrize("layout", ["gap", "heads_first", "row", "padded", "bytes"])
def test_layouts(layout, q_scale):
    T, H = (1, 9) if layout == "row" else (200, 9)
    q, w, pos, cs = _inputs(T, H)
    want = mla.query_absorb(q, w, positions=pos, cos_sin=cs, q_scale=q_scale)
    type_, out = BF if q_scale is None else E4M3, None
    if layout in ("gap", "row"):
        q = torch.cat([torch.full((T, 40), math.nan, dtype=BF, device=DEV), q.flatten(1)], 1)[:, 40:].unflatten(1, (H, 192))
    elif layout == "heads_first":
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    else:
        out = torch.full((T, H + 3, 576), 7.0, device=DEV).to(type_)
        if layout == "bytes" and q_scale:
            out = out.view(torch.uint8)
    got = mla.query_absorb(q, w, positions=pos, cos_sin=cs, q_scale=q_scale, out=out)
    if out is not None:
        assert got.data_ptr() == out.data_ptr()
        assert got.view(E4M3 if q_scale else BF)[:, H:].float().eq(7).all()
        got = got[:, :H].contiguous()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.gpu
def test_rows_behind_the_last_are_left():
    q, w, pos, cs = _inputs(131, 4)
    held = torch.full((140, 4, 576), 3.0, dtype=BF, device=DEV)
    mla.query_absorb(q, w, positions=pos, cos_sin=cs, out=held[:131])
    assert held[131:].eq(3).all() and not held[:131].eq(3).all()


@pytest.mark.gpu
def test_infinite_and_nan_rows_stay_alone():
    q, w, pos, cs = _inputs(70, 3)
    want = mla.query_absorb(q, w, positions=pos, cos_sin=cs)
    bad = q.clone()
    bad[5, 1, 100], bad[9, 2, 130], bad[11, 0, 5] = math.nan, math.inf, math.inf
    got = mla.query_absorb(bad, w, positions=pos, cos_sin=cs)
    assert got[5, 1, :512].isnan().all() and got[11, 0, :512].isfinite().logical_not().all()
    assert not got[9, 2, 512:].isfinite().all() and got[9, 2, :512].isfinite().all()
    for t, h in ((5, 1), (9, 2), (11, 0)):
        got[t, h] = want[t, h]
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_no_rows():
    q, w = torch.zeros(0, 2, 192, dtype=BF, device=DEV), torch.zeros(2, 128, 512, dtype=BF, device=DEV)
    pos, cs = torch.zeros(0, dtype=torch.int64, device=DEV), torch.zeros(8, 64, device=DEV)
    for kw in ({}, dict(positions=pos, cos_sin=cs), dict(positions=pos, cos_sin=cs, q_scale=0.5)):
        assert mla.query_absorb(q, w, **kw).shape == (0, 2, 576)
    assert mla.device_status() == 0


@pytest.mark.gpu
def test_bad_position_is_flagged():
    q, w, pos, cs = _inputs(5, 2)
    pos[2], pos[4] = cs.shape[0], -1
    out = mla.query_absorb(q, w, positions=pos, cos_sin=cs)
    assert mla.device_status() == mla.DEV_BAD_POSITION
    pos[2] = pos[4] = 0
    _check(out, *_plain(q, w, pos, cs, False))


@pytest.mark.gpu
def test_other_stream_and_graph():
    q, w, pos, cs = _inputs(300, 12)
    want = mla.query_absorb(q, w, positions=pos, cos_sin=cs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = mla.query_absorb(q, w, positions=pos, cos_sin=cs, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = mla.query_absorb(q, w, positions=pos, cos_sin=cs)
    q.copy_(q.flip(0))
    pos.copy_(pos.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b.flip(0), want)


@pytest.mark.gpu
def test_past_32_bits():
    # the output's last rows are past 2^31 elements, 2^32 bytes
    T, H = 30000, 128
    q, w, pos, cs = _inputs(1, H)
    big = q.expand(T, H, 192).contiguous()
    big[-3:] = torch.randn(3, H, 192, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).to(BF)
    positions = pos.expand(T).contiguous()
    out = mla.query_absorb(big, w, positions=positions, cos_sin=cs)
    _check(out[-4:], *_plain(big[-4:], w, positions[-4:], cs, False))
    assert torch.equal(out[:-3], out[:1].expand(T - 3, H, 576))


@pytest.mark.gpu
def test_one_row_whose_heads_lie_far_apart():
    # one token of heads kept [H, T, D]: each stride within the limit, the last head past 2^30 elements
    H, T = 96, 1 << 16
    base = torch.empty(H, T, 192, dtype=BF, device=DEV)
    q, w, pos, cs = _inputs(1, H)
    base[:, 77] = q[0]
    far = base[:, 77:78].transpose(0, 1)
    assert far.stride(1) <= 1 << 30 < (H - 1) * far.stride(1)
    assert torch.equal(mla.query_absorb(far, w, positions=pos, cos_sin=cs), mla.query_absorb(q, w, positions=pos, cos_sin=cs))
