"""add_rms_norm: host-side refusals (CPU), then every output form against
the formula in 64 bits on the GPU, at the widths, strides and values where
it can go wrong."""

import ctypes

import pytest
import torch

import mla_decode_paged_gb300 as mla

DEV = "cuda"
NULL = None
A = 1 << 20          # fake 16-byte aligned addresses, far apart: every CPU case fails validation first
B, C, D, E, F = (A + (i << 28) for i in range(1, 6))


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.library()


def _call(lib, **kw):
    a = dict(x=A, xs=64, xt=0, r=NULL, rs=0, rt=0, w=B, eps=1e-5, T=4, D=64, quant=0, scale=0.0, out=C, os=64,
             sc=NULL, ro=NULL, ros=0)
    a.update(kw)
    return lib.mla_add_rms_norm(a["x"], a["xs"], a["xt"], a["r"], a["rs"], a["rt"], a["w"], a["eps"], a["T"], a["D"],
                                a["quant"], a["scale"], a["out"], a["os"], a["sc"], a["ro"], a["ros"], None)


RES = dict(r=D, rs=64, ro=E, ros=64)


@pytest.mark.parametrize("kw,msg", [
    (dict(xt=2), b"x_type"),
    (dict(RES, rt=1), b"residual_type"),
    (dict(quant=4), b"quant"),
    (dict(T=-1), b"negative"),
    (dict(D=0), b"width"),
    (dict(D=60), b"width"),
    (dict(D=32776, xs=32776, os=32776), b"width"),
    (dict(eps=0.0), b"eps"),
    (dict(eps=float("nan")), b"eps"),
    (dict(quant=3, scale=0.0), b"scale"),
    (dict(quant=3, scale=float("inf")), b"scale"),
    (dict(r=D, rs=64), b"together"),
    (dict(ro=D, ros=64), b"together"),
    (dict(xs=56), b"strides"),
    (dict(xs=68), b"strides"),
    (dict(os=60), b"strides"),
    (dict(RES, rs=8), b"strides"),
    (dict(RES, ros=72 + 4), b"strides"),
    (dict(x=NULL), b"null"),
    (dict(quant=1), b"null"),
    (dict(quant=2), b"null"),
    (dict(x=A + 8), b"misaligned"),
    (dict(quant=1, sc=D + 2), b"misaligned"),
    (dict(T=1 << 60), b"too large"),
    (dict(out=A + 128), b"overlaps"),                        # one row further in x
    (dict(out=B), b"overlaps"),                              # over the weight
    (dict(quant=1, out=A, sc=D), b"overlaps"),               # codes over x
    (dict(RES, ro=D + 128), b"overlaps"),
    (dict(RES, ro=C), b"overlaps"),                          # both outputs in one place
    (dict(RES, rt=2, ro=A), b"overlaps"),                    # f32 sums over 16-bit x
    (dict(quant=1, sc=A), b"overlaps"),
    (dict(quant=2, sc=C), b"overlaps"),
    (dict(xs=96, out=A + 64, os=96), b"overlaps"),           # columns 32..95 of a 96-wide buffer under 0..63
])
def test_refusals(lib, kw, msg):
    assert _call(lib, **kw) == mla.MLA_ERR_INVALID
    assert msg in lib.mla_last_error()


def test_no_rows_is_no_launch(lib):
    assert _call(lib, T=0, x=NULL, out=NULL) == mla.MLA_OK


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mla.add_rms_norm(x, w, 1e-5)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        mla.add_rms_norm(x.float(), w, 1e-5)


# ------------------------------------------------------------------- GPU

EPS = 1e-5
# float32 work per element: the sum of squares of at most 32 products a
# thread and ten joining steps (half of its error reaches the root), the
# root, two products, the scale and its reciprocal: under 64 roundings
SLACK = 64 * 2.0**-24


def _formula(x, w, r=None, eps=EPS):
    s = x.double() + (0 if r is None else r.double())
    return s, s / (s.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


def _check16(out, y, what):
    t = torch.finfo(out.dtype)
    tol = (t.eps / 2 + SLACK) * y.abs() + t.tiny * t.eps / 2
    bad = (out.double() - y).abs() > tol
    assert out.isfinite().all() and not bad.any(), "%s: %d off" % (what, int(bad.sum()))


def _groups(y, quant):
    D = y.shape[1]
    width = D if quant == "row" else 128
    return [(g, y[:, g * width:(g + 1) * width]) for g in range(-(-D // width))], width


def _check8(codes, scales, y, quant, static=None):
    assert codes.dtype == torch.float8_e4m3fn
    c = codes.double()
    if quant == "static":
        want = (y / static).clamp(-448, 448)
    else:
        parts, width = _groups(y, quant)
        ref = torch.stack([p.abs().amax(1) for _, p in parts], 1) / 448
        ref = torch.where(ref == 0, torch.ones_like(ref), ref)
        got = scales.double().view(ref.shape)
        assert ((got - ref).abs() <= SLACK * ref).all()
        want = torch.cat([p / ref[:, g:g + 1] for g, p in parts], 1)
    tol = (2.0**-4 + SLACK) * want.abs() + 2.0**-10     # half a step, normal and subnormal codes
    assert ((c - want).abs() <= tol).all()


def _inputs(T, D, xt, rt, seed, pad=0, rpad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, D + pad, generator=g, device=DEV).to(xt)[:, :D]
    w = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(xt)
    r = None if rt is None else torch.randn(T, D + rpad, generator=g, device=DEV).mul_(3).to(rt)[:, :D]
    return x, w, r


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "row", "group", "static"])
@pytest.mark.parametrize("T,D,xt,rt,pad", [
    (1, 8, torch.bfloat16, None, 0),
    (3, 64, torch.float16, torch.float16, 8),
    (5, 136, torch.bfloat16, torch.bfloat16, 0),
    (130, 512, torch.bfloat16, None, 64),
    (7, 520, torch.bfloat16, torch.float32, 24),
    (9, 1024, torch.float16, None, 0),
    (33, 1032, torch.bfloat16, torch.bfloat16, 0),
    (64, 1536, torch.bfloat16, torch.bfloat16, 576),
    (64, 7168, torch.bfloat16, torch.bfloat16, 0),
    (700, 7168, torch.float16, torch.float32, 8),
    (1, 8200, torch.bfloat16, torch.bfloat16, 0),
    (400, 16384, torch.bfloat16, torch.float32, 0),
    (2, 32768, torch.bfloat16, torch.bfloat16, 0),
])
def test_against_the_formula(T, D, xt, rt, pad, quant):
    x, w, r = _inputs(T, D, xt, rt, 7 * T + D, pad, pad)
    s, y = _formula(x, w, r)
    out, scales, ro = mla.add_rms_norm(x, w, EPS, r, quant=quant, scale=0.013 if quant == "static" else None)
    if quant is None:
        assert scales is None
        _check16(out, y, "out")
    else:
        _check8(out, scales, y, quant, 0.013)
    if r is None:
        assert ro is None
    else:
        # one float32 rounding of the sum, then the type's
        tol = (torch.finfo(rt).eps / 2 + 2.0**-24) * s.abs()
        assert ((ro.double() - s).abs() <= tol).all()


@pytest.mark.gpu
def test_many_rows_per_block_and_grid_wrap():
    # more rows than the launch's blocks: every block walks several
    for D in (64, 4096):
        x, w, r = _inputs(20011 if D == 4096 else 60001, D, torch.bfloat16, torch.bfloat16, 5)
        _, y = _formula(x, w, r)
        out, sc, _ = mla.add_rms_norm(x, w, EPS, r, quant="row")
        _check8(out, sc, y, "row")


@pytest.mark.gpu
def test_in_place_and_column_views():
    x, w, r = _inputs(37, 512, torch.bfloat16, torch.bfloat16, 1, 64, 8)
    want = mla.add_rms_norm(x, w, EPS, r)
    x2, r2 = x.clone(), r.clone()
    buf = torch.zeros(37, 1152, dtype=torch.bfloat16, device=DEV)
    buf[:, 576:1088] = x
    view = buf[:, 576:1088]
    out, _, ro = mla.add_rms_norm(view, w, EPS, r2, out=buf[:, :512], residual_out=r2)   # columns side by side
    assert ro is r2 and torch.equal(out, want[0]) and torch.equal(r2, want[2])
    assert torch.equal(view, x) and (buf[:, 512:576] == 0).all() and (buf[:, 1088:] == 0).all()
    out, _, ro = mla.add_rms_norm(x2, w, EPS, r, out=x2)                                  # over x
    assert torch.equal(x2, want[0]) and torch.equal(ro, want[2])
    x3 = x.clone()
    out, _, ro = mla.add_rms_norm(x3, w, EPS, r, residual_out=x3)                         # the sum over x
    assert torch.equal(out, want[0]) and torch.equal(x3, want[2])
    with pytest.raises(mla.MlaError, match="overlaps"):
        mla.add_rms_norm(buf[:, 8:520], w, EPS, out=buf[:, :512])


@pytest.mark.gpu
def test_zero_rows_tiny_rows_and_non_finite():
    D = 384
    x, w, _ = _inputs(9, D, torch.bfloat16, None, 3)
    x[0] = 0
    x[1] *= 2.0**-120
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4, :128] = 0
    x[5] *= 2.0**60            # the squares sum past float32's range
    x[6] = 3e38                # and each is past it
    _, y = _formula(x, w)
    out, _, _ = mla.add_rms_norm(x, w, EPS)
    fine = [0, 1, 4, 5, 6, 7, 8]
    _check16(out[fine], y[fine], "finite rows")
    assert out[2].isnan().all()
    assert out[3, 200].isnan() and (out[3, :200] == 0).all() and (out[3, 201:] == 0).all()
    for quant in ("row", "group"):
        codes, sc, _ = mla.add_rms_norm(x, w, EPS, quant=quant)
        sc = sc.view(9, -1)
        assert (sc[0] == 1).all() and (codes[0].float() == 0).all()
        assert sc[2].isnan().all() and codes[2].float().isnan().all()
        g = 0 if quant == "row" else 1
        assert sc[3, g].isnan() and codes[3].float()[:, None][200].isnan().all()
        if quant == "group":
            assert (sc[3, [0, 2]] == 1).all() and sc[4, 0] == 1
        _check8(codes[[4, 5, 6, 7, 8]], sc[[4, 5, 6, 7, 8]], y[[4, 5, 6, 7, 8]], quant)
        assert (sc[1] >= 2.0**-126).all()
    codes, _, _ = mla.add_rms_norm(x, w, EPS, quant="static", scale=2.0**-20)      # saturates
    assert (codes[[5, 7]].float().abs() == 448).float().mean() > 0.9 and codes[5].float().isfinite().all()


@pytest.mark.gpu
def test_uint8_codes_no_rows_own_stream_and_graph():
    x, w, r = _inputs(50, 1536, torch.bfloat16, torch.float32, 11)
    want, wsc, wro = mla.add_rms_norm(x, w, EPS, r, quant="group")
    o8 = torch.empty(50, 1536, dtype=torch.uint8, device=DEV)
    mla.add_rms_norm(x, w, EPS, r, quant="group", out=o8)
    assert torch.equal(o8, want.view(torch.uint8))
    out, sc, ro = mla.add_rms_norm(x[:0], w, EPS, r[:0], quant="row")
    assert out.shape == (0, 1536) and sc.shape == (0,) and ro.shape == (0, 1536)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, sc, ro = mla.add_rms_norm(x, w, EPS, r, quant="group", stream=side)
    side.synchronize()
    assert torch.equal(out.view(torch.uint8), o8) and torch.equal(sc, wsc) and torch.equal(ro, wro)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gout, gsc, gro = mla.add_rms_norm(x, w, EPS, r, quant="group")
    x.mul_(2)
    g.replay()
    again, asc, aro = mla.add_rms_norm(x, w, EPS, r, quant="group")
    assert torch.equal(gout.view(torch.uint8), again.view(torch.uint8)) and torch.equal(gsc, asc)
    assert torch.equal(gro, aro)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "row", "group", "static"])
@pytest.mark.parametrize("T,D,xt,rt,pad", [
    (1300, 1032, torch.bfloat16, torch.bfloat16, 0),
    (1217, 4096, torch.float16, None, 8),
    (2500, 7168, torch.bfloat16, torch.bfloat16, 0),
    (1300, 7168, torch.bfloat16, torch.float32, 8),
    (1300, 8200, torch.bfloat16, torch.bfloat16, 0),
    (1250, 16384, torch.float16, None, 0),
])
def test_many_wide_rows(T, D, xt, rt, pad, quant):
    x, w, r = _inputs(T, D, xt, rt, T + D, pad, pad)
    x[5] = 0
    x[6] *= 2.0**15 if xt == torch.float16 else 2.0**90
    x[7, 3] = float("nan")
    x[8, D - 1] = float("inf")
    if r is not None:
        r[5] = 0
    _, y = _formula(x, w, r)
    out, scales, ro = mla.add_rms_norm(x, w, EPS, r, quant=quant, scale=0.013 if quant == "static" else None)
    fine = torch.arange(T, device=DEV)
    fine = fine[(fine != 7) & (fine != 8) & x.isfinite().all(1)]
    if quant is None:
        _check16(out[fine], y[fine], "out")
        assert out[7].isnan().all() and out[8, D - 1].isnan() and (out[8, :D - 1] == 0).all()
    else:
        _check8(out[fine], None if scales is None else scales[fine], y[fine], quant, 0.013)
        assert out[7].float().isnan().all() and out[8, D - 1].float().isnan()
        if scales is not None:
            assert scales.view(T, -1)[7].isnan().all() and scales.view(T, -1)[8, -1].isnan()
    if r is not None:
        small = mla.add_rms_norm(x[:64], w, EPS, r[:64])[2]
        assert torch.equal(ro[:64].view(torch.int16 if rt != torch.float32 else torch.int32),
                           small.view(torch.int16 if rt != torch.float32 else torch.int32))
        keep = r.clone()
        again = mla.add_rms_norm(x, w, EPS, keep, quant=quant, scale=0.013 if quant == "static" else None,
                                 residual_out=keep)
        assert torch.equal(again[0].view(torch.uint8), out.view(torch.uint8))
        assert torch.equal(keep.view(torch.uint8), ro.contiguous().view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,rt,quant", [
    (60000, 256, torch.float32, "row"),
    (45000, 1024, torch.bfloat16, None),
    (39000, 520, None, "group"),
    (10000, 24576, torch.bfloat16, None),
])
def test_rows_in_place_do_not_depend_on_the_batch(T, D, rt, quant):
    # more rows than run at once, the next row's loads in flight while one is written over its inputs
    x, w, r = _inputs(T, D, torch.bfloat16, rt, D)
    parts = [slice(0, 50), slice(T // 2, T // 2 + 50), slice(T - 50, T)]
    want = [mla.add_rms_norm(x[p], w, EPS, None if r is None else r[p], quant=quant) for p in parts]
    out, sc, ro = mla.add_rms_norm(x, w, EPS, r, quant=quant, out=x if quant is None else None, residual_out=r)
    for p, (o, s, q) in zip(parts, want):
        assert torch.equal(out[p].view(torch.uint8), o.view(torch.uint8))
        assert s is None or torch.equal(sc[p], s)
        assert q is None or torch.equal(ro[p], q)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "row", "group", "static"])
@pytest.mark.parametrize("T,D,xt", [
    (200, 16392, torch.bfloat16),      # the first width that 512 threads of four vectors do not hold
    (200, 20480, torch.float16),
    (311, 24576, torch.bfloat16),
    (200, 28160, torch.bfloat16),      # the widest of which two rows fit a ring
    (200, 28168, torch.bfloat16),
    (160, 32768, torch.bfloat16),
])
def test_wide_rows_without_a_residual_over_all_sms(T, D, xt, quant):
    x, w, _ = _inputs(T, D, xt, None, T + D)
    _, y = _formula(x, w)
    out, scales, ro = mla.add_rms_norm(x, w, EPS, quant=quant, scale=0.013 if quant == "static" else None)
    assert ro is None
    if quant is None:
        _check16(out, y, "out")
    else:
        _check8(out, scales, y, quant, 0.013)
    few = mla.add_rms_norm(x[:3], w, EPS, quant=quant, scale=0.013 if quant == "static" else None)
    assert torch.equal(out[:3].view(torch.uint8), few[0].view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,quant", [(262200, 8200, "group"), (2100000, 1024, None)])
def test_offsets_past_31_bits(T, D, quant):
    # more than 2^31 elements, by the ring and by a warp a row: the last rows as they are in a small call
    assert T * D > 2**31
    x = torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)
    parts = [slice(0, 40), slice(2**31 // D - 20, 2**31 // D + 20), slice(T - 40, T)]
    for k, p in enumerate(parts):
        x[p] = _inputs(40, D, torch.bfloat16, None, 50 + k)[0]
    w = _inputs(1, D, torch.bfloat16, None, 49)[1]
    out, sc, _ = mla.add_rms_norm(x, w, EPS, quant=quant)
    for p in parts:
        _, y = _formula(x[p], w)
        if quant is None:
            _check16(out[p], y, "rows %s" % p)
        else:
            _check8(out[p], sc[p], y, quant)
    assert bool((out[100:110].float() == 0).all())
    del x, out, sc
    torch.cuda.empty_cache()
