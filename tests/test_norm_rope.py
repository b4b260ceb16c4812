"""norm_rope: host-side refusals (CPU), then heads of every kind against the
formula in 64 bits on the GPU: widths, layouts, rotations, outputs, slots."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

DEV = "cuda"
A = 1 << 20
B, C, D, E, F, G = (A + (i << 32) for i in range(1, 7))
BF, FP = torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.library()


def _call(lib, **kw):
    a = dict(x=A, xr=256, xh=128, type=0, w=B, n=128, eps=1e-6, pos=C, cs=D, np=100, start=0, rope=64, flags=0, T=10, H=2,
             width=128, quant=1, scale=0.0, slots=None, rows=10, out=E, outr=256, outh=128, sc=F)
    a.update(kw)
    return lib.mla_norm_rope(a["x"], a["xr"], a["xh"], a["type"], a["w"], a["n"], a["eps"], a["pos"], a["cs"], a["np"],
                             a["start"], a["rope"], a["flags"], a["T"], a["H"], a["width"], a["quant"], a["scale"],
                             a["slots"], a["rows"], a["out"], a["outr"], a["outh"], a["sc"], None)


@pytest.mark.parametrize("kw,msg", [
    (dict(type=2), b"x_type"),
    (dict(flags=2), b"flag"),
    (dict(quant=2), b"quant"),
    (dict(quant=4), b"quant"),
    (dict(T=-1), b"negative"),
    (dict(rows=-1), b"negative"),
    (dict(H=0), b"heads"),
    (dict(H=65537), b"heads"),
    (dict(width=0), b"width"),
    (dict(width=132), b"width"),
    (dict(width=1032), b"width"),
    (dict(n=0), b"norm_dim"),
    (dict(n=136), b"norm_dim"),
    (dict(n=60), b"norm_dim"),
    (dict(eps=0.0), b"eps"),
    (dict(eps=math.nan), b"eps"),
    (dict(pos=None), b"together"),
    (dict(cs=None), b"together"),
    (dict(rope=0), b"rope"),
    (dict(rope=24), b"rope"),
    (dict(rope=144), b"rope"),
    (dict(start=72), b"rope"),
    (dict(start=-8), b"rope"),
    (dict(start=4), b"rope"),
    (dict(np=0), b"num_positions"),
    (dict(quant=3, scale=0.0), b"scale"),
    (dict(quant=3, scale=math.inf), b"scale"),
    (dict(xr=-8), b"strides"),
    (dict(xh=132), b"strides"),
    (dict(outr=1 << 31), b"strides"),
    (dict(x=None), b"null"),
    (dict(out=None), b"null"),
    (dict(sc=None), b"null"),
    (dict(x=A + 8), b"misaligned"),
    (dict(w=B + 2), b"misaligned"),
    (dict(cs=D + 4), b"misaligned"),
    (dict(pos=C + 4), b"misaligned"),
    (dict(outh=120), b"heads overlap"),
    (dict(outr=128), b"heads overlap"),
    (dict(out=A), b"overlaps"),                         # codes over 16-bit columns
    (dict(quant=0, out=A, outr=264), b"overlaps"),      # x, of other strides
    (dict(quant=0, out=A + 16), b"overlaps"),
    (dict(quant=0, out=A, slots=G), b"overlaps"),       # x's rows, scattered
    (dict(quant=0, out=B), b"overlaps"),
    (dict(quant=0, out=D + 25584), b"overlaps"),
    (dict(sc=E + 2556), b"overlaps"),
    (dict(sc=A + 5116), b"overlaps"),
])
def test_refusals(lib, kw, msg):
    assert _call(lib, **kw) == mla.MLA_ERR_INVALID
    assert msg in lib.mla_last_error()


def test_too_large(lib):
    assert _call(lib, T=1 << 30) == mla.MLA_ERR_UNSUPPORTED
    assert _call(lib, slots=G, rows=1 << 31) == mla.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(quant=0, out=A),                                               # in place
    dict(quant=0, out=A + 512, xr=512, outr=512),                       # columns beside x's
    dict(xr=128, xh=1280, outr=128, outh=1280),                         # heads, each of its rows
    dict(xr=0, xh=0),                                                   # one row, shared
])
def test_calls_that_are_taken(lib, kw):
    # no device here: they get as far as asking for one
    if torch.cuda.is_available():
        pytest.skip("made-up pointers")
    assert _call(lib, **kw) == mla.MLA_ERR_CUDA


def test_empty(lib):
    assert _call(lib, T=0, x=None, out=None, sc=None) == mla.MLA_OK


def test_no_tokens(lib):
    # an empty tensor's pointer is null
    assert _call(lib, T=0, x=None, pos=None, out=None, sc=None) == mla.MLA_OK
    assert _call(lib, T=0, x=None, pos=None, slots=None, out=None, sc=None, quant=0) == mla.MLA_OK


def test_binding_refusals():
    mla.build()
    x, w = torch.zeros(4, 2, 64, dtype=BF), torch.ones(64, dtype=BF)
    pos, cs = torch.zeros(4, dtype=torch.int64), torch.zeros(8, 32)
    for args, kw, msg in [
        ((x.float(),), {}, "bf16"), ((x[0, 0],), {}, r"\[T, H, D\]"), ((x.transpose(1, 2),), {}, "contiguous heads"),
        ((x, w[:0]), {}, "8 to D"), ((x, torch.ones(72, dtype=BF)), {}, "8 to D"), ((x, w.half()), {}, "weight"),
        ((x,), dict(positions=pos), "together"), ((x,), dict(cos_sin=cs), "together"),
        ((x,), dict(positions=pos[:3], cos_sin=cs), "positions"), ((x,), dict(positions=pos.int(), cos_sin=cs), "positions"),
        ((x,), dict(positions=pos, cos_sin=cs.double()), "cos_sin"), ((x,), dict(quant="row"), "quant"),
        ((x,), dict(quant="static"), "scale"), ((x,), dict(scale=1.0), "scale"), ((x,), dict(out_scales=cs), "out_scales"),
        ((x,), dict(slots=pos), "cache"), ((x,), dict(slots=pos, quant="head", out=x.to(E4M3)), "cache"),
        ((x,), dict(slots=pos[:2], out=x), "slots"), ((x,), dict(), "CUDA"), ((x, 1.0), {}, "tensor"),
        ((x,), dict(rope_start=1.5), "rope_start"),
    ]:
        with pytest.raises(ValueError, match=msg):
            mla.norm_rope(*args, **kw)


# ------------------------------------------------------------------- GPU


def _table(n, d):
    freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    a = torch.arange(n, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _plain(x, weight, eps, positions, cs, start, pairs):
    """The rotated and normed heads in 64 bits, and each row's largest normed magnitude (on the CPU)."""
    y = x.cpu().double().clone()
    if weight is not None:
        n = weight.numel()
        y[..., :n] *= torch.rsqrt(y[..., :n].square().mean(-1, keepdim=True) + eps) * weight.cpu().double()
    top = y.abs().amax(-1, keepdim=True)
    if positions is not None:
        t = cs.cpu().double()[positions.cpu()]
        half = t.shape[1] // 2
        c, s = t[:, None, :half], t[:, None, half:]
        span = y[..., start:start + 2 * half]
        u, v = (span[..., 0::2], span[..., 1::2]) if pairs else (span[..., :half], span[..., half:])
        a, b = u * c - v * s, v * c + u * s
        y[..., start:start + 2 * half] = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return y, top


def _check(out, scales, y, top, quant, scale):
    """In float32 every value is off by less than 2^-18 of its row's largest: sums of at most 1,024 squares in lanes of 32
    and five shuffles give the norm to 40 x 2^-24, the products and the rotation add 6 x 2^-24; then one rounding."""
    out = out.cpu()
    if quant is None:
        step = torch.finfo(out.dtype).eps / 2
        tiny = 2.0 ** -25 if out.dtype == FP else 0.0       # half a step of fp16's subnormals
        assert torch.all((out.double() - y).abs() <= y.abs() * step + top * 2.0 ** -18 + tiny)
        return
    codes = out.view(E4M3).float().double()
    if quant == "head":
        want = y.abs().amax(-1) / 448
        want[want == 0] = 1
        assert torch.all((scales.cpu().double() - want).abs() <= want * 2.0 ** -17)
        sc = scales.cpu().double()[..., None]
    else:
        sc = torch.tensor(scale, dtype=torch.float64)
    z = (y / sc).clamp(-448, 448)
    assert torch.all((codes - z).abs() <= z.abs() * 2.0 ** -4 + 2.0 ** -10 + top / sc * 2.0 ** -17)


def _inputs(T, H, width, norm, rope, type_, seed=0, far=5000):
    g = torch.Generator().manual_seed(seed + T + 7 * H + width)
    x = (torch.randn(T, H, width, generator=g) * torch.rand(T, H, 1, generator=g).mul(4).exp()).to(type_).to(DEV)
    w = (1 + 0.2 * torch.randn(norm, generator=g)).to(type_).to(DEV) if norm else None
    pos = torch.randint(0, far, (T,), generator=g).to(DEV) if rope else None
    cs = _table(far, rope).to(DEV) if rope else None
    return x, w, pos, cs


@pytest.mark.gpu
@pytest.mark.parametrize("type_", [BF, FP])
@pytest.mark.parametrize("T,H,width,norm,rope,start,pairs,quant", [
    (1, 1, 8, 8, 0, 0, False, None),
    (1, 1, 16, 0, 16, 0, False, "head"),
    (3, 5, 24, 8, 16, 8, True, None),
    (7, 1, 64, 64, 64, 0, False, "static"),
    (64, 64, 128, 0, 64, 0, False, "head"),
    (5, 3, 128, 128, 128, 0, True, "head"),
    (33, 12, 192, 192, 64, 128, True, None),
    (33, 12, 192, 192, 64, 128, False, None),
    (9, 2, 192, 128, 64, 128, False, "static"),
    (2, 7, 200, 200, 32, 40, False, "head"),
    (17, 3, 256, 0, 128, 64, False, None),
    (5, 1, 264, 264, 16, 248, True, "static"),
    (11, 2, 384, 320, 64, 320, False, "head"),
    (130, 1, 576, 512, 64, 512, False, "static"),
    (130, 1, 576, 512, 64, 512, True, None),
    (4, 3, 776, 0, 256, 520, False, "head"),
    (3, 2, 1024, 1024, 1024, 0, False, None),
    (3, 2, 1024, 1000, 512, 512, True, "head"),
    (700, 33, 40, 40, 32, 0, False, None),
    (2, 65, 48, 0, 0, 0, False, "head"),
])
def test_heads(T, H, width, norm, rope, start, pairs, quant, type_):
    x, w, pos, cs = _inputs(T, H, width, norm, rope, type_)
    scale = 0.11 if quant == "static" else None
    out, scales = mla.norm_rope(x, w, 1e-5, positions=pos, cos_sin=cs, rope_start=start, interleaved=pairs, quant=quant,
                                scale=scale)
    assert out.shape == x.shape and out.dtype == (type_ if quant is None else E4M3)
    y, top = _plain(x, w, 1e-5, pos, cs, start, pairs)
    _check(out, scales, y, top, quant, scale)
    assert mla.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "head", "static"])
@pytest.mark.parametrize("layout", ["padded", "heads_first", "shared", "columns"])
def test_layouts(layout, quant):
    T, H, width = 37, 6, 128
    x, w, pos, cs = _inputs(T, H, width, width, 64, BF)
    out = None
    if layout == "padded":          # a slice of a fused projection; the output's heads apart
        x = torch.cat([torch.zeros(T, 24, dtype=BF, device=DEV), x.flatten(1)], 1)[:, 24:].unflatten(1, (H, width))
        out = torch.zeros(T, H + 2, width + 8, dtype=BF if quant is None else E4M3, device=DEV)[:, :H, :width]
    elif layout == "heads_first":
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
        out = torch.zeros(H, T, width, dtype=BF if quant is None else E4M3, device=DEV).transpose(0, 1)
    elif layout == "shared":
        x = x[:1, :1].expand(T, H, width)
    else:                           # beside x in one buffer
        both = torch.zeros(T, 2 * H, width, dtype=BF, device=DEV)
        both[:, :H] = x
        x = both[:, :H]
        if quant is None:
            out = both[:, H:]
    before = x.clone()
    got, scales = mla.norm_rope(x, w, positions=pos, cos_sin=cs, rope_start=64, quant=quant, out=out,
                                scale=0.05 if quant == "static" else None)
    assert torch.equal(before.view(torch.int16), x.view(torch.int16))
    y, top = _plain(x, w, 1e-6, pos, cs, 64, False)
    _check(got, scales, y, top, quant, 0.05)
    if out is not None:
        assert got.data_ptr() == out.data_ptr() and got.stride() == out.stride()
        if layout == "padded":
            assert not out._base[:, H:].any() if quant is None else not out._base.view(torch.uint8)[:, H:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,H,width,rope", [(5, 3, 64, 64), (300, 12, 192, 64), (2000, 1, 576, 512), (9, 2, 1024, 1024)])
def test_in_place(T, H, width, rope, pairs):
    x, w, pos, cs = _inputs(T, H, width, width, rope, BF)
    want = mla.norm_rope(x, w, positions=pos, cos_sin=cs, interleaved=pairs)[0]
    got = mla.norm_rope(x, w, positions=pos, cos_sin=cs, interleaved=pairs, out=x)[0]
    assert got.data_ptr() == x.data_ptr() and torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "head", "static"])
@pytest.mark.parametrize("flat", [False, True])
def test_slots(quant, flat):
    T, H, width, pool = 50, 1 if flat else 3, 576 if flat else 128, 90
    x, w, pos, cs = _inputs(T, H, width, 128, 64, BF)
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(pool, generator=g)[:T]
    slots[[4, 9, 49]] = torch.tensor([-1, -5, -(1 << 40)])
    pos[4] = 1 << 40                        # of a padding token: no fault, no flag
    held = torch.randn(pool, H, width, generator=g).to(BF if quant is None else E4M3).to(DEV)
    if quant == "static":
        held = held.view(torch.uint8)
    sc = torch.rand(pool, H, generator=g).to(DEV) if quant == "head" else None
    before, sc_before = held.cpu(), sc.cpu() if quant == "head" else None
    view = (lambda t: t[:, 0]) if flat else (lambda t: t)
    scale = 0.02 if quant == "static" else None
    out, scales = mla.norm_rope(view(x), w, positions=pos, cos_sin=cs, rope_start=width - 64, quant=quant, scale=scale,
                                slots=slots.to(DEV), out=view(held), out_scales=None if sc is None else view(sc).contiguous()
                                if flat else sc)
    assert mla.device_status() == 0
    assert out.data_ptr() == held.data_ptr()
    real = (slots >= 0).nonzero().view(-1)
    pos[4] = 0
    y, top = _plain(x, w, 1e-6, pos, cs, width - 64, False)
    if quant:
        held, before = held.view(torch.uint8), before.view(torch.uint8)
    got = held.cpu()
    rows = slots[real]
    s = scales.cpu().view(pool, H) if quant == "head" else None
    _check(got[rows], None if s is None else s[rows], y[real], top[real], quant, scale)
    rest = torch.ones(pool, dtype=torch.bool)
    rest[rows] = False
    assert torch.equal(got[rest].view(torch.uint8), before[rest].view(torch.uint8))
    if s is not None:
        assert torch.equal(s[rest], sc_before[rest])


@pytest.mark.gpu
def test_bad_slots_and_positions_are_flagged():
    x, _, pos, cs = _inputs(6, 2, 64, 0, 32, BF)
    held = torch.zeros(4, 2, 64, dtype=BF, device=DEV)
    slots = torch.tensor([0, 4, 1, 1 << 50, 2, -1], device=DEV)
    mla.norm_rope(x, positions=pos, cos_sin=cs, slots=slots, out=held)
    assert mla.device_status() == mla.DEV_BAD_PAGE
    y, top = _plain(x, None, 0, pos, cs, 0, False)
    _check(held[:3], None, y[[0, 2, 4]], top[[0, 2, 4]], None, None)
    assert not held[3].any()
    bad = pos.clone()
    bad[1], bad[3] = -1, cs.shape[0]
    out = mla.norm_rope(x, positions=bad, cos_sin=cs)[0]
    assert mla.device_status() == mla.DEV_BAD_POSITION
    bad[1] = bad[3] = 0                     # which rotates by nothing
    y, top = _plain(x, None, 0, bad, cs, 0, False)
    _check(out, None, y, top, None, None)


@pytest.mark.gpu
def test_no_cache_rows():
    x = torch.ones(3, 1, 64, dtype=BF, device=DEV)
    mla.norm_rope(x, slots=torch.full((3,), -1, device=DEV), out=torch.empty(0, 1, 64, dtype=BF, device=DEV))
    assert mla.device_status() == 0
    assert mla.norm_rope(x[:0])[0].shape == (0, 1, 64)
    none, table = torch.zeros(0, dtype=torch.int64, device=DEV), torch.zeros(8, 32, device=DEV)
    for quant in (None, "head"):
        out, scales = mla.norm_rope(x[:0], positions=none, cos_sin=table, quant=quant)
        assert out.shape == (0, 1, 64) and (quant is None or scales.shape == (0, 1))
    out = torch.ones(5, 1, 64, dtype=BF, device=DEV)
    mla.norm_rope(x[:0], positions=none, cos_sin=table, slots=none, out=out)
    assert (out == 1).all()


@pytest.mark.gpu
def test_zero_infinite_and_nan_rows():
    x = torch.randn(5, 2, 128, generator=torch.Generator().manual_seed(1)).to(BF)
    x[0] = 0
    x[1, 0, 3] = math.inf
    x[2, 0, 7] = math.nan
    x[3] *= 2.0 ** 125                      # squares overflow float32
    x[4] *= 2.0 ** -120                     # and vanish beside eps
    x = x.to(DEV)
    w = torch.ones(128, dtype=BF, device=DEV)
    out = mla.norm_rope(x, w)[0].float().cpu()
    assert not out[0].any()
    assert out[1, 0, 3].isnan() and not out[1, 0, :3].any() and not out[1, 0, 4:].any()
    assert out[2, 0].isnan().all()
    y, top = _plain(x, w, 1e-6, None, None, 0, False)
    _check(out[3:].to(BF), None, y[3:], top[3:], None, None)
    _check(out[[1, 2]][:, 1].to(BF), None, y[[1, 2]][:, 1], top[[1, 2]][:, 1], None, None)
    codes, scales = mla.norm_rope(x, w, quant="head")
    assert scales[0].eq(1).all() and not codes[0].float().any()
    assert scales[2, 0].isnan() and codes[2, 0].float().isnan().all()
    _check(codes[3:], scales[3:], y[3:], top[3:], "head", None)


@pytest.mark.gpu
def test_other_stream_and_graph():
    x, w, pos, cs = _inputs(40, 4, 128, 128, 64, BF)
    want = mla.norm_rope(x, w, positions=pos, cos_sin=cs, quant="head")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = mla.norm_rope(x, w, positions=pos, cos_sin=cs, quant="head", stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = mla.norm_rope(x, w, positions=pos, cos_sin=cs, quant="head")
    x.copy_(x.flip(0))
    pos.copy_(pos.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(a[i].view(torch.uint8), want[i].view(torch.uint8))
        assert torch.equal(b[i].flip(0).contiguous().view(torch.uint8), want[i].view(torch.uint8))


@pytest.mark.gpu
def test_past_32_bits():
    T, H, width = 1 << 20, 2, 1032 - 8
    x = torch.ones(1, 1, 1, dtype=BF, device=DEV).expand(T, H, width).contiguous()
    x[-1] = torch.randn(H, width, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(BF)
    w = torch.ones(width, dtype=BF, device=DEV)
    pos, cs = torch.zeros(T, dtype=torch.int64, device=DEV), _table(100, 64).to(DEV)
    pos[-1] = 77
    slots = torch.arange(T, device=DEV) + 5
    held = torch.zeros(T + 5, H, width, dtype=BF, device=DEV)
    mla.norm_rope(x, w, positions=pos, cos_sin=cs, slots=slots, out=held)
    y, top = _plain(x[-1:], w, 1e-6, pos[-1:], cs, 0, False)
    _check(held[-1:], None, y, top, None, None)
    assert held[5:-1].eq(1).all() and not held[:5].any()
    assert mla.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [0, 1, 3])
@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("np_,start,rope", [(100, 64, 64), (0, 0, 128), (-1, 3, 4096), (1 << 62, -8, -16), (1, 1 << 30, 1 << 30)])
def test_without_positions_nothing_is_rotated(lib, np_, start, rope, flags, quant):
    # through the C ABI, where sizes of a rotation may be left in a call that has no positions
    T, H, width = 37, 3, 128
    x, w, _, _ = _inputs(T, H, width, width, 0, BF)
    out = torch.empty(T, H, width, dtype=BF if quant == 0 else E4M3, device=DEV)
    sc = torch.empty(T, H, device=DEV)
    scale = 0.05 if quant == 3 else 0.0
    st = lib.mla_norm_rope(x.data_ptr(), H * width, width, 0, w.data_ptr(), width, 1e-6, None, None, np_, start, rope, flags, T,
                           H, width, quant, scale, None, T, out.data_ptr(), H * width, width, sc.data_ptr(), None)
    assert st == mla.MLA_OK
    torch.cuda.synchronize()
    want, scales = mla.norm_rope(x, w, 1e-6, quant={0: None, 1: "head", 3: "static"}[quant], scale=scale or None)
    assert torch.equal(out.view(torch.uint8), want.view(torch.uint8))
    assert quant != 1 or torch.equal(sc, scales)
    y, top = _plain(x, w, 1e-6, None, None, 0, False)
    _check(out, scales, y, top, {0: None, 1: "head", 3: "static"}[quant], scale)
    assert mla.device_status() == 0


def _patterns(type_, width):
    """Every value of a 16-bit type, in rows of `width` (the last ones once more)."""
    bits = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16)
    return bits[torch.arange(-(-(1 << 16) // width) * width) % (1 << 16)].view(type_).view(-1, width)


def _codes(y, sc):
    """e4m3 codes of the float32 quotient y / sc (IEEE division, to nearest), saturating; every NaN one code."""
    q = (y / sc).clamp(-448, 448)
    return torch.where(q.isnan(), torch.tensor(0x7f, dtype=torch.uint8), q.to(E4M3).view(torch.uint8))


def _same_codes(got, want):
    got = got.cpu().view(torch.uint8)
    got = torch.where(got == 0xff, torch.tensor(0x7f, dtype=torch.uint8), got)
    assert torch.equal(got, want)


SCALES = [0.03, 0.05, 1 / 3, 1.0, 0.7853982, 447.0, 3.0e-5, 1.1e18, 3.0e38, 2.0 ** -64, 1.9e19, 5.0e-20, 2.0 ** -126, 1.3e-38,
          math.pi * 2.0 ** -100]


@pytest.mark.gpu
@pytest.mark.parametrize("type_", [BF, FP])
@pytest.mark.parametrize("width", [8, 40, 128, 192, 576, 1024])
def test_codes_with_a_given_scale_are_those_of_the_quotient(width, type_):
    # no norm and no rotation: y is x, so a code is known to the bit, ties among them
    x = _patterns(type_, width)
    for scale in SCALES:
        sc = torch.tensor(scale, dtype=torch.float32)
        want = _codes(x.float(), sc)
        _same_codes(mla.norm_rope(x.to(DEV), quant="static", scale=scale)[0], want)
    want = _codes(x.float(), torch.tensor(0.03))
    heads = x[:x.shape[0] // 2 * 2].view(-1, 2, width)
    _same_codes(mla.norm_rope(heads.to(DEV), quant="static", scale=0.03)[0], want[:heads.shape[0] * 2].view_as(heads))
    many = x.repeat(-(-12000 // x.shape[0]), 1)
    _same_codes(mla.norm_rope(many.to(DEV), quant="static", scale=0.03)[0], want.repeat(many.shape[0] // x.shape[0], 1))
    if width > 40:                  # beside a norm and a rotation: columns 16 to 24 and the last ones are x's
        g, pos = torch.ones(16, dtype=type_, device=DEV), torch.zeros(x.shape[0], dtype=torch.int64, device=DEV)
        for pairs in (False, True):
            got = mla.norm_rope(x.to(DEV), g, positions=pos, cos_sin=_table(1, 16).to(DEV), rope_start=24, interleaved=pairs,
                                quant="static", scale=0.03)[0]
            mine = torch.tensor([*range(16, 24), *range(40, width)])
            _same_codes(got.cpu().view(torch.uint8)[:, mine], want[:, mine])


@pytest.mark.gpu
@pytest.mark.parametrize("k_scale", [0.03, 0.05, 1 / 3, 1.0, 447.0, 2.0 ** -120, 3.0e38])
def test_the_two_writers_of_a_cache_agree(k_scale):
    # kv_append and norm_rope into the same latent rows: every bf16 value
    x = _patterns(BF, 576).to(DEV)
    slots = torch.randperm(x.shape[0] + 3, generator=torch.Generator().manual_seed(1))[:x.shape[0]].to(DEV)
    a, b = (torch.zeros(x.shape[0] + 3, 576, dtype=torch.uint8, device=DEV) for _ in range(2))
    mla.kv_append(a, x[:, :512].contiguous(), x[:, 512:].contiguous(), slots, k_scale)
    mla.norm_rope(x, quant="static", scale=k_scale, slots=slots, out=b)
    nan = x.isnan().cpu()
    a, b = a[slots].cpu(), b[slots].cpu()
    assert torch.equal(a[~nan], b[~nan])
    assert (b[nan] & 0x7f).eq(0x7f).all()


@pytest.mark.gpu
@pytest.mark.parametrize("pairs", [False, True])
def test_quotients_beside_a_tie(pairs):
    # Any float32 comes through the rotation: 1 * c - 0 * s.  With r = RN(1 / b) the quotient is q0 = RN(a r) corrected
    # once by its remainder.  For a >= b (significands) q0 is within one unit and the result is RN(a / b) (Markstein);
    # for a < b it is within 1.5, and the corrected one off, before its rounding, by the remainder (1.5 x 2^-24 b) times
    # r's error (2^-25) and the remainder's own (2^-47) times r: with b times that R = 2^49 |a - b m| is 6 + 4 at most.
    # A code can differ from the division's only where a / b is so near to half a unit beside a border t = k / 64 of two
    # codes: A 2^26 = B (k 2^20 +- 1 or 2) + R.  All such A and B, with room in R:
    found = []
    for k in range(16, 64):
        for by in (-2, -1, 1, 2):
            m = (k << 20) + by
            for r in range(-24, 25):
                step = 1 << 26
                d = math.gcd(m, step)
                if r == 0 or r % d:
                    continue
                b = (-r // d * pow(m // d, -1, step // d)) % (step // d)
                while b < 1 << 24:
                    a = (b * m + r) >> 26
                    if b >= 1 << 23 and 0 < a < 1 << 24:
                        found.append((a, b))
                    b += step // d
    assert len(found) > 500
    for a, b in found:
        width = 24                          # eight columns are not rotated, so codes are the quotient's
        y = torch.tensor([[float(a) * 2.0 ** -e for e in range(18, 26)]], dtype=torch.float32)      # quotients t * 2^(23 - e)
        scale = float(b) * 2.0 ** -23
        cs = torch.cat([y, torch.zeros_like(y)], 1).to(DEV)
        x = torch.zeros(1, 1, width, dtype=BF)
        if pairs:
            x[..., 0:16:2] = 1
        else:
            x[..., :8] = 1
        pos = torch.zeros(1, dtype=torch.int64, device=DEV)
        out = mla.norm_rope(x.to(DEV), positions=pos, cos_sin=cs, interleaved=pairs, quant="static", scale=scale)[0].cpu()[0, 0]
        got = out.view(torch.uint8)[0:16:2] if pairs else out.view(torch.uint8)[:8]
        assert torch.equal(got, _codes(y[0], torch.tensor(scale, dtype=torch.float32))), (a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [None, "head"])
def test_one_row_whose_heads_lie_far_apart(quant):
    # one token of heads kept [H, T, D]: each stride within the limit, the last head past 2^30 elements
    H, T, width = 96, 1 << 16, 192
    base = torch.empty(H, T, width, dtype=BF, device=DEV)
    x, w, pos, cs = _inputs(1, H, width, width, 64, BF)
    base[:, 77] = x[0]
    far = base[:, 77:78].transpose(0, 1)
    assert far.stride(1) <= 1 << 30 < (H - 1) * far.stride(1)
    got = mla.norm_rope(far, w, positions=pos, cos_sin=cs, rope_start=128, quant=quant)
    want = mla.norm_rope(x, w, positions=pos, cos_sin=cs, rope_start=128, quant=quant)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))
    assert quant is None or torch.equal(got[1], want[1])
    if quant is None:
        mla.norm_rope(far, w, positions=pos, cos_sin=cs, rope_start=128, out=far)
        assert torch.equal(base[:, 77], want[0][0])
