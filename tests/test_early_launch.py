"""Kernels that start while the one before them on the stream still runs see
what that one writes: every input changed by the kernel just before the call,
on the call's stream or on another joined by an event, eager and captured."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def _table(n, d, g):
    return torch.randn(n, d, generator=g, device=DEV)


def _norm_rope(g):
    T, H, D = 300, 6, 128
    return dict(x=torch.randn(T, H, D, generator=g, device=DEV).to(BF), weight=(1 + torch.rand(D, generator=g, device=DEV)).to(BF),
                positions=torch.randint(0, 50, (T,), generator=g, device=DEV), cos_sin=_table(50, 64, g),
                slots=torch.randperm(T, generator=g, device=DEV))


def _run_norm_rope(s):
    out = torch.zeros_like(s["x"])
    return mla.norm_rope(s["x"], s["weight"], positions=s["positions"], cos_sin=s["cos_sin"], slots=s["slots"], out=out)[0]


def _query_absorb(g):
    T, H = 200, 12
    return dict(q=torch.randn(T, H, 192, generator=g, device=DEV).to(BF),
                w_uk=torch.randn(H, 128, 512, generator=g, device=DEV).mul(0.1).to(BF),
                positions=torch.randint(0, 50, (T,), generator=g, device=DEV), cos_sin=_table(50, 64, g))


def _run_query_absorb(s):
    return mla.query_absorb(s["q"], s["w_uk"], positions=s["positions"], cos_sin=s["cos_sin"])


def _indptr(R, total, g):
    cut = torch.sort(torch.randint(0, total + 1, (R - 1,), generator=g, device=DEV)).values
    return torch.cat([torch.zeros(1, device=DEV), cut, torch.full((1,), total, device=DEV)]).to(torch.int32)


def _index_scores(g):
    R, qlen, H, total = 40, 2, 32, 9000
    code = lambda *s: torch.randn(*s, generator=g, device=DEV).mul(20).to(E4M3)  # noqa: E731
    return dict(q=code(R * qlen, H, 128), weights=torch.randn(R * qlen, H, generator=g, device=DEV), k=code(total, 128),
                pages=torch.randperm(total, generator=g, device=DEV).to(torch.int32), indptr=_indptr(R, total, g),
                q_scales=torch.rand(R * qlen, H, generator=g, device=DEV))


def _run_index_scores(s):
    return mla.index_scores(s["q"], s["weights"], s["k"], s["pages"], s["indptr"], q_scales=s["q_scales"], qlen=2, causal=True)


def _index_select(g, R=40, qlen=2, total=9000):
    return dict(scores=torch.randn(qlen, total, generator=g, device=DEV),
                pages=torch.randperm(total, generator=g, device=DEV).to(torch.int32), indptr=_indptr(R, total, g))


def _index_select_many(g):
    return _index_select(g, 700, 2, 9000)       # more rows than 1,024: the indptr of a kernel before


def _index_select_long(g):
    return _index_select(g, 3, 1, 90000)        # clusters


def _run_index_select(s):
    return torch.cat(mla.index_select(s["scores"], s["pages"], s["indptr"], 50, recent=2, causal=True))


def _value_gate(g):
    S, H = 24, 12
    return dict(o=torch.randn(3, S, H, 512, generator=g, device=DEV).to(BF), lse=torch.randn(3, S, H, generator=g, device=DEV),
                gate=torch.randn(S, H * 128, generator=g, device=DEV).to(BF),
                lengths=torch.randint(0, 3, (S,), generator=g, device=DEV).to(torch.int32))


def _run_value_gate(s):
    w = _run_value_gate.w
    return mla.merge_value_gate(s["o"], s["lse"], w, s["gate"], s["lengths"], 1)


CASES = {"norm_rope": (_norm_rope, _run_norm_rope), "query_absorb": (_query_absorb, _run_query_absorb),
         "index_scores": (_index_scores, _run_index_scores), "index_select": (_index_select, _run_index_select),
         "index_select_many": (_index_select_many, _run_index_select),
         "index_select_long": (_index_select_long, _run_index_select),
         "merge_value_gate": (_value_gate, _run_value_gate)}


def _write(state, new, names):
    """By kernels (a copy of equal types is none), `names` in order."""
    for n in names:
        a, b = _bytes(state[n]), _bytes(new[n])
        torch.where(torch.ones((), dtype=torch.bool, device=DEV), b, a, out=a)


@pytest.mark.parametrize("name", CASES)
def test_inputs_written_just_before(name):
    mla.build()
    make, run = CASES[name]
    g = torch.Generator(device=DEV).manual_seed(5)
    _run_value_gate.w = torch.randn(12, 128, 512, generator=g, device=DEV).mul(0.05).to(BF)
    sets = [make(g) for _ in range(2)]
    want = []
    for s in sets:
        torch.cuda.synchronize()
        want.append(run(s).clone())
    assert not torch.equal(want[0].view(torch.uint8), want[1].view(torch.uint8))
    names = list(sets[0])
    state = {n: t.clone() for n, t in sets[0].items()}
    side = torch.cuda.Stream()
    main = torch.cuda.current_stream()

    def step(new, last, joined):
        order = [n for n in names if n != last] + [last]        # `last` by the kernel just before the call
        if joined:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                _write(state, new, order)
            torch.mul(state[names[0]].float().sum(), 2.0)       # a kernel of this stream before the call
            main.wait_stream(side)
        else:
            _write(state, new, order)
        return run(state)

    for joined in (False, True):
        for i, last in enumerate(names * 3):
            got = step(sets[i % 2], last, joined)
            assert torch.equal(got.view(torch.uint8), want[i % 2].view(torch.uint8)), (last, joined)
    for joined in (False, True):
        for last in names:
            source = {n: t.clone() for n, t in sets[0].items()}
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                main = torch.cuda.current_stream()
                got = step(source, last, joined)
            main = torch.cuda.current_stream()
            for i in (1, 0, 1):
                for n in names:
                    source[n].copy_(sets[i][n])
                graph.replay()
                assert torch.equal(got.view(torch.uint8), want[i].view(torch.uint8)), (last, joined, "captured")
    assert mla.device_status() == 0
