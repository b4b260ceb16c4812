"""The operators in front of attend run together, as a server uses them: new
tokens' latents and index keys into their caches, the projection's heads to
the absorbed query, index scores, every query row's page list, attention over
it.  Checked against the same steps in 64 bits."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn
H, HI, K_SCALE, I_SCALE, SCALE = 12, 16, 0.03, 0.05, 1 / math.sqrt(192.0)


def _table(n, d):
    freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    a = torch.arange(n, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


class _Server:
    """Caches, weights and a step over them."""

    def __init__(self, lengths, qlen, fp8=False):
        g = torch.Generator(device=DEV).manual_seed(len(lengths) + qlen)
        self.g, self.lengths, self.qlen, self.R, self.fp8 = g, lengths, qlen, len(lengths), fp8
        total = sum(lengths)
        self.pool = total + 100
        self.cs = _table(max(lengths) + 1, 64)
        self.kv = torch.zeros(self.pool, 576, dtype=torch.uint8, device=DEV)
        self.keys = torch.zeros(self.pool, 128, dtype=torch.uint8, device=DEV)
        self.pages = torch.randperm(self.pool, generator=g, device=DEV)[:total].to(torch.int32)
        self.indptr = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device=DEV)
        self.w_c = (1 + 0.1 * self.rand(512)).to(BF)
        self.w_i = (1 + 0.1 * self.rand(128)).to(BF)
        self.w_uk = (self.rand(H, 128, 512) / 16).to(BF)
        self.w_uv = (self.rand(H, 128, 512) / math.sqrt(512)).to(BF)
        self.host_lengths = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        # every token but a request's last qlen is already cached
        self.where = torch.cat([torch.arange(n, device=DEV) for n in lengths])
        self.append(self.pages.long(), self.where, (self.rand(total, 2112)).to(BF))

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV)

    def append(self, slots, positions, proj):
        """proj: a fused projection, 512 + 64 latent and 128 index columns of it."""
        kw = dict(positions=positions, cos_sin=self.cs, slots=slots, quant="static")
        mla.norm_rope(proj[:, 1536:2112], self.w_c, rope_start=512, scale=K_SCALE, out=self.kv, **kw)
        mla.norm_rope(proj[:, :128], self.w_i, rope_start=64, scale=I_SCALE, out=self.keys, **kw)

    def step(self, heads, index, weights, gate, topk, block, recent, sinks):
        """One decode step of qlen rows a request: (out, latent, lse, and what led there)."""
        pos = torch.cat([torch.arange(n - self.qlen, n, device=DEV).clamp(min=0) for n in self.lengths])
        q_scale = 0.05 if self.fp8 else 1.0
        q = mla.query_absorb(heads, self.w_uk, positions=pos, cos_sin=self.cs, q_scale=q_scale if self.fp8 else None)
        qi, qs = mla.norm_rope(index, positions=pos, cos_sin=self.cs, rope_start=64, quant="head")
        scores = mla.index_scores(qi, weights, self.keys, self.pages, self.indptr, q_scales=qs, scale=I_SCALE, qlen=self.qlen,
                                  causal=True)
        pages, indptr = mla.index_select(scores, self.pages, self.indptr, topk, block=block, recent=recent, sinks=sinks,
                                         causal=True)
        ns, st = mla.choose_splits(self.R * self.qlen, 1, H, max_len=topk * block)
        o, lse = mla.attend(q, self.kv, pages, indptr, SCALE, K_SCALE, ns, st, q_scale=q_scale)
        latent, lse = mla.merge(o, lse)
        out = mla.value_gate(latent, self.w_uv, gate, self.host_lengths, self.qlen)
        return out, latent, lse, q, qi, qs, scores, pages, indptr


def _inputs(s):
    S = s.R * s.qlen
    return (s.rand(S, H, 192).to(BF), s.rand(S, HI, 128).to(BF), s.rand(S, HI), s.rand(S, H * 128).to(BF))


def _attention(q, kv, rows):
    k = kv[rows.long()].view(E4M3).double() * K_SCALE
    x = q.double() @ k.T * SCALE
    ls = torch.logsumexp(x, 1)
    return torch.exp(x - ls[:, None]) @ k[:, :512], ls


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths,qlen,topk,block,recent,sinks", [
    ([900, 1, 70, 3000], 1, 128, 1, 16, 4),
    ([900, 7, 70, 3000], 2, 6, 32, 1, 1),
    ([500, 0, 65, 2], 4, 64, 1, 0, 0),
])
def test_sparse_step(lengths, qlen, topk, block, recent, sinks, fp8):
    mla.build()
    s = _Server(lengths, qlen, fp8)
    heads, index, weights, gate = _inputs(s)
    out, latent, lse, q, qi, qs, scores, pages, indptr = s.step(heads, index, weights, gate, topk, block, recent, sinks)
    assert mla.device_status() == 0
    qd = q.view(E4M3).double() * 0.05 if fp8 else q.double()
    starts, lists = s.indptr.tolist(), indptr.tolist()
    for r, n in enumerate(lengths):
        own = s.pages[starts[r]:starts[r + 1]]
        keys = s.keys[own.long()].view(E4M3).double() * I_SCALE
        for tq in range(qlen):
            t = r * qlen + tq
            seen = max(0, n - qlen + tq + 1)
            # the scores, from the codes and scales as they are
            qt = qi[t].view(torch.uint8).view(E4M3).double() * qs[t].double()[:, None]
            ref = torch.relu(qt @ keys.T).T @ weights[t].double()
            mag = (qt.abs() @ keys.abs().T).T @ weights[t].double().abs()
            got = scores[tq, starts[r]:starts[r + 1]]
            assert torch.all((got[:seen].double() - ref[:seen]).abs() <= 2.0 ** -16 * mag[:seen])
            assert got[seen:].eq(-math.inf).all()
            # the list, from the scores as they are
            mine = pages[lists[t]:lists[t + 1]]
            assert mine.numel() == min(seen, topk * block) or block > 1
            count = -(-seen // block)
            best = torch.nn.functional.pad(got[:seen], (0, count * block - seen), value=-math.inf).view(count, block).amax(1) \
                if count else got[:0]
            where = {p: i for i, p in enumerate(own.tolist())}
            chosen = sorted({where[p] // block for p in mine.tolist()})
            assert len(chosen) == min(count, topk)
            assert [where[p] for p in mine.tolist()] == [b * block + i for b in chosen for i in range(block) if b * block + i < seen]
            must = set(range(count - min(recent, len(chosen)), count))
            must |= set(range(min(sinks, len(chosen) - len(must))))
            assert must <= set(chosen)
            free = [b for b in chosen if b not in must]
            left = [b for b in range(count) if b not in chosen]
            if free and left:
                assert best[free].min() >= best[left].max()
            # the attention over it
            if seen == 0:
                assert lse[t].eq(-math.inf).all() and not latent[t].any()
                continue
            lat, ls = _attention(qd[t], s.kv, mine)
            assert ((latent[t].double() - lat).abs() <= 2e-2 + 2e-2 * lat.abs()).all()
            assert ((lse[t].double() - ls).abs() <= 1e-3).all()
            val = torch.einsum("hc,hvc->hv", latent[t].double(), s.w_uv.double()).flatten()
            val = val * torch.sigmoid(gate[t].double())
            assert ((out[t].double() - val).abs() <= 2e-2 + 2e-2 * val.abs()).all()


def test_all_tokens_selected_is_the_dense_step():
    mla.build()
    s = _Server([300, 40, 129], 3)
    heads, index, weights, gate = _inputs(s)
    out, latent, lse, q, _, _, _, pages, indptr = s.step(heads, index, weights, gate, 512, 1, 0, 0)
    ns, st = mla.choose_splits(3, 3, H, max_len=300)
    o, dense = mla.attend(q, s.kv, s.pages, s.indptr, SCALE, K_SCALE, ns, st, qlen=3, causal=True)
    lat, dense = mla.merge(o, dense)
    assert ((lse - dense).abs() <= 2e-3).all()          # two results, each within 1e-3 of the exact one
    assert ((latent.float() - lat.float()).abs() <= 4e-2 + 4e-2 * lat.float().abs()).all()


def test_captured_step():
    mla.build()
    s = _Server([600, 90], 2)
    ins = _inputs(s)
    want = s.step(*ins, 64, 1, 8, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    new = _inputs(s)
    hold = [x.clone() for x in new]
    with torch.cuda.graph(graph):
        got = s.step(*hold, 64, 1, 8, 2)
    for a, b in zip(hold, ins):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert mla.device_status() == 0
