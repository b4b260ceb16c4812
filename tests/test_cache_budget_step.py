"""The operators around a decode step run together, as a server uses them:
norm the new tokens' latents, append them, attend, gather the tokens'
weights, cut the page lists to a budget and decode the next step from what
is left.  Checked against the same steps in 64 bits."""

import math

import pytest
import torch

import mla_decode_paged_gb300 as mla

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _attention(q, kv, pages, lengths, sc, kv_scale):
    lat, lse, mass, at = [], [], [], 0
    for r, n in enumerate(lengths):
        k = kv[pages[at:at + n].long()].view(torch.float8_e4m3fn).double() * kv_scale
        s = q[r].double() @ k.T * sc
        ls = torch.logsumexp(s, 1)
        p = torch.exp(s - ls[:, None])
        lat.append(p @ k[:, :512])
        lse.append(ls)
        mass.append(p.sum(0))
        at += n
    return torch.stack(lat), torch.stack(lse), torch.cat(mass)


def test_two_steps_with_eviction_between():
    mla.build()
    R, heads, budget, scale, kv_scale = 5, 12, 96, 1 / math.sqrt(192.0), 0.5
    lengths = [300, 97, 40, 150, 96]
    g = torch.Generator(device=DEV).manual_seed(0)
    total, pool = sum(lengths), 1000
    pages = torch.randperm(pool, generator=g, device=DEV)[:total].to(torch.int32)
    indptr = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device=DEV)
    kv = torch.zeros(pool, 576, dtype=torch.uint8, device=DEV)

    # the tokens' latents: a 576-wide projection whose first 512 columns are normed
    proj = torch.randn(total, 576, generator=g, device=DEV).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(512, generator=g, device=DEV)).to(torch.bfloat16)
    kv_c, _, _ = mla.add_rms_norm(proj[:, :512], w, 1e-6)
    mla.kv_append(kv, kv_c, proj[:, 512:], pages.long(), kv_scale)

    def step(pages, indptr, lengths, weights, seed):
        q = torch.randn(R, heads, 576, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).mul_(2)
        q = q.to(torch.bfloat16)
        ns, st = mla.choose_splits(R, 1, heads, lengths=lengths)
        o, lse = mla.attend(q, kv, pages, indptr, scale, kv_scale, ns, st)
        latent, lse = mla.merge(o, lse)
        mass = mla.token_weights(q, kv, pages, indptr, scale, kv_scale, lse, weights=weights, decay=0.5)
        return q, latent, lse, mass

    q, latent, lse, mass = step(pages, indptr, lengths, None, 1)
    ref_lat, ref_lse, ref_mass = _attention(q, kv, pages, lengths, scale, kv_scale)
    # the step's own stated tolerances; the weights follow the LSE's error, 1e-3
    assert ((latent.double() - ref_lat).abs() <= 2e-2 + 2e-2 * ref_lat.abs()).all()
    assert ((lse.double() - ref_lse).abs() <= 1e-3).all()
    assert ((mass.double() - ref_mass).abs() <= 2e-3 * ref_mass).all()

    pages2, indptr2, mass2 = mla.kv_evict(pages, indptr, mass, budget, recent=16, sinks=2)
    kept = [min(n, budget) for n in lengths]
    assert indptr2.tolist() == [0] + torch.tensor(kept).cumsum(0).tolist()
    assert sorted(pages2.tolist()) == sorted(pages.tolist())
    at = 0
    for r, n in enumerate(lengths):                  # the heaviest stay
        here = mass[at:at + n]
        mine = pages2[int(indptr2[r]):int(indptr2[r + 1])]
        stays = torch.isin(pages[at:at + n], mine)
        mid = slice(2, n - 16)
        if n > budget:
            assert here[mid][stays[mid]].min() >= here[mid][~stays[mid]].max()
            assert stays[:2].all() and stays[n - 16:].all()
        at += n

    # the next step reads the compacted lists as they are (freed rows behind them)
    q, latent, lse, mass3 = step(pages2, indptr2, kept, mass2, 2)
    ref_lat, ref_lse, ref_mass = _attention(q, kv, pages2, kept, scale, kv_scale)
    K = sum(kept)
    assert ((latent.double() - ref_lat).abs() <= 2e-2 + 2e-2 * ref_lat.abs()).all()
    assert ((mass3[:K].double() - (ref_mass + 0.5 * mass2[:K].double())).abs() <= 2e-3 * (ref_mass + mass2[:K])).all()

    # and the value projection with the tenants' adapters
    lengths_d = torch.tensor(kept, dtype=torch.int32, device=DEV)
    w_uv = torch.randn(heads, 128, 512, generator=g, device=DEV).mul_(0.044).to(torch.bfloat16)
    gate = torch.randn(R, heads * 128, generator=g, device=DEV).to(torch.bfloat16)
    la = torch.randn(2, 16, 512, generator=g, device=DEV).mul_(0.044).to(torch.bfloat16)
    lb = torch.randn(2, heads * 128, 16, generator=g, device=DEV).mul_(0.2).to(torch.bfloat16)
    ad = torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32, device=DEV)
    sc = torch.tensor([1.0, 0.5], device=DEV)
    out = mla.value_gate_lora(latent, w_uv, gate, lengths_d, la, lb, ad, sc)
    x = latent.double()
    val = torch.einsum("rhc,hvc->rhv", x, w_uv.double())
    for r, a in enumerate(ad.tolist()):
        if a >= 0:
            val[r] += float(sc[a]) * torch.einsum("hk,hvk->hv", x[r] @ la[a].double().T, lb[a].double().view(heads, 128, 16))
    ref = val.reshape(R, -1) * torch.sigmoid(gate.double())
    assert ((out.double() - ref).abs() <= 2.0**-8 * ref.abs() + 1e-4).all()
    assert mla.device_status() == 0
