"""The operators in front of attend, with the cases they are measured on.

Four entry points of the package, from the projections' outputs to what attend reads:

  norm_rope      norm and position rotation of every head in one pass, 16 or 8 bits, into a tensor or a cache
  query_absorb   the query's W_UK product beside its rotated columns: the query that attend takes
  index_scores   a cheap score of every cached token for every query row
  index_select   the page list of the best-scored blocks of tokens, a list a query row: the pages that attend takes

``run`` computes an operator in its plain form (elementary torch operations in 32
bits) or, with ``own`` true, by the package's call.
"""

import math

import torch

own = False

D_NOPE, D_ROPE, D_LATENT, D_QK, D_INDEX, E4M3_MAX = 128, 64, 512, 576, 128, 448.0
DEV = "cuda"


# --------------------------------------------------------------------- cases


def _norm_rope(tokens, heads, width, norm=0, rope=0, start=0, interleaved=False, quant="none", pool=0, gap=0,
               type="bf16"):
    return {"op": "norm_rope", "tokens": tokens, "heads": heads, "width": width, "norm": norm, "rope": rope,
            "start": start, "interleaved": interleaved, "quant": quant, "pool": pool, "gap": gap, "type": type}


def _absorb(tokens, heads, rope="halves", out="bf16", gap=0):
    return {"op": "query_absorb", "tokens": tokens, "heads": heads, "rope": rope, "out": out, "gap": gap}


def _scores(requests, qlen, heads, lo, hi, causal=False, q_scales=True, deal=1):
    return {"op": "index_scores", "requests": requests, "qlen": qlen, "heads": heads, "lo": lo, "hi": hi,
            "causal": causal, "q_scales": q_scales, "deal": deal}


def _select(requests, qlen, lo, hi, topk, block=1, recent=0, sinks=0, causal=False, deal=1):
    return {"op": "index_select", "requests": requests, "qlen": qlen, "lo": lo, "hi": hi, "topk": topk, "block": block,
            "recent": recent, "sinks": sinks, "causal": causal, "deal": deal}


def listed():
    return [
        # The index queries of a decode step of 64 requests: 64 heads, rotated in front, a scale a head: latency counts.
        dict(_norm_rope(64, 64, 128, rope=64, quant="head"), name="rope_index_query"),
        # The latent rows of a prefill chunk, normed, rotated behind and written to their slots of the fp8 cache.
        dict(_norm_rope(16384, 1, 576, norm=512, rope=64, start=512, quant="static", pool=65536, gap=1536),
             name="rope_latent_cache"),
        # Query heads normed and rotated over a prefill chunk, 96 heads of 192.
        dict(_norm_rope(4096, 96, 192, norm=192, rope=64, start=128, interleaved=True), name="rope_prefill_heads"),
        # One decode step of 64 requests, 12 local heads: latency counts.
        dict(_absorb(64, 12), name="absorb_decode"),
        # Speculative rows: 256 requests x 8 rows, 12 heads.
        dict(_absorb(2048, 12, rope="pairs"), name="absorb_ragged"),
        # A prefill chunk of 4096 tokens with all 96 heads on one GPU, for the fp8 query.
        dict(_absorb(4096, 96, out="e4m3"), name="absorb_prefill_heads96"),
        # One decode step, 64 requests of 1K to 8K tokens, 64 index heads.
        dict(_scores(64, 1, 64, 1024, 8192), name="scores_decode"),
        # Speculative decoding: 4 rows a request under the causal mask, 4K to 32K tokens, 32 index heads.
        dict(_scores(128, 4, 32, 4096, 32768, causal=True), name="scores_spec"),
        # Long contexts: 32 requests of 32K, 64 index heads.
        dict(_scores(32, 1, 64, 32768, 32768), name="scores_long"),
        # 64 requests of 1K to 8K tokens, the best 2048 of each.
        dict(_select(64, 1, 1024, 8192, 2048), name="select_decode"),
        # One interactive request, the best 2048 of 128K tokens: latency counts.
        dict(_select(1, 1, 131072, 131072, 2048), name="select_one_long"),
        # Speculative rows over 4K to 32K tokens by blocks of 64: 32 blocks, the first and the last two among them.
        dict(_select(128, 4, 4096, 32768, 32, block=64, recent=2, sinks=1, causal=True), name="select_spec_blocks"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "absorb", "scores", "select"])
    if op == "rope":
        width = 8 * _log_int(rng, 4, 128)
        rope = rng.choice([0, 16, 32, 64, 64, 128])
        rope = rope if rope <= width else 16
        norm = rng.choice([width, width - rope, 0]) or (0 if rope else width)
        heads = rng.choice([1, 1, 2, 8, 12, 24, 64, 96])
        tokens = _log_int(rng, 1, min(16384, 4096 * 96 * 192 // (width * heads)))
        pool = rng.choice([0, 0, tokens + _log_int(rng, 1, 4096)])
        if pool * heads * width > 1 << 27:
            pool = 0
        return _norm_rope(tokens, heads, width, norm, rope, rng.choice([0, width - rope]), rng.choice([False, True]),
                          rng.choice(["none", "head", "static"]), pool, 8 * rng.choice([0, 0, 1, 24]),
                          rng.choice(["bf16", "bf16", "fp16"]))
    if op == "absorb":
        heads = rng.choice([1, 5, 8, 12, 16, 24, 32, 64, 96, 128])
        return _absorb(_log_int(rng, 1, min(16384, 4096 * 96 // heads)), heads,
                       rng.choice(["halves", "pairs", "none"]), rng.choice(["bf16", "bf16", "e4m3"]),
                       8 * rng.choice([0, 0, 1, 16]))
    if op == "scores":
        qlen, heads = rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([1, 4, 8, 12, 16, 24, 32, 48, 64, 96, 128])
        # at most the tokens and the token-row products of the largest listed case, half of it on average
        most = min(2300000, 300000000 // (qlen * heads))
        requests = _log_int(rng, 1, 128)
        hi = _log_int(rng, 33, max(34, min(131072, most // requests)))
        return _scores(requests, qlen, heads, _log_int(rng, max(1, hi // 8), hi), hi, rng.choice([False, True]),
                       rng.choice([False, True]), rng.randrange(1 << 16))
    block = 1 << rng.choice([0, 0, 0, 3, 4, 5, 6, 7, 8])
    qlen = rng.choice([1, 1, 2, 4, 8])
    requests = _log_int(rng, 1, 256)
    hi = _log_int(rng, 100, min(131072, 9400000 // (requests * qlen)))
    topk = _log_int(rng, 1, max(2, min(4096, hi // block)))
    return _select(requests, qlen, _log_int(rng, max(1, hi // 100), hi), hi, topk, block,
                   rng.randrange(0 if block == 1 else 1, topk // 4 + 2), rng.randrange(0, 5), rng.choice([False, True]),
                   rng.randrange(1 << 16))


def _lengths(case):
    """Tokens per request, from the case alone (so that a case has one size): uniform over [lo, hi], or over its
    logarithm where it spans more than a factor of ten."""
    lo, hi = case["lo"], case["hi"]
    u = torch.rand(case["requests"], generator=torch.Generator().manual_seed(case["deal"]), dtype=torch.float64)
    if hi > 10 * lo:
        x = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo)))
    else:
        x = lo + u * (hi + 1 - lo)
    return x.to(torch.int64).clamp_(lo, hi)


def _visible(lengths, qlen, causal):
    """Tokens that each query row sees, [requests, qlen]."""
    seen = lengths[:, None].expand(-1, qlen)
    if causal:
        seen = (seen - qlen + 1 + torch.arange(qlen, device=lengths.device)).clamp(min=0)
    return seen


def work(case):
    op = case["op"]
    if op == "norm_rope":
        t, h, d = case["tokens"], case["heads"], case["width"]
        out = 2 if case["quant"] == "none" else 1
        bytes_ = t * h * d * (2 + out) + 2 * case["norm"] + t * (4 * case["rope"] + (8 if case["rope"] else 0))
        bytes_ += (8 * t if case["pool"] else 0) + (4 * t * h if case["quant"] == "head" else 0)
        return {"bytes": bytes_, "flops": t * h * (4 * case["norm"] + 3 * case["rope"])}
    if op == "query_absorb":
        t, h = case["tokens"], case["heads"]
        bytes_ = t * h * ((D_NOPE + D_ROPE) * 2 + D_QK * (2 if case["out"] == "bf16" else 1)) + h * D_NOPE * D_LATENT * 2
        return {"bytes": bytes_ + (t * (8 + 4 * D_ROPE) if case["rope"] != "none" else 0),
                "flops": 2 * t * h * D_NOPE * D_LATENT}
    lengths = _lengths(case)
    total, rows = int(lengths.sum()), case["requests"] * case["qlen"]
    if op == "index_scores":
        return {"bytes": total * (D_INDEX + 4 + 4 * case["qlen"]) + rows * case["heads"] * (D_INDEX + 8),
                "flops": 2 * D_INDEX * total * case["qlen"] * case["heads"]}
    seen = _visible(lengths, case["qlen"], case["causal"])
    kept = torch.minimum(seen, torch.tensor(case["topk"] * case["block"]))
    return {"bytes": 4 * int(seen.sum()) + 8 * int(kept.sum()) + 4 * rows, "flops": 4 * int(seen.sum())}


# -------------------------------------------------------------------- inputs


def _indptr(lengths):
    indptr = torch.zeros(lengths.numel() + 1, dtype=torch.int64)
    indptr[1:] = torch.cumsum(lengths, 0)
    return indptr.to(torch.int32).to(DEV)


def _table(positions, dim):
    """Cosines, then sines of `positions` positions' angles, base 10000, formed in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=DEV) / dim)
    angle = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _positions(tokens, far, g):
    """Prompts of a chunk one after another, or the last tokens of as many requests."""
    if tokens > 1024:
        return torch.arange(tokens, device=DEV) + far - tokens
    return torch.randint(0, far, (tokens,), generator=g, device=DEV)


def _prepare_norm_rope(case, g):
    t, h, d, gap = case["tokens"], case["heads"], case["width"], case["gap"]
    type_ = {"bf16": torch.bfloat16, "fp16": torch.float16}[case["type"]]
    far = 32768
    s = {"x": torch.randn(t, h * d + gap, generator=g, device=DEV).to(type_)[:, gap:].unflatten(1, (h, d)),
         "weight": None, "eps": 1e-6, "positions": None, "cos_sin": None, "start": case["start"],
         "interleaved": case["interleaved"], "quant": None if case["quant"] == "none" else case["quant"],
         "scale": 0.03 if case["quant"] == "static" else None, "slots": None, "out": None, "out_scales": None}
    if case["norm"]:
        s["weight"] = (1 + 0.1 * torch.randn(case["norm"], generator=g, device=DEV)).to(type_)
    if case["rope"]:
        s["positions"], s["cos_sin"] = _positions(t, far, g), _table(far, case["rope"])
    if case["pool"]:
        s["slots"] = torch.randperm(case["pool"], generator=g, device=DEV)[:t]
        if t > 4:       # a padding row of a padded batch
            s["slots"][t // 2] = -1
        held = torch.randn(case["pool"], h, d, generator=g, device=DEV)
        s["out"] = held.to(type_ if s["quant"] is None else torch.float8_e4m3fn)
        if s["quant"] == "head":
            s["out_scales"] = torch.rand(case["pool"], h, generator=g, device=DEV)
    return s


def _prepare_absorb(case, g):
    t, h, gap = case["tokens"], case["heads"], case["gap"]
    far = 32768
    s = {"q": torch.randn(t, h * (D_NOPE + D_ROPE) + gap, generator=g, device=DEV).to(torch.bfloat16)
                   [:, gap:].unflatten(1, (h, D_NOPE + D_ROPE)),
         "w_uk": torch.randn(h, D_NOPE, D_LATENT, generator=g, device=DEV).mul_(1 / math.sqrt(D_LATENT)).to(torch.bfloat16),
         "positions": None, "cos_sin": None, "interleaved": case["rope"] == "pairs",
         "q_scale": 0.02 if case["out"] == "e4m3" else None}
    if case["rope"] != "none":
        s["positions"], s["cos_sin"] = _positions(t, far, g), _table(far, D_ROPE)
    return s


def _prepare_scores(case, g, lengths):
    total, S, h = int(lengths.sum()), case["requests"] * case["qlen"], case["heads"]
    pool = total + 17
    k = torch.empty(pool, D_INDEX, dtype=torch.float8_e4m3fn, device=DEV)
    for at in range(0, pool, 1 << 20):
        n = min(1 << 20, pool - at)
        k[at:at + n] = torch.randn(n, D_INDEX, generator=g, device=DEV).mul_(8).to(torch.float8_e4m3fn)
    return {"q": torch.randn(S, h, D_INDEX, generator=g, device=DEV).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn),
            "weights": torch.randn(S, h, generator=g, device=DEV), "k": k,
            "pages": torch.randperm(pool, generator=g, device=DEV)[:total].to(torch.int32), "indptr": _indptr(lengths),
            "q_scales": torch.rand(S, h, generator=g, device=DEV).add_(0.5).mul_(0.01) if case["q_scales"] else None,
            "scale": 0.05, "qlen": case["qlen"], "causal": case["causal"], "max_len": int(lengths.max())}


def _prepare_select(case, g, lengths):
    total, qlen = int(lengths.sum()), case["qlen"]
    # as index_scores leaves them: many tokens that no head likes (zeros, so ties), -inf where a row does not see
    scores = torch.randn(qlen, total, generator=g, device=DEV).sub_(0.3).clamp_(min=0)
    if case["causal"]:
        seen = _visible(lengths, qlen, True).T.repeat_interleave(lengths, 1)
        pos = torch.cat([torch.arange(n) for n in lengths.tolist()])
        scores.masked_fill_((pos >= seen).to(DEV), float("-inf"))
    return {"scores": scores, "pages": torch.randperm(total + 5, generator=g, device=DEV)[:total].to(torch.int32),
            "indptr": _indptr(lengths), "topk": case["topk"], "block": case["block"], "recent": case["recent"],
            "sinks": case["sinks"], "causal": case["causal"], "max_len": int(lengths.max())}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op in ("index_scores", "index_select"):
        lengths = _lengths(case)[torch.randperm(case["requests"], generator=torch.Generator().manual_seed(seed))]
        state = (_prepare_scores if op == "index_scores" else _prepare_select)(case, g, lengths)
    else:
        state = (_prepare_norm_rope if op == "norm_rope" else _prepare_absorb)(case, g)
    state["op"] = op
    return state


# --------------------------------------------------------------- plain forms


def _rotate(y, positions, cos_sin, interleaved):
    """y [T, H, d] by the angles of its tokens' positions: column pairs (i, i + d/2), or (2i, 2i + 1)."""
    half = y.shape[2] // 2
    cs = cos_sin[positions][:, None, :]
    c, s = cs[..., :half], cs[..., half:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], 3).flatten(2)
    a, b = y[..., :half], y[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], 2)


def _plain_norm_rope(s):
    y = s["x"].float()
    if s["weight"] is not None:
        n = s["weight"].numel()
        head = y[..., :n]
        head = head * torch.rsqrt(head.square().mean(2, keepdim=True) + s["eps"]) * s["weight"].float()
        y = torch.cat([head, y[..., n:]], 2)
    if s["positions"] is not None:
        a, b = s["start"], s["start"] + s["cos_sin"].shape[1]
        y = torch.cat([y[..., :a], _rotate(y[..., a:b], s["positions"], s["cos_sin"], s["interleaved"]), y[..., b:]], 2)
    scales = None
    if s["quant"] is None:
        out = y.to(s["x"].dtype)
    else:
        sc = s["scale"]
        if s["quant"] == "head":
            amax = y.abs().amax(2)
            scales = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
            sc = scales[..., None]
        out = (y / sc).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    if s["slots"] is None:
        return {"out": out, "scales": scales}
    real = s["slots"] >= 0
    rows = s["slots"][real]
    held = s["out"].view(torch.uint8) if s["quant"] else s["out"]
    held[rows] = (out.view(torch.uint8) if s["quant"] else out)[real]
    if scales is not None:
        s["out_scales"][rows] = scales[real]
    return {"out": s["out"], "scales": s["out_scales"]}


def _plain_absorb(s):
    q = s["q"].float()
    latent = torch.bmm(q[..., :D_NOPE].transpose(0, 1), s["w_uk"].float()).transpose(0, 1)
    rope = q[..., D_NOPE:]
    if s["positions"] is not None:
        rope = _rotate(rope, s["positions"], s["cos_sin"], s["interleaved"])
    out = torch.cat([latent, rope], 2)
    if s["q_scale"] is None:
        return {"out": out.to(torch.bfloat16)}
    return {"out": (out / s["q_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)}


def _padded(s):
    """Positions of every request's tokens in the page list, padded to the longest request, and which are tokens."""
    start, end = s["indptr"][:-1].long()[:, None], s["indptr"][1:].long()[:, None]
    at = start + torch.arange(s["max_len"], device=DEV)
    return at, at < end


def _plain_scores(s):
    at, real = _padded(s)
    R, T = real.shape
    S, H, _ = s["q"].shape
    rows = s["pages"].long()[at.clamp(max=s["pages"].numel() - 1)]
    k = s["k"].view(torch.uint8)[rows.reshape(-1)].view(torch.float8_e4m3fn).float().view(R, T, D_INDEX)
    q = s["q"].float().view(R, s["qlen"] * H, D_INDEX)
    w = s["weights"] if s["q_scales"] is None else s["weights"] * s["q_scales"]
    dots = torch.bmm(q, k.transpose(1, 2)).clamp_(min=0).view(R, s["qlen"], H, T)
    scores = torch.einsum("rqht,rqh->rqt", dots, w.view(R, s["qlen"], H)) * s["scale"]
    if s["causal"]:
        seen = _visible(real.sum(1), s["qlen"], True)
        scores = scores.masked_fill(torch.arange(T, device=DEV) >= seen[..., None], float("-inf"))
    out = torch.empty(s["qlen"], s["pages"].numel(), device=DEV)
    out[:, at[real]] = scores.transpose(0, 1)[:, real]
    return {"scores": out}


def _plain_select(s):
    at, real = _padded(s)
    R, T = real.shape
    qlen, total = s["scores"].shape
    B, block, n = R * qlen, s["block"], s["topk"]
    seen = _visible(real.sum(1), qlen, s["causal"]).reshape(B, 1)
    blocks = -(-T // block)
    pos, tok = torch.arange(blocks, device=DEV), torch.arange(blocks * block, device=DEV)
    best = s["scores"][:, at.clamp(max=total - 1)].transpose(0, 1).reshape(B, T)
    best = torch.where(best.isnan() | (tok[:T] >= seen), torch.full_like(best, float("-inf")), best)
    best = torch.nn.functional.pad(best, (0, blocks * block - T), value=float("-inf")).view(B, blocks, block).amax(2)
    count = (seen + block - 1) // block
    kept = count.clamp(max=n)
    recent = kept.clamp(max=s["recent"])
    sinks = (kept - recent).clamp(max=s["sinks"])
    inside = pos < count
    always = ((pos < sinks) | (pos >= count - recent)) & inside
    # the blocks that may go first, heaviest first, ties to the lowest; the others sort behind them
    order = torch.sort((always | ~inside).to(torch.int8), dim=1, stable=True).indices
    heavy = torch.sort(torch.where(always | ~inside, torch.full_like(best, float("-inf")), best).gather(1, order), dim=1,
                       descending=True, stable=True).indices
    first = order.gather(1, heavy)
    rank = torch.empty_like(first).scatter_(1, first, pos.expand_as(first).contiguous())
    keep = always | (inside & ~always & (rank < kept - recent - sinks))
    keep = keep.repeat_interleave(block, 1)[:, :T] & (tok[:T] < seen)
    pages = s["pages"][at.clamp(max=total - 1)].repeat_interleave(qlen, 0)[keep]
    indptr = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    indptr[1:] = torch.cumsum(keep.sum(1), 0).to(torch.int32)
    out = torch.full((min(B * n * block, qlen * total),), -1, dtype=torch.int32, device=DEV)
    out[:pages.numel()] = pages
    return {"pages": out, "indptr": indptr}


# ----------------------------------------------------------------- own calls


def _own_norm_rope(s):
    import mla_decode_paged_gb300 as mla

    out, scales = mla.norm_rope(s["x"], s["weight"], s["eps"], positions=s["positions"], cos_sin=s["cos_sin"],
                                rope_start=s["start"], interleaved=s["interleaved"], quant=s["quant"], scale=s["scale"],
                                slots=s["slots"], out=s["out"], out_scales=s["out_scales"])
    return {"out": out, "scales": scales}


def _own_absorb(s):
    import mla_decode_paged_gb300 as mla

    return {"out": mla.query_absorb(s["q"], s["w_uk"], positions=s["positions"], cos_sin=s["cos_sin"],
                                    interleaved=s["interleaved"], q_scale=s["q_scale"])}


def _own_scores(s):
    import mla_decode_paged_gb300 as mla

    return {"scores": mla.index_scores(s["q"], s["weights"], s["k"], s["pages"], s["indptr"], q_scales=s["q_scales"],
                                       scale=s["scale"], qlen=s["qlen"], causal=s["causal"])}


def _own_select(s):
    import mla_decode_paged_gb300 as mla

    pages, indptr = mla.index_select(s["scores"], s["pages"], s["indptr"], s["topk"], block=s["block"],
                                     recent=s["recent"], sinks=s["sinks"], causal=s["causal"])
    return {"pages": pages, "indptr": indptr}


def run(state):
    if own:
        return {"norm_rope": _own_norm_rope, "query_absorb": _own_absorb, "index_scores": _own_scores,
                "index_select": _own_select}[state["op"]](state)
    return {"norm_rope": _plain_norm_rope, "query_absorb": _plain_absorb, "index_scores": _plain_scores,
            "index_select": _plain_select}[state["op"]](state)


# ------------------------------------------------------------ 64-bit results


def _exact_turn(y, s):
    """The rotation as a product of complex numbers."""
    half = y.shape[2] // 2
    cs = s["cos_sin"].double()[s["positions"]]
    turn = torch.complex(cs[:, :half], cs[:, half:])[:, None, :]
    if s["interleaved"]:
        return torch.view_as_real(torch.view_as_complex(y.reshape(*y.shape[:2], half, 2)) * turn).reshape(y.shape)
    z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn
    return torch.cat([z.real, z.imag], 2)


def _exact_norm_rope(s):
    y = s["x"].double().clone()
    if s["weight"] is not None:
        n = s["weight"].numel()
        power = torch.einsum("thd,thd->th", y[..., :n], y[..., :n]) / n
        y[..., :n] *= (s["weight"].double() / (power + s["eps"]).sqrt()[..., None])
    if s["positions"] is not None:
        a, b = s["start"], s["start"] + s["cos_sin"].shape[1]
        y[..., a:b] = _exact_turn(y[..., a:b].contiguous(), s)
    scales = None
    if s["quant"] == "static":
        y = (y / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX)
    elif s["quant"] == "head":
        scales = torch.maximum(y.max(2).values, -y.min(2).values) / E4M3_MAX
        scales[scales == 0] = 1
        y = y / scales[..., None]
    if s["slots"] is None:
        return {"out": y, "scales": scales}
    out = s["out"].double()
    held = None if scales is None else s["out_scales"].double()
    real = (s["slots"] >= 0).nonzero().view(-1)
    out.index_copy_(0, s["slots"][real], y[real])
    if scales is not None:
        held.index_copy_(0, s["slots"][real], scales[real])
    return {"out": out, "scales": held}


def _exact_absorb(s):
    T, H, _ = s["q"].shape
    out = torch.empty(T, H, D_QK, dtype=torch.float64, device=DEV)
    for h in range(H):
        out[:, h, :D_LATENT] = s["q"][:, h, :D_NOPE].double() @ s["w_uk"][h].double()
    rope = s["q"][..., D_NOPE:].double().contiguous()
    out[..., D_LATENT:] = rope if s["positions"] is None else _exact_turn(rope, s)
    return {"out": out if s["q_scale"] is None else (out / s["q_scale"]).clamp(-E4M3_MAX, E4M3_MAX)}


def _exact_scores(s):
    starts = s["indptr"].tolist()
    qlen = s["qlen"]
    out = torch.empty(qlen, s["pages"].numel(), dtype=torch.float64, device=DEV)
    for r, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        for at in range(a, b, 1 << 15):
            to = min(b, at + (1 << 15))
            k = s["k"].view(torch.uint8)[s["pages"][at:to].long()].view(torch.float8_e4m3fn).double()
            for i in range(qlen):
                t = r * qlen + i
                w = s["weights"][t].double() * s["scale"]
                if s["q_scales"] is not None:
                    w = w * s["q_scales"][t].double()
                out[i, at:to] = torch.relu(k @ s["q"][t].double().T) @ w
                if s["causal"]:
                    out[i, max(at, b - qlen + i + 1):to] = -math.inf
    return {"scores": out}


def _exact_select(s):
    starts, pages, scores = s["indptr"].tolist(), s["pages"].cpu(), s["scores"].double().cpu()
    qlen, block = scores.shape[0], s["block"]
    lists, indptr = [], [0]
    for a, b in zip(starts[:-1], starts[1:]):
        for i in range(qlen):
            n = max(0, b - a - qlen + i + 1) if s["causal"] else b - a
            x = torch.nan_to_num(scores[i, a:a + n], nan=-math.inf, posinf=math.inf, neginf=-math.inf)
            count = -(-n // block)
            keep = min(count, s["topk"])
            recent = min(s["recent"], keep)
            sinks = min(s["sinks"], keep - recent)
            x = torch.cat([x, torch.full((count * block - n,), -math.inf, dtype=torch.float64)])
            middle = torch.arange(sinks, count - recent)
            top = x.view(count, block).max(1).values[middle] if count else x
            mark = torch.zeros(count, dtype=torch.bool)
            mark[:sinks] = True
            mark[count - recent:] = True
            mark[middle[torch.argsort(-top, stable=True)[:keep - recent - sinks]]] = True
            chosen = (mark.nonzero() * block + torch.arange(block)).view(-1)
            chosen = chosen[chosen < n]
            lists.append(pages[a + chosen])
            indptr.append(indptr[-1] + chosen.numel())
    out = torch.full((min((len(indptr) - 1) * s["topk"] * block, qlen * pages.numel()),), -1, dtype=torch.int32)
    out[:indptr[-1]] = torch.cat(lists)
    return {"pages": out, "indptr": torch.tensor(indptr, dtype=torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "query_absorb": _exact_absorb, "index_scores": _exact_scores,
            "index_select": _exact_select}[s["op"]](s)
