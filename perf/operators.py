"""The operators around one MLA decode step, with the cases they are measured on.

Four entry points of the package beside attend / merge / value_gate / kv_append:

  add_rms_norm     residual addition, root-mean-square norm, output in 16 or 8 bits
  token_weights    attention weight that each cached token received, accumulated
  kv_evict         the tokens of every request that stay in the cache, by that weight
  value_gate_lora  the W_UV projection and gate with one low-rank adapter per request

``run`` computes an operator in its plain form (elementary torch operations in 32
bits) or, with ``own`` true, by the package's call.
"""

import math

import torch

own = False

D_QK, D_LATENT, D_V, E4M3_MAX = 576, 512, 128, 448.0
DEV = "cuda"


# --------------------------------------------------------------------- cases


def _norm(tokens, width, residual="none", quant="none", stride=0, type="bf16"):
    return {"op": "add_rms_norm", "tokens": tokens, "width": width, "stride": stride or width, "residual": residual,
            "quant": quant, "type": type, "eps": 1e-5}


def _weights(requests, qlen, heads, lo, hi, pad=0, causal=False, query="bf16", deal=1):
    return {"op": "token_weights", "requests": requests, "qlen": qlen, "heads": heads, "pad": pad or heads, "lo": lo,
            "hi": hi, "causal": causal, "query": query, "deal": deal}


def _evict(requests, lo, hi, budget, recent, sinks, deal=1):
    return {"op": "kv_evict", "requests": requests, "lo": lo, "hi": hi, "budget": budget, "recent": recent,
            "sinks": sinks, "deal": deal}


def _lora(requests, qlen, heads, rank, adapters):
    return {"op": "value_gate_lora", "requests": requests, "qlen": qlen, "heads": heads, "rank": rank,
            "adapters": adapters}


def listed():
    return [
        # The layer's input norm in a decode step of 64 requests (hidden size 7168): latency counts.
        dict(_norm(64, 7168, residual="same"), name="norm_decode"),
        # The norm of the 512 latent columns of a 576-wide projection, one speculative step of 256 x 8 rows.
        dict(_norm(2048, 512, stride=576), name="norm_latent"),
        # The input norm of a prefill chunk that feeds 8-bit projections with scales per 128 columns.
        dict(_norm(16384, 7168, residual="same", quant="group"), name="norm_prefill_fp8"),
        # One decode step's weights, 64 requests of 1K to 8K tokens, 12 heads.
        dict(_weights(64, 1, 12, 1024, 8192), name="weights_decode"),
        # Speculative decoding: 4 rows a request under the causal mask, 4K to 32K tokens (the largest case).
        dict(_weights(128, 4, 12, 4096, 32768, causal=True), name="weights_spec"),
        # Long contexts, all 96 heads on one GPU, the query padded to 128 heads.
        dict(_weights(32, 1, 96, 32768, 32768, pad=128), name="weights_long"),
        # One interactive request whose 128K context is cut to 8K: latency counts.
        dict(_evict(1, 131072, 131072, 8192, 512, 4), name="evict_one_long"),
        # 64 requests of 1K to 8K tokens held to 2K.
        dict(_evict(64, 1024, 8192, 2048, 128, 4), name="evict_decode"),
        # A ragged batch, 128 to 128K tokens, held to 16K.
        dict(_evict(256, 128, 131072, 16384, 1024, 16), name="evict_ragged"),
        # A decode step of 64 tenants with small adapters of their own.
        dict(_lora(64, 1, 12, 16, 64), name="lora_decode"),
        # 96 heads, few long requests, a handful of adapters.
        dict(_lora(32, 1, 96, 32, 8), name="lora_heads96"),
        # Speculative rows: 256 requests x 8 rows, 32 adapters of rank 64.
        dict(_lora(256, 8, 12, 64, 32), name="lora_ragged"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "weights", "evict", "lora"])
    if op == "norm":
        width = 8 * _log_int(rng, 16, 1024)
        quant = rng.choice(["none", "row", "group", "static"])
        tokens = _log_int(rng, 1, min(32768, 16384 * 7168 // width // 2))
        return _norm(tokens, width, rng.choice(["none", "same", "f32"]), quant,
                     width + 8 * rng.choice([0, 0, 1, 8]), rng.choice(["bf16", "bf16", "fp16"]))
    if op == "weights":
        qlen, heads = rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([8, 12, 16, 24, 32, 64, 96, 128])
        rows = qlen * heads
        # at most the tokens and the token-row products of the largest listed case, half of it on average
        most = min(1100000, 110000000 // rows)
        requests = _log_int(rng, 1, 128)
        hi = _log_int(rng, 33, max(34, min(65536, most // requests)))
        return _weights(requests, qlen, heads, _log_int(rng, max(1, hi // 8), hi), hi, heads + rng.choice([0, 0, 4]),
                        rng.choice([False, True]), rng.choice(["bf16", "bf16", "e4m3"]), rng.randrange(1 << 16))
    if op == "evict":
        requests = _log_int(rng, 1, 256)
        hi = _log_int(rng, 100, min(131072, 16000000 // requests))
        lo = _log_int(rng, max(1, hi // 100), hi)
        budget = _log_int(rng, max(1, hi // 32), hi)
        return _evict(requests, lo, hi, budget, rng.randrange(0, budget // 2 + 1), rng.randrange(0, 33),
                      rng.randrange(1 << 16))
    heads = rng.choice([8, 12, 16, 32, 96])
    rank = 8 * rng.choice([1, 2, 3, 4, 5, 8, 16])
    qlen = rng.choice([1, 1, 2, 4, 5, 8])
    requests = _log_int(rng, 1, max(1, 24576 // (heads * qlen)))
    return _lora(requests, qlen, heads, rank, _log_int(rng, 1, 32))


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


def work(case):
    op = case["op"]
    if op == "add_rms_norm":
        n = case["tokens"] * case["width"]
        res = {"none": 0, "same": 4, "f32": 8}[case["residual"]]
        scales = {"none": 0, "static": 0, "row": case["tokens"], "group": case["tokens"] * -(-case["width"] // 128)}
        out = 2 if case["quant"] == "none" else 1
        return {"bytes": n * (2 + res + out) + 2 * case["width"] + 4 * scales[case["quant"]], "flops": 6 * n}
    if op == "token_weights":
        rows = case["requests"] * case["qlen"] * case["heads"]
        total = int(_lengths(case).sum())
        return {"bytes": total * (D_QK + 12) + rows * (D_QK * (1 if case["query"] == "e4m3" else 2) + 4),
                "flops": 2 * D_QK * total * case["qlen"] * case["heads"]}
    if op == "kv_evict":
        total = int(_lengths(case).sum())
        return {"bytes": 16 * total + 8 * case["requests"], "flops": 4 * total}
    rows = case["requests"] * case["qlen"] * case["heads"]
    used = min(case["adapters"], case["requests"])
    bytes_ = (rows * (D_LATENT + 2 * D_V) * 2 + case["heads"] * D_V * D_LATENT * 2
              + used * case["rank"] * (D_LATENT + case["heads"] * D_V) * 2 + 8 * case["requests"])
    return {"bytes": bytes_, "flops": 2 * rows * (D_V * D_LATENT + case["rank"] * (D_LATENT + D_V))}


# -------------------------------------------------------------------- inputs


def _indptr(lengths):
    indptr = torch.zeros(lengths.numel() + 1, dtype=torch.int64)
    indptr[1:] = torch.cumsum(lengths, 0)
    return indptr.to(torch.int32).to(DEV)


def _prepare_norm(case, g):
    t = {"bf16": torch.bfloat16, "fp16": torch.float16}[case["type"]]
    n, d = case["tokens"], case["width"]
    x = torch.randn(n, case["stride"], generator=g, device=DEV).to(t)[:, :d]
    residual = None
    if case["residual"] != "none":
        residual = torch.randn(n, d, generator=g, device=DEV).mul_(2).to(t if case["residual"] == "same" else torch.float32)
    weight = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(t)
    return {"x": x, "residual": residual, "weight": weight, "eps": case["eps"],
            "quant": None if case["quant"] == "none" else case["quant"],
            "scale": 0.02 if case["quant"] == "static" else None}


def _prepare_weights(case, g, lengths):
    total, R = int(lengths.sum()), case["requests"]
    S, H, P = R * case["qlen"], case["heads"], case["pad"]
    pool = total + 17
    pages = torch.randperm(pool, generator=g, device=DEV)[:total].to(torch.int32)
    kv = torch.empty(pool, D_QK, dtype=torch.uint8, device=DEV)
    for at in range(0, pool, 1 << 18):
        x = torch.randn(min(1 << 18, pool - at), D_QK, generator=g, device=DEV).mul_(0.5)
        kv[at:at + x.shape[0]] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn(S, P, D_QK, generator=g, device=DEV)
    q = q.to(torch.bfloat16) if case["query"] == "bf16" else q.to(torch.float8_e4m3fn)
    state = {"q": q, "kv": kv, "pages": pages, "indptr": _indptr(lengths), "scale": 1 / math.sqrt(192.0),
             "kv_scale": 0.8, "q_scale": 1.0 if case["query"] == "bf16" else 0.9, "heads": H, "qlen": case["qlen"],
             "max_len": int(lengths.max()), "causal": case["causal"], "decay": 0.97,
             # a few steps' weights already gathered
             "weights": torch.rand(total, generator=g, device=DEV).mul_(4 * S * H / total)}
    # the log-sum-exp of every row's scores, as the step's merge leaves it
    scores, _, _ = _scores(state)
    state["lse"] = torch.logsumexp(scores, 2).reshape(S, H).contiguous()
    return state


def _prepare_lora(case, g):
    R, H, r, n = case["requests"], case["heads"], case["rank"], case["adapters"]
    S = R * case["qlen"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(torch.bfloat16)

    lengths = torch.randint(1, 4096, (R,), generator=g, device=DEV, dtype=torch.int32)
    adapters = torch.randint(0, n, (R,), generator=g, device=DEV, dtype=torch.int32)
    if n >= R:  # each request its own
        adapters = torch.randperm(n, generator=g, device=DEV)[:R].to(torch.int32)
    if R > 4:  # one request without an adapter, one without tokens
        adapters[1], lengths[3] = -1, 0
    return {"latent": normal(S, H, D_LATENT, std=0.05), "w_uv": normal(H, D_V, D_LATENT, std=1 / math.sqrt(D_LATENT)),
            "gate": normal(S, H * D_V), "lengths": lengths, "lora_a": normal(n, r, D_LATENT, std=1 / math.sqrt(D_LATENT)),
            "lora_b": normal(n, H * D_V, r, std=0.2), "adapters": adapters,
            "lora_scale": torch.rand(n, generator=g, device=DEV) + 0.5, "qlen": case["qlen"]}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op in ("token_weights", "kv_evict"):
        lengths = _lengths(case)[torch.randperm(case["requests"], generator=torch.Generator().manual_seed(seed))]
    if op == "add_rms_norm":
        state = _prepare_norm(case, g)
    elif op == "token_weights":
        state = _prepare_weights(case, g, lengths)
    elif op == "kv_evict":
        total = int(lengths.sum())
        # weights that fall off steeply from a few heavy tokens
        state = {"pages": torch.randperm(total + 5, generator=g, device=DEV)[:total].to(torch.int32),
                 "indptr": _indptr(lengths), "weights": torch.randn(total, generator=g, device=DEV).mul_(2).exp_(),
                 "budget": case["budget"], "recent": case["recent"], "sinks": case["sinks"],
                 "max_len": int(lengths.max())}
    else:
        state = _prepare_lora(case, g)
    state["op"] = op
    return state


# --------------------------------------------------------------- plain forms


def _plain_norm(s):
    x = s["x"].float()
    residual_out = None
    if s["residual"] is not None:
        x = x + s["residual"].float()
        residual_out = x.to(s["residual"].dtype)
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    if s["quant"] is None:
        return {"out": y.to(s["x"].dtype), "residual_out": residual_out}
    n, d = y.shape
    if s["quant"] == "static":
        return {"out": (y / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn),
                "residual_out": residual_out}
    width = d if s["quant"] == "row" else 128
    groups = -(-d // width)
    y = torch.nn.functional.pad(y, (0, groups * width - d)).view(n, groups, width)
    amax = y.abs().amax(2, keepdim=True)
    scales = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
    codes = (y / scales).clamp(-E4M3_MAX, E4M3_MAX).reshape(n, groups * width)[:, :d].to(torch.float8_e4m3fn)
    return {"out": codes, "scales": scales.view(n, groups), "residual_out": residual_out}


def _padded(s):
    """Positions of every request's tokens in the page list, padded to the longest request, and which are tokens."""
    start, end = s["indptr"][:-1].long()[:, None], s["indptr"][1:].long()[:, None]
    at = start + torch.arange(s["max_len"], device=DEV)
    return at, at < end


def _scores(s, dtype=torch.float32):
    """Scores [requests, qlen * heads, tokens] (-inf where a row does not see the token), positions, what is a token."""
    at, real = _padded(s)
    R, T = real.shape
    rows = s["pages"].long()[at.clamp(max=s["pages"].numel() - 1)]
    k = s["kv"][rows.reshape(-1)].view(torch.float8_e4m3fn).to(dtype).view(R, T, D_QK)
    q = s["q"][:, :s["heads"]].to(dtype).reshape(R, s["qlen"] * s["heads"], D_QK)
    scores = torch.bmm(q, k.transpose(1, 2)) * (s["scale"] * s["q_scale"] * s["kv_scale"])
    seen = real[:, None, :]
    if s["causal"]:
        length = real.sum(1)[:, None, None]
        row = torch.arange(s["qlen"], device=DEV).repeat_interleave(s["heads"])[None, :, None]
        seen = seen & (torch.arange(T, device=DEV) < length - s["qlen"] + row + 1)
    return scores.masked_fill(~seen, float("-inf")), at, real


def _plain_weights(s):
    scores, at, real = _scores(s)
    lse = s["lse"].view(scores.shape[0], scores.shape[1], 1)
    p = torch.where(lse == float("-inf"), torch.zeros_like(scores), torch.exp(scores - lse))
    out = s["weights"] * s["decay"]
    out[at[real]] += p.sum(1)[real]
    return {"weights": out}


def _plain_evict(s):
    at, real = _padded(s)
    w = s["weights"][at.clamp(max=s["weights"].numel() - 1)]
    pos = torch.arange(at.shape[1], device=DEV)
    length = real.sum(1, keepdim=True)
    kept = length.clamp(max=max(s["budget"], 0))
    recent = kept.clamp(max=s["recent"])
    sinks = (kept - recent).clamp(max=s["sinks"])
    always = ((pos < sinks) | (pos >= length - recent)) & real
    w = torch.where(w.isnan() | always | ~real, torch.full_like(w, float("-inf")), w)
    # the tokens that may go, heaviest first, ties to the lowest position; the others sort behind them
    order = torch.sort((always | ~real).to(torch.int8), dim=1, stable=True).indices
    heavy = torch.sort(w.gather(1, order), dim=1, descending=True, stable=True).indices
    free = (real & ~always).sum(1, keepdim=True)
    first = order.gather(1, heavy)
    rank = torch.empty_like(first).scatter_(1, first, pos.expand_as(first).contiguous())
    # among equal values (-inf), the tokens that may go come before those that sorted behind them
    keep = always | (real & ~always & (rank < torch.minimum(kept - recent - sinks, free)))
    keep_flat, pages = keep[real], s["pages"]
    indptr_out = torch.zeros_like(s["indptr"])
    indptr_out[1:] = torch.cumsum(kept.view(-1), 0).to(torch.int32)
    weights = s["weights"][keep_flat]
    return {"pages": torch.cat([pages[keep_flat], pages[~keep_flat]]), "indptr": indptr_out,
            "weights": torch.cat([weights, weights.new_zeros(pages.numel() - weights.numel())])}


def _plain_lora(s):
    S, H, _ = s["latent"].shape
    a = s["adapters"].long()
    R, qlen = a.numel(), s["qlen"]
    latent = s["latent"].float()
    value = torch.einsum("shc,hvc->shv", latent, s["w_uv"].float())
    used = a.clamp(min=0)
    t = torch.bmm(latent.view(R, qlen * H, D_LATENT), s["lora_a"][used].float().transpose(1, 2))
    b = s["lora_b"][used].float().view(R, H, D_V, -1)
    delta = torch.einsum("rqhk,rhvk->rqhv", t.view(R, qlen, H, -1), b)
    factor = torch.where(a >= 0, s["lora_scale"][used], torch.zeros_like(s["lora_scale"][used]))
    value = value + (delta * factor.view(R, 1, 1, 1)).reshape(S, H, D_V)
    out = value.reshape(S, H * D_V) * torch.sigmoid(s["gate"].float())
    live = (s["lengths"] > 0).repeat_interleave(qlen)[:, None]
    return {"out": torch.where(live, out, torch.zeros_like(out)).to(torch.bfloat16)}


# --------------------------------------------------------------- own calls


def _own_norm(s):
    import mla_decode_paged_gb300 as mla

    out, scales, residual_out = mla.add_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"],
                                                 quant=s["quant"], scale=s["scale"])
    if scales is None:
        return {"out": out, "residual_out": residual_out}
    return {"out": out, "scales": scales.view(out.shape[0], -1), "residual_out": residual_out}


def _own_weights(s):
    import mla_decode_paged_gb300 as mla

    return {"weights": mla.token_weights(s["q"], s["kv"], s["pages"], s["indptr"], s["scale"], s["kv_scale"], s["lse"],
                                         heads=s["heads"], qlen=s["qlen"], weights=s["weights"], decay=s["decay"],
                                         causal=s["causal"], q_scale=s["q_scale"])}


def _own_evict(s):
    import mla_decode_paged_gb300 as mla

    pages, indptr, weights = mla.kv_evict(s["pages"], s["indptr"], s["weights"], s["budget"], recent=s["recent"],
                                          sinks=s["sinks"])
    return {"pages": pages, "indptr": indptr, "weights": weights}


def _own_lora(s):
    import mla_decode_paged_gb300 as mla

    return {"out": mla.value_gate_lora(s["latent"], s["w_uv"], s["gate"], s["lengths"], s["lora_a"], s["lora_b"],
                                       s["adapters"], s["lora_scale"], s["qlen"])}


def run(state):
    if own:
        return {"add_rms_norm": _own_norm, "token_weights": _own_weights, "kv_evict": _own_evict,
                "value_gate_lora": _own_lora}[state["op"]](state)
    return {"add_rms_norm": _plain_norm, "token_weights": _plain_weights, "kv_evict": _plain_evict,
            "value_gate_lora": _plain_lora}[state["op"]](state)


# ------------------------------------------------------------ 64-bit results


def _exact_norm(s):
    x = s["x"].double()
    total = x if s["residual"] is None else x + s["residual"].double()
    residual_out = None if s["residual"] is None else total
    y = total / ((total * total).sum(1, keepdim=True) / total.shape[1] + s["eps"]).sqrt() * s["weight"].double()
    if s["quant"] is None:
        return {"out": y, "residual_out": residual_out}
    if s["quant"] == "static":
        return {"out": (y / s["scale"]).clamp(-E4M3_MAX, E4M3_MAX), "residual_out": residual_out}
    parts = y.split(y.shape[1] if s["quant"] == "row" else 128, 1)
    scales = torch.stack([p.abs().max(1).values / E4M3_MAX for p in parts], 1)
    scales = torch.where(scales == 0, torch.ones_like(scales), scales)
    codes = torch.cat([p / scales[:, i:i + 1] for i, p in enumerate(parts)], 1)
    return {"out": codes, "scales": scales, "residual_out": residual_out}


def _exact_weights(s):
    starts = s["indptr"].tolist()
    out = s["weights"].double() * s["decay"]
    qlen, H = s["qlen"], s["heads"]
    factor = s["scale"] * s["q_scale"] * s["kv_scale"]
    for r, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        rows = slice(r * qlen, (r + 1) * qlen)
        for at in range(a, b, 1 << 16):
            to = min(b, at + (1 << 16))
            k = s["kv"][s["pages"][at:to].long()].view(torch.float8_e4m3fn).double()
            for i in range(qlen):
                q = s["q"][rows][i, :H].double()
                lse = s["lse"][rows][i].double()
                p = torch.exp(q @ k.T * factor - lse[:, None]).sum(0)
                if s["causal"]:
                    p[max(0, b - a - qlen + i + 1 - (at - a)):] = 0
                out[at:to] += p
    return {"weights": out}


def _exact_evict(s):
    starts, pages, weights = s["indptr"].tolist(), s["pages"].cpu(), s["weights"].double().cpu()
    kept_all, freed_all, indptr = [], [], [0]
    for a, b in zip(starts[:-1], starts[1:]):
        n = b - a
        keep = min(n, max(s["budget"], 0))
        recent = min(s["recent"], keep)
        sinks = min(s["sinks"], keep - recent)
        mark = torch.zeros(n, dtype=torch.bool)
        mark[:sinks] = True
        mark[n - recent:] = True
        middle = torch.arange(sinks, n - recent)
        w = torch.nan_to_num(weights[a:b][middle], nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        best = torch.argsort(-w, stable=True)[:keep - recent - sinks]
        mark[middle[best]] = True
        kept_all.append(a + mark.nonzero().view(-1))
        freed_all.append(a + (~mark).nonzero().view(-1))
        indptr.append(indptr[-1] + keep)
    kept, freed = torch.cat(kept_all), torch.cat(freed_all)
    return {"pages": pages[torch.cat([kept, freed])], "indptr": torch.tensor(indptr, dtype=torch.int32),
            "weights": torch.cat([weights[kept], torch.zeros(freed.numel(), dtype=torch.float64)])}


def _exact_lora(s):
    S, H, _ = s["latent"].shape
    out = torch.zeros(S, H * D_V, dtype=torch.float64, device=DEV)
    gate = 1 / (1 + torch.exp(-s["gate"].double()))
    w = s["w_uv"].double()
    for r, (a, live) in enumerate(zip(s["adapters"].tolist(), (s["lengths"] > 0).tolist())):
        rows = slice(r * s["qlen"], (r + 1) * s["qlen"])
        x = s["latent"][rows].double().transpose(0, 1)
        value = x @ w.transpose(1, 2)
        if a >= 0:
            b = s["lora_b"][a].double().view(H, D_V, -1)
            value = value + float(s["lora_scale"][a]) * ((x @ s["lora_a"][a].double().T) @ b.transpose(1, 2))
        if live:
            out[rows] = value.transpose(0, 1).reshape(-1, H * D_V) * gate[rows]
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"add_rms_norm": _exact_norm, "token_weights": _exact_weights, "kv_evict": _exact_evict,
            "value_gate_lora": _exact_lora}[s["op"]](s)
