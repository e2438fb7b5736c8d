"""Cases of the rotary-position and scored-attention operators, with their plain forms.

Three families, each with its plain form in elementary torch operations and
the call that a user makes:

* ``rotary``: rotary positions of q and k (forward, and the gradients' way
  back), from the projections' [Z, N, heads, D] layout to the attention's
  [Z, heads, N, D] one and back; and the serving form that writes the rotated
  keys and the values into a paged cache.
* ``scored``: attention whose scores are capped, biased by distance and
  restricted to a range of keys per query (documents, prefix, window,
  causal); forward alone (prefill) or with its gradients (training).
* ``paged``: the same scores for a chunk of new tokens per sequence, or
  single tokens, over a paged cache.
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
NEG = float("-inf")


# ------------------------------------------------------------------- cases


def _rotary(name, kind, Z, H, Hkv, N, D, rot, interleaved, dtype, far=0, page=64, live=1.0):
    return {"name": name, "op": "rotary", "kind": kind, "Z": Z, "H": H, "Hkv": Hkv, "N": N, "D": D, "rot": rot,
            "interleaved": interleaved, "dtype": dtype, "far": far, "page": page, "live": live}


def _scored(name, train, Z, H, Hkv, Nq, Nk, D, mask, cap, bias, dtype):
    return {"name": name, "op": "scored", "train": train, "Z": Z, "H": H, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "D": D,
            "mask": mask, "cap": cap, "bias": bias, "dtype": dtype}


def _paged(name, B, H, Hkv, Nq, ctx, D, page, window, cap, bias, dtype, ragged=True):
    return {"name": name, "op": "paged", "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "ctx": ctx, "D": D, "page": page,
            "window": window, "cap": cap, "bias": bias, "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # one decode step of a small batch: positions and cache write of one new token per sequence
        _rotary("rotary_cache_token", "cache", 16, 32, 8, 1, 128, 128, False, "fp16", far=30000),
        # chunked prefill: up to 512 new tokens per sequence, part of the head rotated, padded rows skipped
        _rotary("rotary_cache_chunk", "cache", 8, 32, 8, 512, 128, 64, True, "bf16", far=100000, live=0.8),
        # a training micro-batch's projections, whole head rotated
        _rotary("rotary_train", "fwd", 4, 32, 8, 8192, 128, 128, False, "bf16"),
        # its gradients on the way back, odd length, a quarter of the head
        _rotary("rotary_grad_odd", "bwd", 3, 16, 16, 1021, 64, 16, False, "fp16", far=5000),
        # the smallest call: one tile per head, capped and biased
        _scored("scored_small", False, 1, 2, 2, 128, 128, 64, "causal", 30.0, True, "fp16"),
        # prefill of a capped model with wide heads behind a sliding window
        _scored("scored_window_d256", False, 4, 8, 4, 2048, 2048, 256, "window", 50.0, False, "bf16"),
        # training step of packed documents, grouped heads, distance bias
        _scored("train_docs", True, 2, 16, 4, 4096, 4096, 128, "docs", 0.0, True, "bf16"),
        # training step at the benchmark's head shape, capped scores, causal
        _scored("train_cap_causal", True, 32, 8, 8, 1024, 1024, 128, "causal", 50.0, False, "fp16"),
        # training step with a bidirectional prefix, odd length, small heads
        _scored("train_prefix_odd", True, 3, 8, 8, 1021, 1021, 64, "prefix", 20.0, True, "fp16"),
        # decode of a small batch over long contexts
        _paged("paged_token_long", 4, 32, 8, 1, 32768, 128, 64, 0, 50.0, False, "fp16", ragged=False),
        # decode of a large batch of uneven contexts with a distance bias
        _paged("paged_token_batch", 64, 32, 8, 1, 8192, 128, 16, 0, 0.0, True, "bf16"),
        # chunked prefill: up to 512 new tokens per sequence behind up to 8192 cached ones, sliding window
        _paged("paged_chunk", 8, 32, 8, 512, 8192, 128, 64, 4096, 30.0, False, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _score_cells(case):
    """Scores that the plain form holds at once."""
    if case["op"] == "rotary":
        return 0
    return case.get("Z", case.get("B")) * case["H"] * case["Nq"] * case.get("Nk", case.get("ctx"))


def draw(rng):
    op = rng.choice(["rotary", "scored", "scored", "paged", "paged"])
    dtype = rng.choice(["fp16", "bf16"])
    D = rng.choice([64, 64, 128, 128, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 8])
    if op == "rotary":
        kind = rng.choice(["fwd", "bwd", "cache"])
        N = _log(rng, 1, 8192 if kind != "cache" else 1024)
        c = _rotary("", kind, _log(rng, 1, 16), H, Hkv, N, D, rng.choice([D, D, D // 2, D // 4, 20]),
                    rng.random() < 0.5, dtype, far=_log(rng, 1, 1000000), page=rng.choice([16, 32, 64]),
                    live=rng.choice([1.0, 0.7]))
        shrink = ("Z", "N")
    elif op == "scored":
        mask = rng.choice(["none", "causal", "window", "docs", "prefix"])
        train = rng.random() < 0.6
        # a softmax over one key has no gradient, so training starts at lengths that have some
        Nk = _log(rng, 32 if train else 1, 4096)
        Nq = Nk if mask == "docs" or rng.random() < 0.7 else _log(rng, 1, Nk)
        c = _scored("", train, _log(rng, 1, 32), H, Hkv, Nq, Nk, D, mask, rng.choice([0.0, 20.0, 50.0]),
                    rng.random() < 0.5, dtype)
        shrink = ("Z", "Hkv")
    else:
        Nq = 1 if rng.random() < 0.6 else _log(rng, 2, 512)
        B = _log(rng, 1, 64) if Nq == 1 else _log(rng, 1, 8)
        ctx = _log(rng, max(1, Nq), 32768 if Nq == 1 else 8192)
        c = _paged("", B, H, Hkv, Nq, ctx, D, rng.choice([16, 32, 64]), rng.choice([0, 0, 1024, 257]),
                   rng.choice([0.0, 30.0, 50.0]), rng.random() < 0.5, dtype, ragged=rng.random() < 0.8)
        shrink = ("B", "Hkv")
    most = {"rotary": (6.7e8, 1e12), "scored": (6e8, 2.4e11), "paged": (1.35e9, 2.4e11)}[op]
    while work(c)["bytes"] > most[0] or work(c)["flops"] > most[1] or _score_cells(c) > 6e8:
        at = shrink[0] if c[shrink[0]] > 1 else shrink[1]
        if at == "Hkv" and c["Hkv"] == 1:  # one key head left: fewer query heads
            c["H"] = max(1, c["H"] // 2)
        elif at == "Hkv":
            group, c["Hkv"] = c["H"] // c["Hkv"], c["Hkv"] // 2
            c["H"] = group * c["Hkv"]
        else:
            c[at] = (c[at] + 1) // 2
    c.pop("name")
    return c


# ------------------------------------------------------------------ inputs


def _lengths(case, gen, device):
    """(context_lens, q_lens) of a paged case: the first sequence has the longest context and a full chunk."""
    B, Nq, ctx = case["B"], case["Nq"], case["ctx"]
    if not case["ragged"]:
        return torch.full((B,), ctx, dtype=torch.int32, device=device), torch.full((B,), Nq, dtype=torch.int32,
                                                                                   device=device)
    lens = torch.randint(max(1, ctx // 4), ctx + 1, (B,), generator=gen, device=device, dtype=torch.int64)
    qs = torch.randint(1, Nq + 1, (B,), generator=gen, device=device, dtype=torch.int64)
    lens[0], qs[0] = ctx, Nq
    return lens.to(torch.int32), torch.minimum(qs, lens).to(torch.int32)


def _slopes(H, device):
    """The usual geometric slopes of a distance bias: 2^(-8 (h + 1) / H)."""
    return torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H).to(torch.float32).to(device)


def _doc_ids(Z, N, gen, device):
    """Packed documents: a new one starts at each position with probability 6 / N."""
    new = torch.rand((Z, N), generator=gen, device=device) < 6.0 / N
    return torch.cumsum(new.to(torch.int32), 1).to(torch.int32)


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=device).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, mul=1.0):
        return (torch.randn(shape, generator=gen, device=device, dtype=torch.float32) * mul).to(dt)

    s = {"case": case}
    if case["op"] == "rotary":
        Z, H, Hkv, N, D, rot = (case[x] for x in ("Z", "H", "Hkv", "N", "D", "rot"))
        s["freqs"] = torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64) / rot).to(device)
        first = torch.randint(0, case["far"] + 1, (Z, 1), generator=gen, device=device)
        s["positions"] = first + torch.arange(N, device=device)[None, :]
        if case["kind"] == "bwd":  # gradients as the attention's backward leaves them
            s["dq"], s["dk"] = normal(Z, H, N, D), normal(Z, Hkv, N, D)
        else:  # one projection's output, q, k and v beside each other
            qkv = normal(Z, N, H + 2 * Hkv, D)
            s["q"] = qkv[:, :, :H].transpose(1, 2)
            s["k"] = qkv[:, :, H:H + Hkv].transpose(1, 2)
            s["v"] = qkv[:, :, H + Hkv:].transpose(1, 2)
        if case["kind"] == "cache":
            page = case["page"]
            pages = (Z * N + page - 1) // page + 3
            s["k_cache"] = torch.zeros((pages, page, Hkv, D), device=device, dtype=dt)
            s["v_cache"] = torch.zeros_like(s["k_cache"])
            slots = torch.randperm(pages * page, generator=gen, device=device)[:Z * N].reshape(Z, N)
            if N > 1:  # rows of the padded batch behind a sequence's new tokens
                live = torch.randint(1, N + 1, (Z, 1), generator=gen, device=device) if case["live"] < 1 else N
                slots = torch.where(torch.arange(N, device=device)[None, :] < live, slots, -1)
            s["slots"] = slots.contiguous()
        return s
    D, H, Hkv = case["D"], case["H"], case["Hkv"]
    s["scale"] = 1.0 / math.sqrt(D)
    s["slopes"] = _slopes(H, device) if case["bias"] else None
    # a cap is there because scores get large: wide queries reach into its bend
    wide = 4.0 if case["cap"] else 1.0
    if case["op"] == "scored":
        Z, Nq, Nk = case["Z"], case["Nq"], case["Nk"]
        s["q"], s["k"], s["v"] = normal(Z, H, Nq, D, mul=wide), normal(Z, Hkv, Nk, D), normal(Z, Hkv, Nk, D)
        s["do"] = normal(Z, H, Nq, D) if case["train"] else None
        if case["mask"] == "docs":
            s["docs"] = _doc_ids(Z, Nk, gen, device)
        if case["mask"] == "prefix":
            s["prefix"] = torch.randint(0, Nk + 1, (Z,), generator=gen, device=device).to(torch.int32)
        s["window"] = max(1, Nk // 4) if case["mask"] == "window" else 0
        return s
    B, Nq, page = case["B"], case["Nq"], case["page"]
    s["q"] = normal(B, H, Nq, D, mul=wide)
    s["context_lens"], s["q_lens"] = _lengths(case, gen, device)
    max_pages = (case["ctx"] + page - 1) // page
    pages = B * max_pages + 1
    s["k_cache"], s["v_cache"] = normal(pages, page, Hkv, D), normal(pages, page, Hkv, D)
    s["block_table"] = torch.randperm(pages, generator=gen, device=device)[:B * max_pages].reshape(
        B, max_pages).to(torch.int32).contiguous()
    if not case["ragged"]:
        s["q_lens"] = None
    return s


# ------------------------------------------------------------- plain forms


def _rotate(x, positions, freqs, interleaved, inverse):
    """x [Z, heads, N, D] by positions [Z, N]; angles in 64 bits, products in 32."""
    rot = 2 * freqs.numel()
    angle = positions.double()[:, None, :, None] * freqs
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if inverse:
        sin = -sin
    f = x.float()
    part, rest = f[..., :rot], f[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1).to(x.dtype)


def _run_rotary(s):
    case = s["case"]
    il = case["interleaved"]
    if case["kind"] == "fwd":
        if own:
            return fa().rotary(s["q"], s["k"], s["positions"], s["freqs"], interleaved=il)
        return (_rotate(s["q"], s["positions"], s["freqs"], il, False).contiguous(),
                _rotate(s["k"], s["positions"], s["freqs"], il, False).contiguous())
    if case["kind"] == "bwd":
        # back to the projections' layout
        if own:
            dq, dk = (torch.empty((t.shape[0], t.shape[2], t.shape[1], t.shape[3]), dtype=t.dtype,
                                  device=t.device).transpose(1, 2) for t in (s["dq"], s["dk"]))
            fa().rotary_bwd(s["dq"], s["dk"], s["positions"], s["freqs"], interleaved=il, out=(dq, dk))
            return dq, dk
        return (_rotate(s["dq"], s["positions"], s["freqs"], il, True),
                _rotate(s["dk"], s["positions"], s["freqs"], il, True))
    if own:
        q = fa().rotary_and_cache(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["slots"], s["k_cache"],
                                  s["v_cache"], interleaved=il)
        return q, s["k_cache"], s["v_cache"]
    q = _rotate(s["q"], s["positions"], s["freqs"], il, False).contiguous()
    k = _rotate(s["k"], s["positions"], s["freqs"], il, False).transpose(1, 2).flatten(0, 1)
    v = s["v"].transpose(1, 2).flatten(0, 1)
    slots = s["slots"].flatten()
    live = slots >= 0
    # a token without a slot rewrites the row of one that has one
    spare = torch.argmax(live.to(torch.int32))
    source = torch.where(live, torch.arange(slots.numel(), device=slots.device), spare)
    target = slots[source]
    s["k_cache"].flatten(0, 1)[target] = k[source]
    s["v_cache"].flatten(0, 1)[target] = v[source]
    return q, s["k_cache"], s["v_cache"]


def _visible(s):
    """[Z or 1, Nq, Nk] truth values: which keys a query of a dense case sees."""
    case = s["case"]
    Nq, Nk, mask = case["Nq"], case["Nk"], case["mask"]
    device = s["q"].device
    pos = torch.arange(Nk - Nq, Nk, device=device)[:, None]
    key = torch.arange(Nk, device=device)[None, :]
    if mask == "none":
        return torch.ones((1, Nq, Nk), dtype=torch.bool, device=device)
    if mask == "prefix":
        return (key <= pos)[None] | (key[None] < s["prefix"][:, None, None])
    seen = (key <= pos)[None]
    if mask == "window":
        seen = seen & (key > pos - s["window"])[None]
    if mask == "docs":
        seen = seen & (s["docs"][:, Nk - Nq:, None] == s["docs"][:, None, :])
    return seen


def _scores(q, k, scale, cap, slopes, pos, key, seen):
    """q [Z, Hkv, G, Nq, D], k [Z, Hkv, 1, Nk, D] in 32 bits -> (scores with -inf where hidden, tanh or None)."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    t = None
    if cap:
        t = torch.tanh(x / cap)
        x = cap * t
    if slopes is not None:
        x = x - slopes * (pos - key).abs()
    return torch.where(seen, x, NEG), t


def _softmax(x):
    """(p, lse) of each row; a row of -inf gives p = 0 and lse = -inf."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == NEG, 0.0, m))
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l > 0, l, 1.0), torch.where(m == NEG, 0.0, m) + torch.log(l)


def _run_scored(s):
    case = s["case"]
    cap, causal = case["cap"], case["mask"] in ("causal", "window", "docs")
    Z, H, Hkv, Nq, Nk, D = (case[x] for x in ("Z", "H", "Hkv", "Nq", "Nk", "D"))
    if own:
        ranges = None
        if case["mask"] == "docs":
            ranges = fa().key_ranges(Nq, Nk, doc_ids=s["docs"])
        elif case["mask"] == "prefix":
            ranges = fa().key_ranges(Nq, Nk, prefix_lens=s["prefix"])
        how = dict(causal=causal, scale=s["scale"], softcap=cap, slopes=s["slopes"], window=s["window"],
                   key_ranges=ranges)
        o, lse = fa().fwd_scored(s["q"], s["k"], s["v"], **how)
        if not case["train"]:
            return o, lse
        return (o, lse) + tuple(fa().bwd_scored(s["q"], s["k"], s["v"], o, s["do"], lse, **how))
    G = H // Hkv
    q = s["q"].float().reshape(Z, Hkv, G, Nq, D)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    pos = torch.arange(Nk - Nq, Nk, device=q.device, dtype=torch.float32)[:, None]
    key = torch.arange(Nk, device=q.device, dtype=torch.float32)[None, :]
    slopes = s["slopes"].reshape(1, Hkv, G, 1, 1) if s["slopes"] is not None else None
    x, t = _scores(q, k, s["scale"], cap, slopes, pos, key, _visible(s)[:, None, None])
    p, lse = _softmax(x)
    del x
    o = torch.matmul(p, v)
    out = (o.reshape(Z, H, Nq, D).to(s["q"].dtype), lse.reshape(Z, H, Nq))
    if not case["train"]:
        return out
    do = s["do"].float().reshape(Z, Hkv, G, Nq, D)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds = p * (ds - (o * do).sum(-1, keepdim=True))
    if cap:
        ds = ds * (1.0 - t * t)
    dq = torch.matmul(ds, k) * s["scale"]
    dk = (torch.matmul(ds.transpose(-1, -2), q) * s["scale"]).sum(2)
    dt = s["q"].dtype
    return out + (dq.reshape(Z, H, Nq, D).to(dt), dk.to(dt), dv.to(dt))


def _run_paged(s):
    case = s["case"]
    B, H, Hkv, Nq, D, page = (case[x] for x in ("B", "H", "Hkv", "Nq", "D", "page"))
    if own:
        return fa().fwd_paged_scored(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context_lens"],
                                     q_lens=s["q_lens"], causal=True, scale=s["scale"], softcap=case["cap"],
                                     slopes=s["slopes"], window=case["window"])
    G = H // Hkv
    table = s["block_table"].long()
    L = table.shape[1] * page
    k = s["k_cache"][table].reshape(B, L, Hkv, D).float().transpose(1, 2)[:, :, None]
    v = s["v_cache"][table].reshape(B, L, Hkv, D).float().transpose(1, 2)[:, :, None]
    q = s["q"].float().reshape(B, Hkv, G, Nq, D)
    ctx = s["context_lens"].long()[:, None, None]
    qn = ctx * 0 + Nq if s["q_lens"] is None else s["q_lens"].long()[:, None, None]
    row = torch.arange(Nq, device=q.device)[None, :, None]
    key = torch.arange(L, device=q.device)[None, None, :]
    pos = ctx - qn + row
    seen = (key <= pos) & (key < ctx) & (row < qn)
    if case["window"]:
        seen = seen & (key > pos - case["window"])
    slopes = s["slopes"].reshape(1, Hkv, G, 1, 1) if s["slopes"] is not None else None
    x, _ = _scores(q, k, s["scale"], case["cap"], slopes, pos.float()[:, None, None], key.float()[:, None, None],
                   seen[:, None, None])
    p, lse = _softmax(x)
    o = torch.matmul(p, v)
    return o.reshape(B, H, Nq, D).to(s["q"].dtype), lse.reshape(B, H, Nq)


def fa():
    import attention_sm_flashattention_gb300
    return attention_sm_flashattention_gb300


def run(state):
    return {"rotary": _run_rotary, "scored": _run_scored, "paged": _run_paged}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work


def _pairs(case):
    """Visible (query, key) pairs of one head, averaged over what the inputs draw."""
    Nq, Nk, mask = case["Nq"], case["Nk"], case["mask"]
    causal = Nq * (Nq + 1) / 2 + Nq * (Nk - Nq)
    if mask == "none":
        return Nq * Nk
    if mask == "window":
        w = max(1, Nk // 4)
        return float(sum(min(Nk - Nq + i + 1, w) for i in range(Nq)))
    if mask == "docs":  # documents of about N / 6 tokens
        r = 1.0 - 6.0 / max(Nk, 7)
        return min(causal, float(sum((1 - r ** (i + 1)) / (1 - r) for i in range(Nq))))
    if mask == "prefix":  # a prefix drawn evenly from 0 .. Nk
        return float(sum(n + (Nk - n) ** 2 / (2.0 * Nk) for n in (Nk - Nq + i + 1 for i in range(Nq))))
    return causal


def work(case):
    D, H, Hkv = case["D"], case["H"], case["Hkv"]
    if case["op"] == "rotary":
        Z, N = case["Z"], case["N"]
        heads = H + Hkv * (2 if case["kind"] == "cache" else 1)
        tokens = Z * N
        extra = tokens * (16 if case["kind"] == "cache" else 8)
        return {"bytes": 2 * 2 * tokens * heads * D + extra, "flops": 3 * tokens * (H + Hkv) * case["rot"]}
    if case["op"] == "scored":
        Z, Nq, Nk = case["Z"], case["Nq"], case["Nk"]
        q, kv = Z * H * Nq * D * 2, Z * Hkv * Nk * D * 2
        fwd = 4.0 * D * Z * H * _pairs(case)
        if not case["train"]:
            return {"bytes": 2 * q + 2 * kv + 4 * Z * H * Nq, "flops": fwd}
        return {"bytes": 4 * q + 4 * kv + 4 * Z * H * Nq, "flops": 3.5 * fwd}
    B, Nq, ctx = case["B"], case["Nq"], case["ctx"]
    # ragged: lengths drawn evenly from a quarter of the longest to the longest, chunks from 1 to Nq
    n = ctx if not case["ragged"] else (ctx + (B - 1) * 0.625 * ctx) / B
    nq = Nq if not case["ragged"] else (Nq + (B - 1) * (Nq + 1) / 2) / B
    seen = min(n, nq - 1 + case["window"]) if case["window"] else n
    pairs = nq * min(n - (nq - 1) / 2, case["window"] or n)
    return {"bytes": 2 * 2 * B * H * nq * D + 2 * 2 * B * Hkv * seen * D + 4 * B * H * nq,
            "flops": 4.0 * D * B * H * pairs}


# ------------------------------------------------------------------- exact


def _exact_turn(x, positions, freqs, interleaved, sign):
    """As a complex product: each pair of values times e^(i angle)."""
    rot = 2 * freqs.numel()
    w = torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(positions.shape + freqs.shape),
                    sign * positions.double()[..., None] * freqs)[:, None]
    y = x.double().clone()
    if interleaved:
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * w
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_attend(q, k, v, scale, cap, bias, hidden):
    """One softmax attention in 64 bits over heads of equal number; hidden: truth values, bias: added."""
    x = torch.einsum("bhid,bhjd->bhij", q, k) * scale
    if cap:
        x = torch.tanh(x / cap) * cap
    if bias is not None:
        x = x + bias
    x = x.masked_fill(hidden, -1e300)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None]).masked_fill(hidden, 0.0)
    none = hidden.expand_as(x).all(-1)
    return torch.einsum("bhij,bhjd->bhid", p, v), lse.masked_fill(none, NEG)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        il = case["interleaved"]
        if case["kind"] == "bwd":
            return tuple(_exact_turn(s[n], s["positions"], s["freqs"], il, -1.0) for n in ("dq", "dk"))
        q = _exact_turn(s["q"], s["positions"], s["freqs"], il, 1.0)
        k = _exact_turn(s["k"], s["positions"], s["freqs"], il, 1.0)
        if case["kind"] == "fwd":
            return q, k
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        z, i = torch.nonzero(s["slots"] >= 0, as_tuple=True)
        at = s["slots"][z, i]
        kc[at // case["page"], at % case["page"]] = k[z, :, i]
        vc[at // case["page"], at % case["page"]] = s["v"][z, :, i].double()
        return q, kc, vc
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    G = H // Hkv
    device = s["q"].device
    if case["op"] == "scored":
        Z, Nq, Nk = case["Z"], case["Nq"], case["Nk"]
        leaves = [s[n].double().requires_grad_(case["train"]) for n in ("q", "k", "v")]
        pos = torch.arange(Nq, device=device) + (Nk - Nq)
        key = torch.arange(Nk, device=device)
        far = pos[:, None] - key[None, :]
        if case["mask"] == "none":
            hidden = torch.zeros_like(far, dtype=torch.bool)[None]
        elif case["mask"] == "prefix":
            hidden = (far < 0)[None] & (key[None, None, :] >= s["prefix"][:, None, None])
        else:
            hidden = (far < 0)[None]
            if case["mask"] == "window":
                hidden = hidden | (far >= s["window"])[None]
            if case["mask"] == "docs":
                hidden = hidden | (s["docs"][:, Nk - Nq:][:, :, None] != s["docs"][:, None, :])
        bias = None if s["slopes"] is None else -s["slopes"].double()[None, :, None, None] * far.abs()
        q, k, v = leaves
        o, lse = _exact_attend(q, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1), s["scale"], case["cap"], bias,
                               hidden[:, None])
        if not case["train"]:
            return o, lse
        grads = torch.autograd.grad(o, leaves, s["do"].double())
        return (o.detach(), lse.detach()) + tuple(grads)
    B, Nq, page = case["B"], case["Nq"], case["page"]
    o = torch.zeros((B, H, Nq, D), dtype=torch.float64, device=device)
    lse = torch.full((B, H, Nq), NEG, dtype=torch.float64, device=device)
    for b in range(B):
        n = int(s["context_lens"][b])
        m = Nq if s["q_lens"] is None else int(s["q_lens"][b])
        at = torch.arange(n, device=device)
        page_of = s["block_table"][b].long()[at // page]
        k = s["k_cache"][page_of, at % page].double().transpose(0, 1).repeat_interleave(G, 0)[None]
        v = s["v_cache"][page_of, at % page].double().transpose(0, 1).repeat_interleave(G, 0)[None]
        far = (torch.arange(m, device=device) + (n - m))[:, None] - at[None, :]
        hidden = far < 0
        if case["window"]:
            hidden = hidden | (far >= case["window"])
        bias = None if s["slopes"] is None else -s["slopes"].double()[None, :, None, None] * far.abs()
        o[b:b + 1, :, :m], lse[b:b + 1, :, :m] = _exact_attend(s["q"][b:b + 1, :, :m].double(), k, v, s["scale"],
                                                              case["cap"], bias, hidden[None, None])
    return o, lse
