"""Cases of the page-table, several-axes rotary and window-with-sinks operators, with their plain forms.

Three families, each with its plain form in elementary torch operations and the call that a user makes:

* ``step`` / ``release``: the paged cache's tables, kept on the GPU: pages for the new tokens of every sequence from a
  stack of free ones, the slots and positions of those tokens, and the pages of finished sequences back on the stack.
* ``rotary``: rotary positions with several axes (time, height, width), each pair of values turned by the position on
  its own axis: forward, the gradients' way back, and the serving form that writes the paged cache.
* ``sinks``: attention within a sliding window that also sees the first few tokens: forward, with its gradients, and
  over a paged cache for a chunk of new tokens per sequence or for single ones.
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
NEG = float("-inf")


# ------------------------------------------------------------------- cases


def _step(name, B, N, ctx, page, ragged):
    return {"name": name, "op": "step", "B": B, "N": N, "ctx": ctx, "page": page, "ragged": ragged}


def _release(name, B, ctx, page, share):
    return {"name": name, "op": "release", "B": B, "ctx": ctx, "page": page, "share": share}


def _rotary(name, kind, Z, H, Hkv, N, D, rot, axes, dealt, interleaved, dtype, far, page=64):
    return {"name": name, "op": "rotary", "kind": kind, "Z": Z, "H": H, "Hkv": Hkv, "N": N, "D": D, "rot": rot,
            "axes": axes, "dealt": dealt, "interleaved": interleaved, "dtype": dtype, "far": far, "page": page}


def _dense(name, train, Z, H, Hkv, Nq, Nk, D, window, sinks, cap, dtype):
    return {"name": name, "op": "dense", "train": train, "Z": Z, "H": H, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "D": D,
            "window": window, "sinks": sinks, "cap": cap, "dtype": dtype}


def _paged(name, B, H, Hkv, Nq, ctx, D, page, window, sinks, cap, dtype, ragged):
    return {"name": name, "op": "paged", "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "ctx": ctx, "D": D, "page": page,
            "window": window, "sinks": sinks, "cap": cap, "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # one decode step of a batch: a slot and a position per sequence, a new page for some
        _step("step_token", 64, 1, 8192, 16, False),
        # prefill of a large batch of uneven prompts behind uneven caches
        _step("step_prefill", 512, 2048, 16384, 64, True),
        # a third of a serving batch has finished: its pages go back
        _release("release_batch", 256, 32768, 16, 0.33),
        # one sequence of a small batch has finished
        _release("release_few", 16, 4096, 64, 0.05),
        # a training micro-batch of video tokens: three axes in blocks, whole head turned
        _rotary("rotary_video_train", "fwd", 4, 32, 8, 8192, 128, 128, 3, False, False, "bf16", 1000),
        # gradients of an image encoder: two axes, odd number of patches, half of the head
        _rotary("rotary_image_grad_odd", "bwd", 3, 16, 16, 1021, 64, 32, 2, False, False, "fp16", 0),
        # chunked prefill of image and text tokens: three axes dealt in turn, into the cache
        _rotary("rotary_chunk_cache", "cache", 8, 32, 8, 512, 128, 128, 3, True, True, "bf16", 30000),
        # training step at a long context: grouped heads, four first tokens stay visible
        _dense("sinks_train_long", True, 2, 16, 4, 8192, 8192, 128, 1024, 4, 0.0, "bf16"),
        # training step of odd length with small heads and a hundred kept tokens
        _dense("sinks_train_odd", True, 3, 8, 8, 1021, 1021, 64, 257, 100, 0.0, "fp16"),
        # prefill of a capped model with wide heads
        _dense("sinks_prefill_d256", False, 4, 8, 4, 4096, 4096, 256, 512, 4, 50.0, "bf16"),
        # decode of a large batch far behind the window's start: only the window and the sinks are read
        _paged("sinks_token", 64, 32, 8, 1, 32768, 128, 16, 4096, 4, 0.0, "bf16", True),
        # chunked prefill behind a long cache
        _paged("sinks_chunk", 8, 32, 8, 512, 8192, 128, 64, 1024, 64, 30.0, "fp16", True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "release", "rotary", "rotary", "dense", "dense", "paged", "paged"])
    dtype = rng.choice(["fp16", "bf16"])
    page = rng.choice([16, 32, 64])
    D = rng.choice([64, 64, 128, 128, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 8])
    if op == "step":
        B, N = _log(rng, 1, 2048), 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        while B * N > 512 * 2048:
            B = (B + 1) // 2
        c = _step("", B, N, _log(rng, max(16, N), 32768), page, rng.random() < 0.7)
    elif op == "release":
        c = _release("", _log(rng, 1, 1024), _log(rng, 16, 32768), page, rng.choice([0.05, 0.33, 0.9]))
    elif op == "rotary":
        kind = rng.choice(["fwd", "bwd", "cache"])
        c = _rotary("", kind, _log(rng, 1, 16), H, Hkv, _log(rng, 1, 8192 if kind != "cache" else 1024), D,
                    rng.choice([D, D, D // 2, D // 4, 20]), rng.choice([2, 3, 3, 4]), rng.random() < 0.5,
                    rng.random() < 0.5, dtype, _log(rng, 1, 1000000), page)
        while work(c)["bytes"] > 6.7e8:
            at = "Z" if c["Z"] > 1 else "N"
            c[at] = (c[at] + 1) // 2
    elif op == "dense":
        train = rng.random() < 0.6
        # a softmax over one key has no gradient, so training starts at lengths that have some
        Nk = _log(rng, 32 if train else 1, 8192)
        Nq = Nk if rng.random() < 0.7 else _log(rng, 1, Nk)
        c = _dense("", train, _log(rng, 1, 16), H, Hkv, Nq, Nk, D, _log(rng, 16 if train else 1, 2048),
                   _log(rng, 1, 256), rng.choice([0.0, 0.0, 50.0]), dtype)
        _shrink(c, "Z", 2 * 16 * 8192 * 8192)
    else:
        Nq = 1 if rng.random() < 0.6 else _log(rng, 2, 512)
        c = _paged("", _log(rng, 1, 64) if Nq == 1 else _log(rng, 1, 8), H, Hkv, Nq,
                   _log(rng, max(1, Nq), 32768 if Nq == 1 else 8192), D, page, _log(rng, 1, 4096), _log(rng, 1, 256),
                   rng.choice([0.0, 0.0, 30.0]), dtype, rng.random() < 0.8)
        _shrink(c, "B", 8 * 32 * 512 * 8192)
    c.pop("name")
    return c


def _shrink(c, batch, cells):
    """Fewer sequences, then heads, until the plain form's scores and the cache are no larger than the listed cases'."""
    def over():
        keys = c.get("Nk", c.get("ctx"))
        return c[batch] * c["H"] * c["Nq"] * keys > cells or c[batch] * c["Hkv"] * keys * c["D"] > 64 * 8 * 32768 * 128 \
            or work(c)["flops"] > 2e12

    while over():
        if c[batch] > 1:
            c[batch] = (c[batch] + 1) // 2
        elif c["Hkv"] > 1:
            group, c["Hkv"] = c["H"] // c["Hkv"], c["Hkv"] // 2
            c["H"] = group * c["Hkv"]
        else:
            c["H"] = max(1, c["H"] // 2)


# ------------------------------------------------------------------ inputs


def _slots_free(gen, pages, used, device):
    """(the pages that are taken, the stack of free ones and its height) of a pool of `pages`."""
    order = torch.randperm(pages, generator=gen, device=device).to(torch.int32)
    stack = torch.zeros(pages, dtype=torch.int32, device=device)
    stack[:pages - used] = order[used:]
    return order[:used], stack, torch.tensor([pages - used], dtype=torch.int32, device=device)


def _grid_positions(gen, Z, N, axes, far, device):
    """[axes, Z, N]: tokens of frames of 28 by 28 patches behind up to `far` earlier positions, time first where there is
    one; a fourth axis counts the tokens."""
    first = torch.randint(0, far + 1, (Z, 1), generator=gen, device=device)
    n = torch.arange(N, device=device)[None, :] + torch.randint(0, 784, (Z, 1), generator=gen, device=device)
    time, height, width = n // 784, n // 28 % 28, n % 28
    return torch.stack([time, height, width, n][:axes] if axes > 2 else [height, width]) + first


def _axis_of(rot, axes, dealt, device):
    """int32 [rot / 2]: the axis of each pair, in blocks (the first takes what does not divide) or dealt in turn."""
    pairs = torch.arange(rot // 2, device=device)
    if dealt:
        return (pairs % axes).to(torch.int32)
    block = rot // 2 // axes
    return torch.clamp((pairs - (rot // 2 - block * axes)) // max(block, 1), min=0, max=axes - 1).to(torch.int32)


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=device).manual_seed(int(seed))
    s = {"case": case}
    if case["op"] in ("step", "release"):
        B, page = case["B"], case["page"]
        max_pages = (case["ctx"] + page - 1) // page
        cached = torch.randint(0, case["ctx"] + 1, (B,), generator=gen, device=device)
        if case["op"] == "step":
            N = case["N"]
            cached = torch.clamp(cached, max=case["ctx"] - N) if case["ctx"] > N else cached * 0
            s["q_lens"] = torch.randint(0, N + 1, (B,), generator=gen, device=device).to(torch.int32) \
                if case["ragged"] else None
        else:
            s["finished"] = torch.rand((B,), generator=gen, device=device) < case["share"]
        taken = (cached + page - 1) // page
        table = torch.full((B, max_pages), -1, dtype=torch.int32, device=device)
        live = torch.arange(max_pages, device=device)[None, :] < taken[:, None]
        pages = B * max_pages + 7
        ids, s["free_pages"], s["free_count"] = _slots_free(gen, pages, int(taken.sum()), device)
        table[live] = ids
        s["block_table"], s["lens"] = table, cached.to(torch.int32)
        return s
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=device, dtype=torch.float32)

    D, H, Hkv = case["D"], case["H"], case["Hkv"]
    if case["op"] == "rotary":
        Z, N, rot = case["Z"], case["N"], case["rot"]
        s["freqs"] = torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64) / rot).to(device)
        s["positions"] = _grid_positions(gen, Z, N, case["axes"], case["far"], device)
        s["axes"] = _axis_of(rot, case["axes"], case["dealt"], device)
        if case["kind"] == "bwd":  # gradients as the attention's backward leaves them
            s["dq"], s["dk"] = normal(Z, H, N, D).to(dt), normal(Z, Hkv, N, D).to(dt)
        else:  # one projection's output, q, k and v beside each other
            qkv = normal(Z, N, H + 2 * Hkv, D).to(dt)
            s["q"] = qkv[:, :, :H].transpose(1, 2)
            s["k"] = qkv[:, :, H:H + Hkv].transpose(1, 2)
            s["v"] = qkv[:, :, H + Hkv:].transpose(1, 2)
        if case["kind"] == "cache":
            page = case["page"]
            pages = (Z * N + page - 1) // page + 3
            s["k_cache"] = torch.zeros((pages, page, Hkv, D), device=device, dtype=dt)
            s["v_cache"] = torch.zeros_like(s["k_cache"])
            s["slots"] = torch.randperm(pages * page, generator=gen, device=device)[:Z * N].reshape(Z, N).contiguous()
        return s
    # what makes first tokens sinks: queries share a direction that those keys have too, and their values are small
    # (capped scores: there because products get large, so the queries are wider)
    s["scale"] = 1.0 / math.sqrt(D)
    wide = 2.0 if case["cap"] else 1.0
    Nq, sinks = case["Nq"], case["sinks"]
    if case["op"] == "dense":
        Z, Nk = case["Z"], case["Nk"]
        s["q"] = ((normal(Z, H, Nq, D) + 0.5) * wide).to(dt)
        k, v = normal(Z, Hkv, Nk, D), normal(Z, Hkv, Nk, D)
        k[:, :, :sinks] += 0.7
        v[:, :, :sinks] *= 0.1
        s["k"], s["v"] = k.to(dt), v.to(dt)
        s["do"] = normal(Z, H, Nq, D).to(dt) if case["train"] else None
        return s
    B, page, ctx = case["B"], case["page"], case["ctx"]
    s["q"] = ((normal(B, H, Nq, D) + 0.5) * wide).to(dt)
    lens = torch.full((B,), ctx, device=device)
    s["q_lens"] = None
    if case["ragged"]:  # the first sequence has the longest context and a full chunk
        lens = torch.randint(max(1, ctx // 4), ctx + 1, (B,), generator=gen, device=device)
        qs = torch.randint(1, Nq + 1, (B,), generator=gen, device=device)
        lens[0], qs[0] = ctx, Nq
        s["q_lens"] = torch.minimum(qs, lens).to(torch.int32)
    s["context_lens"] = lens.to(torch.int32)
    max_pages = (ctx + page - 1) // page
    pages = B * max_pages + 1
    s["k_cache"], s["v_cache"] = normal(pages, page, Hkv, D).to(dt), normal(pages, page, Hkv, D).to(dt)
    table = torch.randperm(pages, generator=gen, device=device)[:B * max_pages].reshape(B, max_pages)
    s["block_table"] = table.to(torch.int32).contiguous()
    at = torch.arange(min(sinks, ctx), device=device)
    where = (table[:, at // page], (at % page)[None, :].expand(B, -1))
    s["k_cache"][where] += 0.7
    s["v_cache"][where] *= 0.1
    return s


# ------------------------------------------------------------- plain forms


def _run_step(s):
    case = s["case"]
    N, page, table = case["N"], case["page"], s["block_table"]
    if own:
        slots, positions, lens, count = fa().cache_step(s["free_pages"], s["free_count"], table, s["lens"], s["q_lens"],
                                                        N, page)
        return slots, positions, lens, count, table
    pages = s["free_pages"].numel()
    max_pages = table.shape[1]
    have = s["lens"].long().clamp(min=0)
    new = torch.full_like(have, N) if s["q_lens"] is None else s["q_lens"].long().clamp(0, N)
    end = have + new
    first = ((have + page - 1) // page).clamp(max=max_pages)
    need = ((end + page - 1) // page).clamp(max=max_pages) - first
    before = torch.cumsum(need, 0) - need
    free = s["free_count"].long().clamp(0, pages)
    at = torch.arange(max_pages, device=table.device)[None, :]
    nth = at - first[:, None] + before[:, None]  # of the pages that this step takes
    taken = s["free_pages"][(free - 1 - nth).clamp(0, pages - 1)]
    taken = torch.where(nth < free, taken, -1)
    fresh = (at >= first[:, None]) & (at < (first + need)[:, None])
    table.copy_(torch.where(fresh, taken, table))
    n = torch.arange(N, device=table.device)[None, :]
    positions = have[:, None] + n
    entry = torch.gather(table.long(), 1, (positions // page).clamp(max=max_pages - 1))
    live = (n < new[:, None]) & (positions // page < max_pages) & (entry >= 0) & (entry < pages)
    slots = torch.where(live, entry * page + positions % page, -1)
    return slots, positions, end.to(torch.int32), (free - need.sum()).to(torch.int32), table


def _run_release(s):
    case = s["case"]
    page, table = case["page"], s["block_table"]
    if own:
        lens, count = fa().cache_release(s["free_pages"], s["free_count"], table, s["lens"], s["finished"], page)
        return lens, count, s["free_pages"]
    pages = s["free_pages"].numel()
    held = (s["lens"].long().clamp(min=0) + page - 1) // page
    at = torch.arange(table.shape[1], device=table.device)[None, :]
    back = s["finished"][:, None] & (at < held[:, None]) & (table >= 0) & (table < pages)
    free = s["free_count"].long().clamp(0, pages)
    place = free + torch.cumsum(back.flatten().long(), 0) - 1  # where each goes on the stack
    # entries that stay write the last place of a longer copy
    place = torch.where(back.flatten() & (place < pages), place, pages)
    stack = torch.cat((s["free_pages"], s["free_pages"][:1]))
    stack[place] = table.flatten()
    s["free_pages"].copy_(stack[:pages])
    count = (free + back.sum()).clamp(max=pages).to(torch.int32)
    return torch.where(s["finished"], 0, s["lens"]), count, s["free_pages"]


def _rotate(x, positions, axes, freqs, interleaved, inverse):
    """x [Z, heads, N, D] by positions [axes, Z, N]; angles in 64 bits, products in 32."""
    rot = 2 * freqs.numel()
    angle = (positions[axes.long()].double() * freqs[:, None, None]).permute(1, 2, 0)[:, None]
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
    il, how = case["interleaved"], (s["positions"], s["axes"], s["freqs"])
    if case["kind"] == "fwd":
        if own:
            return fa().rotary(s["q"], s["k"], s["positions"], s["freqs"], interleaved=il, axes=s["axes"])
        return _rotate(s["q"], *how, il, False).contiguous(), _rotate(s["k"], *how, il, False).contiguous()
    if case["kind"] == "bwd":
        # back to the projections' layout
        if own:
            dq, dk = (torch.empty((t.shape[0], t.shape[2], t.shape[1], t.shape[3]), dtype=t.dtype,
                                  device=t.device).transpose(1, 2) for t in (s["dq"], s["dk"]))
            fa().rotary_bwd(s["dq"], s["dk"], s["positions"], s["freqs"], interleaved=il, out=(dq, dk), axes=s["axes"])
            return dq, dk
        return _rotate(s["dq"], *how, il, True), _rotate(s["dk"], *how, il, True)
    if own:
        q = fa().rotary_and_cache(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["slots"], s["k_cache"],
                                  s["v_cache"], interleaved=il, axes=s["axes"])
        return q, s["k_cache"], s["v_cache"]
    q = _rotate(s["q"], *how, il, False).contiguous()
    slots = s["slots"].flatten()
    s["k_cache"].flatten(0, 1)[slots] = _rotate(s["k"], *how, il, False).transpose(1, 2).flatten(0, 1)
    s["v_cache"].flatten(0, 1)[slots] = s["v"].transpose(1, 2).flatten(0, 1)
    return q, s["k_cache"], s["v_cache"]


def _softmax(q, k, scale, cap, seen):
    """q [.., Nq, D], k [.., Nk, D] in 32 bits -> (p, lse, tanh or None); a row that sees nothing: p = 0, lse = -inf."""
    x, t = torch.matmul(q, k.transpose(-1, -2)) * scale, None
    if cap:
        t = torch.tanh(x / cap)
        x = cap * t
    x = torch.where(seen, x, NEG)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, 0.0, m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0), m + torch.log(total), t


def _run_dense(s):
    case = s["case"]
    cap, window, sinks = case["cap"], case["window"], case["sinks"]
    Z, H, Hkv, Nq, Nk, D = (case[x] for x in ("Z", "H", "Hkv", "Nq", "Nk", "D"))
    if own:
        how = dict(causal=True, scale=s["scale"], softcap=cap, window=window, sinks=sinks)
        o, lse = fa().fwd_scored(s["q"], s["k"], s["v"], **how)
        if not case["train"]:
            return o, lse
        return (o, lse) + tuple(fa().bwd_scored(s["q"], s["k"], s["v"], o, s["do"], lse, **how))
    q = s["q"].float().reshape(Z, Hkv, H // Hkv, Nq, D)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    pos = torch.arange(Nk - Nq, Nk, device=q.device)[:, None]
    key = torch.arange(Nk, device=q.device)[None, :]
    seen = (key <= pos) & ((key > pos - window) | (key < sinks))
    p, lse, t = _softmax(q, k, s["scale"], cap, seen)
    o = torch.matmul(p, v)
    dt = s["q"].dtype
    out = (o.reshape(Z, H, Nq, D).to(dt), lse.reshape(Z, H, Nq))
    if not case["train"]:
        return out
    do = s["do"].float().reshape(q.shape)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (o * do).sum(-1, keepdim=True))
    if cap:
        ds = ds * (1.0 - t * t)
    dq = torch.matmul(ds, k) * s["scale"]
    dk = (torch.matmul(ds.transpose(-1, -2), q) * s["scale"]).sum(2)
    return out + (dq.reshape(Z, H, Nq, D).to(dt), dk.to(dt), dv.to(dt))


def _run_paged(s):
    case = s["case"]
    B, H, Hkv, Nq, D, page = (case[x] for x in ("B", "H", "Hkv", "Nq", "D", "page"))
    if own:
        return fa().fwd_paged_scored(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context_lens"],
                                     q_lens=s["q_lens"], causal=True, scale=s["scale"], softcap=case["cap"],
                                     window=case["window"], sinks=case["sinks"])
    table = s["block_table"].long()
    L = table.shape[1] * page
    k = s["k_cache"][table].reshape(B, L, Hkv, D).float().transpose(1, 2)[:, :, None]
    v = s["v_cache"][table].reshape(B, L, Hkv, D).float().transpose(1, 2)[:, :, None]
    ctx = s["context_lens"].long()[:, None, None]
    qn = torch.full_like(ctx, Nq) if s["q_lens"] is None else s["q_lens"].long()[:, None, None]
    row = torch.arange(Nq, device=k.device)[None, :, None]
    key = torch.arange(L, device=k.device)[None, None, :]
    pos = ctx - qn + row
    seen = (key <= pos) & (row < qn) & ((key > pos - case["window"]) | (key < case["sinks"]))
    q = s["q"].float().reshape(B, Hkv, H // Hkv, Nq, D)
    p, lse, _ = _softmax(q, k, s["scale"], case["cap"], seen[:, None, None])
    return torch.matmul(p, v).reshape(B, H, Nq, D).to(s["q"].dtype), lse.reshape(B, H, Nq)


def fa():
    import attention_sm_flashattention_gb300
    return attention_sm_flashattention_gb300


_RUN = {"step": _run_step, "release": _run_release, "rotary": _run_rotary, "dense": _run_dense, "paged": _run_paged}


def run(state):
    return _RUN[state["case"]["op"]](state)


# -------------------------------------------------------------------- work


def _seen_keys(last, window, sinks):
    """Keys that the query at position `last` sees."""
    return min(last + 1, window) + max(0, min(sinks, last + 1 - window))


def work(case):
    op = case["op"]
    if op == "step":  # lengths in and out, a slot and a position per token, the pages of the new tokens in and out
        B, N, page = case["B"], case["N"], case["page"]
        new = N / 2 if case["ragged"] else N
        return {"bytes": B * (12 + 16 * N + 8 * new / page + 4), "flops": 0}
    if op == "release":  # the finished rows' entries, to the stack
        B, page = case["B"], case["page"]
        return {"bytes": B * (9 + case["share"] * 8 * (case["ctx"] / 2 / page + 0.5)), "flops": 0}
    D, H, Hkv = case["D"], case["H"], case["Hkv"]
    if op == "rotary":
        heads = H + Hkv * (2 if case["kind"] == "cache" else 1)
        tokens = case["Z"] * case["N"]
        extra = tokens * 8 * (case["axes"] + (1 if case["kind"] == "cache" else 0))
        return {"bytes": 2 * 2 * tokens * heads * D + extra, "flops": 3 * tokens * (H + Hkv) * case["rot"]}
    window, sinks = case["window"], case["sinks"]
    if op == "dense":
        Z, Nq, Nk = case["Z"], case["Nq"], case["Nk"]
        # keys from the first query's window on, and the sinks
        keys = min(Nk, Nq - 1 + min(window, Nk - Nq + 1) + min(sinks, max(0, Nk - Nq + 1 - window)))
        q, kv = Z * H * Nq * D * 2, Z * Hkv * keys * D * 2
        pairs = float(sum(_seen_keys(Nk - Nq + i, window, sinks) for i in range(Nq)))
        fwd = 4.0 * D * Z * H * pairs
        if not case["train"]:
            return {"bytes": 2 * q + 2 * kv + 4 * Z * H * Nq, "flops": fwd}
        return {"bytes": 4 * q + 2 * kv + 2 * Z * Hkv * Nk * D * 2 + 4 * Z * H * Nq, "flops": 3.5 * fwd}
    B, Nq, ctx = case["B"], case["Nq"], case["ctx"]
    # ragged: lengths drawn evenly from a quarter of the longest to the longest, chunks from 1 to Nq
    n = ctx if not case["ragged"] else (ctx + (B - 1) * 0.625 * ctx) / B
    nq = Nq if not case["ragged"] else (Nq + (B - 1) * (Nq + 1) / 2) / B
    keys = min(n, nq - 1 + window + sinks)
    pairs = nq * _seen_keys(n - (nq + 1) / 2, window, sinks)
    return {"bytes": 2 * 2 * B * H * nq * D + 2 * 2 * B * Hkv * keys * D + 4 * B * H * nq, "flops": 4.0 * D * B * H * pairs}


# ------------------------------------------------------------------- exact


def _exact_turn(x, positions, axes, freqs, interleaved, sign):
    """As a complex product: each pair of values times e^(i angle)."""
    rot = 2 * freqs.numel()
    turns = torch.stack([positions[int(a)].double() * f for a, f in zip(axes.tolist(), freqs)], -1) * sign
    w = torch.polar(torch.ones_like(turns), turns)[:, None]
    y = x.double().clone()
    if interleaved:
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * w
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_attend(q, k, v, scale, cap, hidden):
    """One softmax attention in 64 bits over heads of equal number; hidden: truth values."""
    x = torch.einsum("bhid,bhjd->bhij", q, k) * scale
    if cap:
        x = torch.tanh(x / cap) * cap
    x = x.masked_fill(hidden, -1e300)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None]).masked_fill(hidden, 0.0)
    none = hidden.expand_as(x).all(-1)
    return torch.einsum("bhij,bhjd->bhid", p, v), lse.masked_fill(none, NEG)


def _hidden(pos, keys, window, sinks):
    far = pos[:, None] - torch.arange(keys, device=pos.device)[None, :]
    hidden = (far < 0) | (far >= window)
    hidden[:, :sinks] = far[:, :sinks] < 0
    return hidden


def exact(case, seed):
    if case["op"] in ("step", "release"):
        return None  # whole numbers
    s = prepare(case, seed)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        il, how = case["interleaved"], (s["positions"], s["axes"], s["freqs"])
        if case["kind"] == "bwd":
            return tuple(_exact_turn(s[n], *how, il, -1.0) for n in ("dq", "dk"))
        q, k = _exact_turn(s["q"], *how, il, 1.0), _exact_turn(s["k"], *how, il, 1.0)
        if case["kind"] == "fwd":
            return q, k
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        at, page = s["slots"].flatten(), case["page"]
        kc[at // page, at % page] = k.transpose(1, 2).flatten(0, 1)
        vc[at // page, at % page] = s["v"].double().transpose(1, 2).flatten(0, 1)
        return q, kc, vc
    G, window, sinks = H // Hkv, case["window"], case["sinks"]
    device = s["q"].device
    if case["op"] == "dense":
        Nq, Nk = case["Nq"], case["Nk"]
        hidden = _hidden(torch.arange(Nk - Nq, Nk, device=device), Nk, window, sinks)
        out = []
        for z in range(case["Z"]):  # one sequence and key head at a time: the scores in 64 bits are large
            for h in range(Hkv):
                part = [s[n][z:z + 1, i * h:i * h + i].double().requires_grad_(case["train"])
                        for n, i in (("q", G), ("k", 1), ("v", 1))]
                q, k, v = part
                o, lse = _exact_attend(q, k.expand(-1, G, -1, -1), v.expand(-1, G, -1, -1), s["scale"], case["cap"],
                                       hidden)
                grads = torch.autograd.grad(o, part, s["do"][z:z + 1, G * h:G * h + G].double()) if case["train"] else ()
                out.append((o.detach(), lse.detach()) + tuple(grads))
        return tuple(torch.cat([torch.cat(x[z * Hkv:(z + 1) * Hkv], 1) for z in range(case["Z"])]) for x in zip(*out))
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
        pos = torch.arange(n - m, n, device=device)
        first = max(0, m - n)  # rows before position 0 see nothing
        o[b, :, first:m], lse[b, :, first:m] = (x[0] for x in _exact_attend(
            s["q"][b:b + 1, :, first:m].double(), k, v, s["scale"], case["cap"], _hidden(pos[first:], n, window, sinks)))
    return o, lse
