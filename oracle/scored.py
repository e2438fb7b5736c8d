"""fp64 CPU oracle of scored attention and rotary positions.

Scores x = scale * q.k, capped to cap * tanh(x / cap), minus slope * |position
- key|, hidden outside each query's visible keys; forward, gradients, and the
paged form.  Everything is materialised per head in float64 numpy.  Besides
the values, each function returns how far a 16-bit kernel that rounds P, dS
and its outputs once each may be off, element by element.
"""

from __future__ import annotations

import numpy as np
import torch

# Half a step of each 16-bit type, relative to the value, and the absolute
# rounding below its smallest normal number (fp16: half of 2^-24; bf16 has
# fp32's range).
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
F32 = 2.0 ** -24


def _f64(t):
    return t.detach().to(torch.float64).cpu().numpy() if isinstance(t, torch.Tensor) else np.asarray(t, np.float64)


def _scale64(scale):
    """The scale as the calls take it: a 32-bit float."""
    return float(np.float32(scale))


def visible(Nq, Nk, causal=False, window=0, docs=None, prefix=None, ranges=None):
    """[Nq, Nk] truth values for one sequence (the queries are the last Nq of
    Nk positions)."""
    pos = np.arange(Nk - Nq, Nk)[:, None]
    key = np.arange(Nk)[None, :]
    seen = np.ones((Nq, Nk), bool)
    if causal:
        seen &= key <= pos
    if window:
        seen &= key > pos - window
    if docs is not None:
        docs = np.asarray(docs)
        run = np.cumsum(np.concatenate([[0], (docs[1:] != docs[:-1]).astype(int)]))
        seen &= run[Nk - Nq:][:, None] == run[None, :]
    if prefix is not None:
        seen &= (key <= pos) | (key < int(prefix))
    if ranges is not None:
        r = np.asarray(ranges)
        seen &= (key >= r[:, :1]) & (key < r[:, 1:])
    return seen


def head_scores(q, k, scale, cap, slope, pos, key):
    """(x, tanh or None) of one head, before hiding."""
    x = (q @ k.T) * scale
    t = None
    if cap:
        t = np.tanh(x / cap)
        x = cap * t
    if slope:
        x = x - slope * np.abs(pos[:, None] - key[None, :])
    return x, t


def head_fwd(q, k, v, scale, cap, slope, seen, pos, key):
    """(o, lse, p, tanh) of one head; rows that see nothing give 0 and -inf."""
    x, t = head_scores(q, k, scale, cap, slope, pos, key)
    x = np.where(seen, x, -np.inf)
    m = x.max(1, keepdims=True)
    some = np.isfinite(m)
    with np.errstate(all="ignore"):
        e = np.where(seen, np.exp(x - np.where(some, m, 0.0)), 0.0)
        l = e.sum(1, keepdims=True)
        p = e / np.where(l > 0, l, 1.0)
        lse = np.where(l > 0, np.where(some, m, 0.0) + np.log(np.where(l > 0, l, 1.0)), -np.inf)[:, 0]
    return p @ v, lse, p, t


def score_slack(q, k, scale, cap, slope, pos, key):
    """Absolute error of an fp32 score: the dot product's D roundings, the cap's
    exp2, reciprocal and fma (16 half steps of cap), and the bias."""
    D = q.shape[1]
    dot = (np.abs(q) @ np.abs(k).T).max() * scale
    far = np.abs(pos[:, None] - key[None, :]).max() * abs(slope) if slope else 0.0
    return F32 * (D * dot + 16 * cap + 8 * far + 8)


def fwd_bound(o, p, v, slack, dtype, Nk):
    """How far a kernel's o may be from exact: P rounded (and, in fp16, below
    2^-14 of the row's largest, to 2^-25), its own rounding, the scores'."""
    u = HALF_STEP[dtype]
    pv = p @ np.abs(v)
    far = 2 * (slack + F32 * 64) * pv + u * pv + u * np.abs(o) + TINY[dtype]
    return far + TINY[dtype] * Nk * np.abs(v).max()


def scored_fwd(q, k, v, scale, cap=0.0, slopes=None, seen=None, dtype=torch.float16):
    """q [Z,H,Nq,D], k, v [Z,Hkv,Nk,D], seen(z) -> [Nq,Nk].  Returns (o, lse,
    bound of o, bound of lse)."""
    q, k, v, scale = _f64(q), _f64(k), _f64(v), _scale64(scale)
    Z, H, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    pos, key = np.arange(Nk - Nq, Nk), np.arange(Nk)
    o, lse = np.zeros((Z, H, Nq, D)), np.zeros((Z, H, Nq))
    bo, bl = np.zeros((Z, H, Nq, D)), np.zeros((Z, H, Nq))
    for z in range(Z):
        vis = seen(z)
        for h in range(H):
            s = 0.0 if slopes is None else float(slopes[h])
            kh, vh = k[z, h // (H // Hkv)], v[z, h // (H // Hkv)]
            oo, ll, p, _ = head_fwd(q[z, h], kh, vh, scale, cap, s, vis, pos, key)
            slack = score_slack(q[z, h], kh, scale, cap, s, pos, key)
            o[z, h], lse[z, h] = oo, ll
            bo[z, h] = fwd_bound(oo, p, vh, slack, dtype, Nk)
            bl[z, h] = slack + F32 * (64 + 4 * np.abs(np.where(np.isfinite(ll), ll, 0.0)))
    return o, lse, bo, bl


def scored_bwd(q, k, v, do, scale, cap=0.0, slopes=None, seen=None, dtype=torch.float16):
    """(dq, dk, dv) and their bounds."""
    q, k, v, do, scale = _f64(q), _f64(k), _f64(v), _f64(do), _scale64(scale)
    Z, H, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    G = H // Hkv
    pos, key = np.arange(Nk - Nq, Nk), np.arange(Nk)
    out = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    off = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    u, tiny = HALF_STEP[dtype], TINY[dtype]
    for z in range(Z):
        vis = seen(z)
        for h in range(H):
            g = h // G
            s = 0.0 if slopes is None else float(slopes[h])
            oo, _, p, t = head_fwd(q[z, h], k[z, g], v[z, g], scale, cap, s, vis, pos, key)
            slack = 2 * score_slack(q[z, h], k[z, g], scale, cap, s, pos, key) + F32 * 64
            dp = do[z, h] @ v[z, g].T
            delta = (oo * do[z, h]).sum(1, keepdims=True)
            fac = 1.0 - t * t if cap else 1.0
            ds = p * (dp - delta) * fac
            out[0][z, h] = scale * ds @ k[z, g]
            out[1][z, g] += scale * ds.T @ q[z, h]
            out[2][z, g] += p.T @ do[z, h]
            # dS: its own rounding, the row's delta (from the rounded o), dP's
            # and P's fp32 errors
            d_delta = (fwd_bound(oo, p, v[z, g], slack, dtype, Nk) * np.abs(do[z, h])).sum(1, keepdims=True)
            d_dp = F32 * D * (np.abs(do[z, h]) @ np.abs(v[z, g]).T)
            e_ds = (u + slack + F32 * 64) * np.abs(ds) + p * fac * (d_delta + d_dp) + slack * p * np.abs(dp - delta)
            e_ds = np.where(vis, e_ds + tiny, 0.0)
            e_p = np.where(vis, (u + slack) * p + tiny, 0.0)
            off[0][z, h] = scale * e_ds @ np.abs(k[z, g])
            off[1][z, g] += scale * e_ds.T @ np.abs(q[z, h])
            off[2][z, g] += e_p.T @ np.abs(do[z, h])
    for a, b in zip(out, off):
        b += u * (np.abs(a) + b) + F32 * 64 * np.abs(a) + tiny
    return out, off


def paged_scored_fwd(q, k_cache, v_cache, table, context_lens, q_lens, causal, scale, cap=0.0, slopes=None, window=0,
                     dtype=torch.float16):
    """(o, lse, bound of o, bound of lse) over a paged cache; table entries
    outside the cache read as zeros."""
    q, kc, vc, scale = _f64(q), _f64(k_cache), _f64(v_cache), _scale64(scale)
    table = np.asarray(table)
    B, H, Nq, D = q.shape
    pages, page, Hkv, _ = kc.shape
    o, lse = np.zeros((B, H, Nq, D)), np.full((B, H, Nq), -np.inf)
    bo, bl = np.zeros((B, H, Nq, D)), np.zeros((B, H, Nq))
    for b in range(B):
        n = int(min(max(int(context_lens[b]), 0), table.shape[1] * page))
        m = Nq if q_lens is None else int(min(max(int(q_lens[b]), 0), Nq))
        if m == 0 or n == 0:
            continue
        key = np.arange(n)
        phys = table[b][key // page]
        ok = (phys >= 0) & (phys < pages)
        k = np.where(ok[:, None, None], kc[np.where(ok, phys, 0), key % page], 0.0)
        v = np.where(ok[:, None, None], vc[np.where(ok, phys, 0), key % page], 0.0)
        pos = np.arange(n - m, n)
        seen = np.repeat(pos[:, None] >= 0, n, 1)  # rows before position 0 are no tokens
        if causal:
            seen &= key[None, :] <= pos[:, None]
            if window:
                seen &= key[None, :] > pos[:, None] - window
        for h in range(H):
            g = h // (H // Hkv)
            s = 0.0 if slopes is None else float(slopes[h])
            oo, ll, p, _ = head_fwd(q[b, h, :m], k[:, g], v[:, g], scale, cap, s, seen, pos, key)
            slack = score_slack(q[b, h, :m], k[:, g], scale, cap, s, pos, key)
            o[b, h, :m], lse[b, h, :m] = oo, ll
            bo[b, h, :m] = fwd_bound(oo, p, v[:, g], slack, dtype, n)
            bl[b, h, :m] = slack + F32 * (64 + 4 * np.abs(np.where(np.isfinite(ll), ll, 0.0)))
    return o, lse, bo, bl


def rotary(x, positions, freqs, interleaved=False, inverse=False, mscale=1.0):
    """x [Z, heads, N, D] turned by positions [Z, N]; float64."""
    y = _f64(x).copy()
    f = np.asarray(freqs.cpu() if isinstance(freqs, torch.Tensor) else freqs, np.float64)
    pos = np.asarray(positions.cpu() if isinstance(positions, torch.Tensor) else positions)
    rot = 2 * f.size
    # the angle in extended precision: far positions times 1 / (2 pi) lose
    # digits in 64 bits
    turn = pos.astype(np.longdouble)[:, None, :, None] * (f.astype(np.longdouble) / (2 * np.arccos(np.longdouble(-1))))
    turn = (turn - np.floor(turn)).astype(np.float64)
    c, s = np.cos(2 * np.pi * turn) * mscale, np.sin(2 * np.pi * turn) * mscale * (-1.0 if inverse else 1.0)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    x0, x1 = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = x0 * c - x1 * s, x1 * c + x0 * s
    return y
