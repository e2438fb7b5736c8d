"""Scored attention (fa_fwd_scored, fa_bwd_scored, fa_key_ranges) against the
fp64 oracle: caps, distance bias, documents, prefix, window, empty rows, at
lengths from one token up, for every head dimension and type.

Tolerances are the oracle's element-wise bounds: each rounding to 16 bits at
half a step, each fp32 score at its worst case (oracle/scored.py)."""

import math

import numpy as np
import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300.inputs import make_inputs
from oracle import scored as orc

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


def within(got, want, bound, what):
    got = got.detach().double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine), f"{what}: finite elsewhere"
    assert np.array_equal(got[~fine], want[~fine]), f"{what}: infinities differ"
    d = np.zeros(want.shape)
    d[fine] = np.abs(got[fine] - want[fine])
    at = np.unravel_index(np.argmax(d - bound), d.shape)
    assert (d <= bound).all(), f"{what}: off by {d[at]:.3e} (bound {bound[at]:.3e}) at {at}"


def doc_ids(Z, N, seed, mean):
    g = torch.Generator().manual_seed(seed)
    return torch.cumsum((torch.rand((Z, N), generator=g) < 1.0 / mean).int(), 1).to(torch.int32)


def rules(mask, Z, Nq, Nk, seed):
    """(arguments of the call, seen(z), key-range source) of a named mask."""
    g = torch.Generator().manual_seed(seed + 7)
    if mask == "none":
        return dict(causal=False), lambda z: orc.visible(Nq, Nk), None
    if mask == "causal":
        return dict(causal=True), lambda z: orc.visible(Nq, Nk, causal=True), None
    if mask == "window":
        w = max(1, Nk // 3)
        return dict(causal=True, window=w), lambda z: orc.visible(Nq, Nk, causal=True, window=w), None
    if mask in ("docs", "docs_both"):
        ids = doc_ids(Z, Nk, seed, max(1, Nk // 5))
        c = mask == "docs"
        return (dict(causal=c), lambda z: orc.visible(Nq, Nk, causal=c, docs=ids[z].numpy()), dict(doc_ids=ids))
    if mask == "prefix":
        p = torch.randint(0, Nk + 1, (Z,), generator=g).int()
        return dict(causal=False), lambda z: orc.visible(Nq, Nk, prefix=p[z]), dict(prefix_lens=p)
    assert mask == "ranges"  # arbitrary, about a fifth of the rows empty
    r = torch.randint(-2, Nk + 3, (Z, Nq, 2), generator=g).int().sort(-1).values
    r[torch.rand((Z, Nq), generator=g) < 0.2] = torch.tensor([3, 3], dtype=torch.int32)
    return dict(causal=False), lambda z: orc.visible(Nq, Nk, ranges=r[z].numpy()), dict(ranges=r.contiguous())


def slopes_of(H):
    return torch.exp2(-8.0 * torch.arange(1, H + 1) / H).float()


def run_case(Z, H, Hkv, Nq, Nk, D, mask, cap, bias, dtype, seed, train=True, wide=1.0):
    q, k, v, do = make_inputs(Z, H, Nq, D, seed, dtype=dtype, Hkv=Hkv, Nk=Nk)
    q = (q.float() * wide).to(dtype)
    how, seen, src = rules(mask, Z, Nq, Nk, seed)
    scale = 1.0 / math.sqrt(D)
    sl = slopes_of(H) if bias else None
    kr = fa.key_ranges(Nq, Nk, **{n: t.cuda() for n, t in src.items()}) if src else None
    args = dict(scale=scale, softcap=cap, slopes=sl.cuda() if bias else None, key_ranges=kr, **how)
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    o, lse = fa.fwd_scored(qd, kd, vd, **args)
    assert fa.device_status() == 0
    ro, rl, bo, bl = orc.scored_fwd(q, k, v, scale, cap, sl, seen, dtype)
    within(lse, rl, bl, "lse")
    within(o, ro, bo, "o")
    if not train:
        return
    grads = fa.bwd_scored(qd, kd, vd, o, dod, lse, **args)
    assert fa.device_status() == 0
    ref, bound = orc.scored_bwd(q, k, v, do, scale, cap, sl, seen, dtype)
    for n, a, r, b in zip(("dq", "dk", "dv"), grads, ref, bound):
        within(a, r, b, n)


MASKS = ["none", "causal", "window", "docs", "docs_both", "prefix", "ranges"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("mask", MASKS)
def test_masks(mask, D, dtype):
    run_case(2, 4, 2, 333, 333, D, mask, 0.0, False, dtype, 11)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("mask", MASKS)
def test_cap_and_bias(mask, D):
    run_case(2, 4, 2, 300, 300, D, mask, 20.0, True, torch.float16, 12, wide=4.0)
    run_case(1, 4, 4, 257, 257, D, mask, 30.0, False, torch.bfloat16, 13, wide=4.0)
    run_case(1, 3, 1, 200, 200, D, mask, 0.0, True, torch.bfloat16, 14)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Nq,Nk", [(1, 1), (1, 2), (2, 2), (1, 300), (127, 128), (128, 128), (129, 129), (64, 65),
                                   (129, 385), (5, 1021), (640, 640)])
@pytest.mark.parametrize("mask", ["causal", "prefix", "ranges"])
def test_lengths(mask, Nq, Nk, D):
    run_case(2, 6, 2, Nq, Nk, D, mask, 25.0, True, torch.float16, 15, wide=2.0)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (6, 2), (16, 2), (5, 5)])
@pytest.mark.parametrize("mask", ["window", "docs", "none"])
def test_grouped_heads(mask, H, Hkv):
    run_case(2, H, Hkv, 150, 150, 128, mask, 0.0, True, torch.float16, 16)
    run_case(2, H, Hkv, 3, 150, 128, "causal" if mask == "docs" else mask, 10.0, True, torch.float16, 17)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_key_ranges_allow_more_queries_than_keys(D):
    run_case(1, 2, 1, 400, 70, D, "ranges", 0.0, False, torch.float16, 18)


def test_steep_bias_and_large_cap():
    Z, H, N, D = 1, 4, 300, 64
    q, k, v, do = make_inputs(Z, H, N, D, 19)
    sl = torch.tensor([0.0, 1.0, 5.0, -0.01])
    seen = lambda z: orc.visible(N, N, causal=True)  # noqa: E731
    for cap in (0.0, 1000.0, 0.5):
        args = dict(causal=True, scale=0.125, softcap=cap, slopes=sl.cuda())
        o, lse = fa.fwd_scored(q.cuda(), k.cuda(), v.cuda(), **args)
        ro, rl, bo, bl = orc.scored_fwd(q, k, v, 0.125, cap, sl, seen)
        within(lse, rl, bl, "lse")
        within(o, ro, bo, "o")
        g = fa.bwd_scored(q.cuda(), k.cuda(), v.cuda(), o, do.cuda(), lse, **args)
        ref, bound = orc.scored_bwd(q, k, v, do, 0.125, cap, sl, seen)
        for n, a, r, b in zip(("dq", "dk", "dv"), g, ref, bound):
            within(a, r, b, n)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [4096.0, 1e-3, 1e-20])
def test_largest_and_small_caps(cap, D):
    run_case(1, 4, 2, 200, 200, D, "causal", cap, False, torch.float16, 20, wide=4.0)
    run_case(1, 4, 2, 200, 200, D, "prefix", cap, True, torch.bfloat16, 22)


# More work units than a GPU has SMs: several rounds of them with a ragged last
# one, a list that is nearly full (290 tiles x 50 heads), one unit count past
# it (300 x 50), and more tiles than a block has threads (130 x 3).
@pytest.mark.parametrize("mask", ["causal", "docs", "prefix"])
@pytest.mark.parametrize("Z,H,Hkv,N,D", [(3, 32, 16, 700, 64), (2, 40, 8, 650, 128), (290, 50, 50, 16, 64),
                                         (300, 50, 50, 16, 64), (130, 2, 1, 300, 128), (130, 2, 2, 300, 64)])
def test_many_units(Z, H, Hkv, N, D, mask):
    run_case(Z, H, Hkv, N, N, D, mask, 0.0, True, torch.float16, 21)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
def test_hidden_values_may_be_anything(D, junk):
    """Padded batches: keys no query sees and queries that see no key hold NaN
    or infinities in every tensor; nothing of them shows."""
    Z, H, N, live = 2, 2, 300, (170, 257)
    q, k, v, do = make_inputs(Z, H, N, D, 20)
    r = torch.zeros((Z, N, 2), dtype=torch.int32)
    for z in range(Z):
        r[z, : live[z], 1] = live[z]
    bad = [t.clone() for t in (q, k, v, do)]
    for z in range(Z):
        for t in bad:
            t[z, :, live[z]:] = junk
        for t in (q, k, v, do):
            t[z, :, live[z]:] = 0
    for causal in (False, True):
        args = dict(causal=causal, key_ranges=fa.key_ranges(N, N, ranges=r.cuda()), softcap=10.0)
        out = []
        for t in ((q, k, v, do), bad):
            qd, kd, vd, dod = (x.cuda() for x in t)
            o, lse = fa.fwd_scored(qd, kd, vd, **args)
            out.append((o, lse) + tuple(fa.bwd_scored(qd, kd, vd, o, dod, lse, **args)))
        for a, b in zip(*out):
            assert torch.equal(a, b)
        for z in range(Z):
            assert not out[0][0][z, :, live[z]:].any() and torch.isinf(out[0][1][z, :, live[z]:]).all()
            for g in out[0][2:]:
                assert not g[z, :, live[z]:].any()


def test_visible_nan_shows():
    q, k, v, _ = (t.cuda() for t in make_inputs(1, 1, 130, 64, 21))
    k[0, 0, 5] = float("nan")
    o, lse = fa.fwd_scored(q, k, v, causal=True, softcap=5.0)
    assert torch.isfinite(o[0, 0, :5]).all() and torch.isnan(o[0, 0, 5:]).all()


def test_key_ranges_rows():
    Z, N = 3, 1500
    ids = doc_ids(Z, N, 5, 300)
    ids[1] = 7                                     # one document
    ids[2] = torch.arange(N, dtype=torch.int32) % 2  # documents of one token
    for Nq in (1, 128, 700, N):
        rows = fa.key_ranges(Nq, N, doc_ids=ids.cuda()).rows.cpu().numpy()
        for z in range(Z):
            seen = orc.visible(Nq, N, docs=ids[z].numpy())
            assert np.array_equal(rows[z, :, 0], seen.argmax(1))
            assert np.array_equal(rows[z, :, 1] - rows[z, :, 0], seen.sum(1))
    p = torch.tensor([0, 700, 9999], dtype=torch.int32)
    rows = fa.key_ranges(800, N, prefix_lens=p.cuda()).rows.cpu()
    pos = torch.arange(N - 800, N)
    for z in range(Z):
        assert (rows[z, :, 0] == 0).all() and torch.equal(rows[z, :, 1].long(), torch.clamp(pos + 1, min=min(int(p[z]), N)))
    r = torch.randint(-50, N + 50, (Z, 90, 2), generator=torch.Generator().manual_seed(1)).int()
    rows = fa.key_ranges(90, N, ranges=r.cuda()).rows.cpu()
    lo, hi = r[..., 0].clamp(min=0), r[..., 1].clamp(max=N)
    some = lo < hi
    assert torch.equal(rows[..., 0], torch.where(some, lo, 0)) and torch.equal(rows[..., 1], torch.where(some, hi, 0))


def test_repeat_is_bitwise_and_graph_replays():
    q, k, v, do = (t.cuda() for t in make_inputs(2, 4, 700, 128, 23))
    ids = doc_ids(2, 700, 3, 90).cuda()
    sl = slopes_of(4).cuda()

    def step():
        kr = fa.key_ranges(700, 700, doc_ids=ids)
        args = dict(causal=True, softcap=30.0, slopes=sl, key_ranges=kr)
        o, lse = fa.fwd_scored(q, k, v, **args)
        return (o, lse) + tuple(fa.bwd_scored(q, k, v, o, do, lse, **args))

    want = [t.clone() for t in step()]
    for a, b in zip(step(), want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in (q, k, v, do):
        t.copy_(torch.roll(t, 1, 0))
    ids.copy_(torch.roll(ids, 1, 0))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, torch.roll(b, 1, 0))


def test_side_stream_and_out():
    q, k, v, do = (t.cuda() for t in make_inputs(1, 2, 200, 64, 24))
    want = fa.fwd_scored(q, k, v, causal=True, softcap=4.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = (torch.empty_like(q), torch.empty((1, 2, 200), device="cuda"))
    o, lse = fa.fwd_scored(q, k, v, causal=True, softcap=4.0, out=out, stream=s)
    g = fa.bwd_scored(q, k, v, o, do, lse, causal=True, softcap=4.0, stream=s)
    s.synchronize()
    assert o is out[0] and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for a, b in zip(g, fa.bwd_scored(q, k, v, want[0], do, want[1], causal=True, softcap=4.0)):
        assert torch.equal(a, b)


def test_gradients_against_differences():
    """Central differences of sum(o * w) in the exact forward, at the kernel's
    own gradient, along random directions."""
    Z, H, N, D, cap = 1, 2, 40, 64, 6.0
    q, k, v, w = make_inputs(Z, H, N, D, 25)
    q = (q.float() * 3).half()
    sl = torch.tensor([0.05, 0.2])
    args = dict(causal=True, scale=0.125, softcap=cap, slopes=sl.cuda())
    qd, kd, vd, wd = (t.cuda() for t in (q, k, v, w))
    o, lse = fa.fwd_scored(qd, kd, vd, **args)
    grads = [t.double().cpu().numpy() for t in fa.bwd_scored(qd, kd, vd, o, wd, lse, **args)]
    seen = lambda z: orc.visible(N, N, causal=True)  # noqa: E731
    _, bounds = orc.scored_bwd(q, k, v, w, 0.125, cap, sl, seen)
    rng = np.random.default_rng(0)
    x = [t.double().numpy() for t in (q, k, v)]

    def loss(a):
        return float((orc.scored_fwd(*a, 0.125, cap, sl, seen)[0] * w.double().numpy()).sum())

    for i in range(3):
        for _ in range(3):
            d = rng.standard_normal(x[i].shape)
            e = 1e-4
            up, down = list(x), list(x)
            up[i], down[i] = x[i] + e * d, x[i] - e * d
            slope = (loss(up) - loss(down)) / (2 * e)
            # the bound of each element, along d, and the difference's own error (third derivative, cancellation)
            far = float((bounds[i] * np.abs(d)).sum()) + 1e-4 * abs(slope) + 1e-6
            assert abs(float((grads[i] * d).sum()) - slope) <= far


def test_two_backward_graphs_share_a_workspace_and_streams_run_at_once():
    from attention_sm_flashattention_gb300 import api
    args = dict(causal=True, softcap=9.0)
    cases = []
    for seed in (31, 32):
        q, k, v, do = (t.cuda() for t in make_inputs(2, 8, 600, 128, seed))
        o, lse = fa.fwd_scored(q, k, v, **args)
        cases.append((q, k, v, o, do, lse))
    want = [fa.bwd_scored(*c, **args) for c in cases]
    ws = torch.empty(api.bwd_workspace_size(2, 8, 600, 128, True), dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(fa.bwd_scored(*c, **args, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):  # each call with a workspace of its own
        got = [fa.bwd_scored(*c, **args, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
