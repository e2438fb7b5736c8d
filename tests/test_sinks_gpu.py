"""Attention within a window that also sees the first tokens (fwd_scored,
bwd_scored and fwd_paged_scored with sinks) against the fp64 oracle: lengths
from one token up, windows and sinks around the tile sizes, every head
dimension and type, splits, hidden NaN, short contexts.

Tolerances are the oracle's element-wise bounds: each rounding to 16 bits at
half a step, each fp32 score at its worst case (oracle/scored.py).  The partial
sums of dK and dV are in fp32, so they add none."""

import math

import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300.inputs import make_inputs, make_paged_inputs
from oracle import scored as orc
from test_scored_gpu import within

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


def run_case(Z, H, Hkv, Nq, Nk, D, window, sinks, cap, dtype, seed, train=True, wide=1.0, spoil=None):
    q, k, v, do = make_inputs(Z, H, Nq, D, seed, dtype=dtype, Hkv=Hkv, Nk=Nk)
    q = (q.float() * wide).to(dtype)
    scale = 1.0 / math.sqrt(D)
    how = dict(causal=True, scale=scale, softcap=cap, window=window, sinks=sinks)
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    if spoil:
        spoil(kd, vd)
    o, lse = fa.fwd_scored(qd, kd, vd, **how)
    assert fa.device_status() == 0
    seen = lambda z: orc.visible(Nq, Nk, causal=True, window=window, sinks=sinks)  # noqa: E731
    ro, rl, bo, bl = orc.scored_fwd(q, k, v, scale, cap, None, seen, dtype)
    within(lse, rl, bl, "lse")
    within(o, ro, bo, "o")
    if not train:
        return
    grads = fa.bwd_scored(qd, kd, vd, o, dod, lse, **how)
    assert fa.device_status() == 0
    ref, bound = orc.scored_bwd(q, k, v, do, scale, cap, None, seen, dtype)
    for n, a, r, b in zip(("dq", "dk", "dv"), grads, ref, bound):
        within(a, r, b, n)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_types_and_heads(cap, D, dtype):
    run_case(2, 4, 2, 333, 333, D, 70, 4, cap, dtype, 11, wide=4.0 if cap else 1.0)
    run_case(1, 3, 3, 700, 700, D, 130, 130, cap, dtype, 12, wide=4.0 if cap else 1.0)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Nq,Nk", [(1, 1), (1, 2), (2, 2), (1, 300), (127, 128), (128, 128), (129, 129), (64, 65),
                                   (129, 385), (5, 1021), (640, 640), (1021, 1021), (200, 1500)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (17, 4), (128, 64)])
def test_lengths(window, sinks, Nq, Nk, D):
    run_case(2, 6, 2, Nq, Nk, D, window, sinks, 0.0, torch.float16, 15)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("window", [1, 63, 64, 127, 128, 129, 300])
@pytest.mark.parametrize("sinks", [1, 63, 128, 129, 200, 256])
def test_around_the_tiles(window, sinks, D):
    run_case(1, 2, 1, 700, 700, D, window, sinks, 0.0, torch.float16, 16)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_sinks(D):
    run_case(1, 2, 2, 1100, 1100, D, 40, 700, 0.0, torch.float16, 17)
    run_case(1, 2, 1, 1100, 1100, D, 40, 1059, 15.0, torch.bfloat16, 18)


def test_nothing_hidden_is_plain_causal():
    q, k, v, do = (t.cuda() for t in make_inputs(1, 4, 300, 128, 19, Hkv=2))
    o, lse = fa.fwd_scored(q, k, v, causal=True)
    g = fa.bwd_scored(q, k, v, o, do, lse, causal=True)
    for window, sinks in ((200, 100), (300, 4), (1, 1 << 40), (1 << 40, 1)):
        how = dict(causal=True, window=window, sinks=sinks)
        o2, lse2 = fa.fwd_scored(q, k, v, **how)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(a, b) for a, b in zip(g, fa.bwd_scored(q, k, v, o, do, lse, **how)))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (6, 2), (16, 2), (40, 40)])
def test_grouped_heads_and_many_units(H, Hkv):
    run_case(2, H, Hkv, 600, 600, 128, 100, 5, 0.0, torch.float16, 20)
    run_case(2, H, Hkv, 3, 600, 128, 100, 5, 10.0, torch.float16, 21)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_several_rounds_of_units(D):
    run_case(6, 8, 8, 520, 520, D, 60, 3, 0.0, torch.bfloat16, 22)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_keys_that_nobody_sees_may_hold_anything(D, cap):
    """The queries are the last 40 of 900 positions: keys 9 .. 809 are seen by none."""
    def spoil(k, v):
        for t in (k, v):
            t[:, :, 9:900 - 40 - 50 + 1] = float("nan")
            t[:, :, 300:310] = float("inf")
    Nq, Nk, window, sinks = 40, 900, 50, 9
    q, k, v, do = make_inputs(2, 4, Nq, D, 23, Hkv=2, Nk=Nk)
    scale = 1.0 / math.sqrt(D)
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    spoil(kd, vd)
    how = dict(causal=True, scale=scale, softcap=cap, window=window, sinks=sinks)
    o, lse = fa.fwd_scored(qd, kd, vd, **how)
    seen = lambda z: orc.visible(Nq, Nk, causal=True, window=window, sinks=sinks)  # noqa: E731
    ro, rl, bo, bl = orc.scored_fwd(q, k, v, scale, cap, None, seen)
    within(lse, rl, bl, "lse")
    within(o, ro, bo, "o")
    grads = fa.bwd_scored(qd, kd, vd, o, dod, lse, **how)
    ref, bound = orc.scored_bwd(q, k, v, do, scale, cap, None, seen)
    for n, a, r, b in zip(("dq", "dk", "dv"), grads, ref, bound):
        within(a, r, b, n)
    assert all((g[:, :, 9:811] == 0).all() for g in grads[1:])


def test_gradients_against_differences():
    """dq, dk, dv of sum(o * w), by central differences of the oracle's own forward in 64 bits at the same inputs."""
    Z, H, N, D, window, sinks = 1, 2, 270, 64, 20, 3
    q, k, v, w = make_inputs(Z, H, N, D, 24)
    scale = 1.0 / math.sqrt(D)
    seen = lambda z: orc.visible(N, N, causal=True, window=window, sinks=sinks)  # noqa: E731
    o, lse = fa.fwd_scored(q.cuda(), k.cuda(), v.cuda(), causal=True, window=window, sinks=sinks)
    grads = fa.bwd_scored(q.cuda(), k.cuda(), v.cuda(), o, w.cuda(), lse, causal=True, window=window, sinks=sinks)
    _, bound = orc.scored_bwd(q, k, v, w, scale, seen=seen)
    h = 1e-5
    for name, at in (("q", (0, 1, 200, 5)), ("k", (0, 0, 1, 7)), ("k", (0, 1, 150, 3)), ("v", (0, 1, 2, 9)),
                     ("v", (0, 0, 269, 0)), ("q", (0, 0, 0, 1))):
        totals = []
        for s in (1, -1):
            x = {"q": q.double().clone(), "k": k.double().clone(), "v": v.double().clone()}
            x[name][at] += s * h
            oo, _, _, _ = orc.scored_fwd(x["q"], x["k"], x["v"], scale, seen=seen)
            totals.append(float((oo * w.double().numpy()).sum()))
        i = "qkv".index(name)
        got, want = float(grads[i][at]), (totals[0] - totals[1]) / (2 * h)
        assert abs(got - want) <= bound[i][at] + 1e-6 * (1 + abs(want)), (name, at, got, want)


def test_same_bits_every_time_and_any_workspace():
    q, k, v, do = (t.cuda() for t in make_inputs(2, 8, 1500, 128, 25, Hkv=2))
    how = dict(causal=True, window=100, sinks=6)
    o, lse = fa.fwd_scored(q, k, v, **how)
    g = fa.bwd_scored(q, k, v, o, do, lse, **how)
    need = fa.bwd_workspace_size(2, 8, 1500, 128, True, Hkv=2, window=100, sinks=6)
    for fill in (0, 255):
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        again = fa.bwd_scored(q, k, v, o, do, lse, workspace=ws[:need], **how)
        assert all(torch.equal(a, b) for a, b in zip(g, again))
        assert (ws[need:] == fill).all()
    with pytest.raises(Exception, match="workspace"):
        fa.bwd_scored(q, k, v, o, do, lse, workspace=ws[:need - 256], **how)


# ------------------------------------------------------------------- paged


def run_paged(B, H, Hkv, Nq, lens, D, page, seed, window, sinks, q_lens=None, cap=0.0, dtype=torch.float16, splits=0,
              wide=1.0, ctx_edit=None, table_edit=None):
    q, kc, vc, table, ctx = make_paged_inputs(B, H, Hkv, Nq, lens, D, page, seed, dtype=dtype)
    q = (q.float() * wide).to(dtype)
    if ctx_edit:
        ctx_edit(ctx)
    if table_edit:
        table_edit(table)
    ql = torch.tensor(q_lens, dtype=torch.int32) if q_lens is not None else None
    scale = 1.0 / math.sqrt(D)
    o, lse = fa.fwd_paged_scored(*(t.cuda() for t in (q, kc, vc, table, ctx)),
                                 q_lens=ql.cuda() if ql is not None else None, scale=scale, softcap=cap, window=window,
                                 sinks=sinks, splits=splits)
    assert fa.device_status() == 0
    ro, rl, bo, bl = orc.paged_scored_fwd(q, kc, vc, table.numpy(), ctx.numpy(), q_lens, True, scale, cap, None, window,
                                          dtype, sinks)
    within(lse, rl, bl, "lse")
    within(o, ro, bo, "o")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 64), (256, 16), (256, 64)])
@pytest.mark.parametrize("splits", [0, 1, 3, 4, 9])
def test_paged_tokens(D, page, splits, dtype):
    run_paged(4, 8, 2, 1, [1, 130, 1517, 400], D, page, 31, 100, 4, dtype=dtype, splits=splits)
    run_paged(2, 2, 2, 1, [900, 5], D, page, 31, 30, 150, cap=20.0, dtype=dtype, splits=splits, wide=3.0)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("Nq,q_lens", [(5, [5, 1, 3]), (40, [40, 0, 17]), (200, [129, 200, 1]), (130, None)])
def test_paged_chunks(Nq, q_lens, splits, D):
    run_paged(3, 6, 2, Nq, [800, 1450, 211], D, 32, 32, 90, 20, q_lens=q_lens, splits=splits)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("splits", [1, 3])
def test_paged_chunks_mostly_without_rows(D, cap, splits):
    """Several rounds of units, of which most have no new token: single ones, none, whole chunks."""
    q_lens = [300, 1, 0, 1, 129, 0, 1, 128, 0, 1] * 2
    run_paged(20, 8, 4, 300, [max(n, 1) + 37 * b for b, n in enumerate(q_lens)], D, 32, 47, 90, 20, q_lens=q_lens,
              cap=cap, splits=splits)


@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("window", [1, 16, 100, 129, 100000])
@pytest.mark.parametrize("sinks", [1, 16, 129, 300])
def test_paged_window_and_sinks(window, sinks, splits):
    for Nq in (1, 70):
        run_paged(2, 4, 2, Nq, [777, 300], 128, 64, 33, window, sinks, q_lens=[Nq, max(1, Nq // 2)], splits=splits)


@pytest.mark.parametrize("splits", [1, 3, 4])
@pytest.mark.parametrize("Nq", [1, 4, 140])
def test_paged_short_and_empty_contexts(Nq, splits):
    def edit(ctx):
        ctx[0], ctx[1], ctx[2] = 0, -5, min(2, Nq)
    run_paged(4, 4, 2, Nq, [200, 200, 200, 200], 128, 32, 35, 20, 3, ctx_edit=edit, splits=splits)
    run_paged(4, 4, 2, Nq, [200, 200, 200, 200], 128, 32, 35, 20, 3, q_lens=[0, 0, 0, 0], splits=splits)


def test_paged_bad_table_entries_read_as_zeros():
    def edit(table):
        table[0, 0], table[0, 5], table[1, 3] = -1, 1 << 30, -7
    run_paged(2, 4, 2, 3, [300, 300], 64, 16, 36, 250, 20, table_edit=edit)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("splits", [1, 4])
def test_paged_keys_that_nobody_sees_may_hold_anything(D, splits):
    """Rows past the contexts, and pages and parts of pages between the sinks and the windows, hold NaN."""
    page, lens, window, sinks = 16, [500, 411], 60, 21
    q, kc, vc, table, ctx = make_paged_inputs(2, 4, 2, 1, lens, D, page, 37)
    clean = [t.clone() for t in (kc, vc)]
    for t in (kc, vc):
        for b, n in enumerate(lens):
            for p in list(range(sinks, n - window)) + list(range(n, (n + page - 1) // page * page)):
                t[table[b, p // page], p % page] = float("nan")
    o, lse = fa.fwd_paged_scored(*(t.cuda() for t in (q, kc, vc, table, ctx)), window=window, sinks=sinks, splits=splits)
    ro, rl, bo, bl = orc.paged_scored_fwd(q, *clean, table.numpy(), ctx.numpy(), None, True, 1.0 / math.sqrt(D),
                                          window=window, sinks=sinks)
    within(lse, rl, bl, "lse")
    within(o, ro, bo, "o")


def test_refusals():
    q, k, v, _ = (t.cuda() for t in make_inputs(1, 2, 64, 64, 38))
    sl = torch.ones(2, device="cuda")
    kr = fa.key_ranges(64, 64, prefix_lens=torch.tensor([3], dtype=torch.int32, device="cuda"))
    for bad in (dict(causal=False, window=0), dict(causal=True, window=0), dict(causal=True, window=4, slopes=sl),
                dict(causal=True, window=4, key_ranges=kr), dict(causal=True, window=4, sinks=-1)):
        with pytest.raises(ValueError, match="sinks"):
            fa.fwd_scored(q, k, v, **{"sinks": 2, **bad})


# --------------------------------------------------------- several far units


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks,cap", [(50, 3, 0.0), (130, 140, 0.0), (60, 5, 15.0)])
def test_several_far_units(D, window, sinks, cap):
    """Queries enough for two to five far units of a key tile with sinks, grouped heads."""
    run_case(1, 2, 1, 2700, 2700, D, window, sinks, cap, torch.float16, 40)
    run_case(1, 1, 1, 1700, 2900, D, window, sinks, cap, torch.bfloat16, 41)


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16), (256, torch.bfloat16)])
def test_long(D, dtype):
    """16384 tokens, against the definition in 64 bits on the GPU, a block of queries at a time.

    Relative error of the whole result: o, dk and dv are rounded once, after P or dS were (half a step of each value at
    random signs, so at most sqrt(2) of one rounding in the 2-norm, doubled for the accumulators and the scores); dq may
    be off by another rounding's worth of Delta in tiles without the sinks."""
    Z, H, Hkv, N, window, sinks = 1, 2, 1, 16384, 1000, 37
    q, k, v, do = (t.cuda() for t in make_inputs(Z, H, N, D, 42, dtype=dtype, Hkv=Hkv))
    k[:, :, :sinks] += 0.5
    q += 0.5
    scale = 1.0 / math.sqrt(D)
    how = dict(causal=True, window=window, sinks=sinks)
    o, lse = fa.fwd_scored(q, k, v, **how)
    grads = fa.bwd_scored(q, k, v, o, do, lse, **how)
    assert fa.device_status() == 0
    want = [torch.zeros_like(t, dtype=torch.float64) for t in (q, q, k, v)]  # o, dq, dk, dv
    far = 0.0
    for h in range(H):
        kh, vh = k[0, 0].double(), v[0, 0].double()
        key = torch.arange(N, device="cuda")[None, :]
        for i in range(0, N, 2048):
            pos = torch.arange(i, i + 2048, device="cuda")[:, None]
            seen = (key <= pos) & ((key > pos - window) | (key < sinks))
            qh, dh = q[0, h, i:i + 2048].double(), do[0, h, i:i + 2048].double()
            x = (qh @ kh.T * scale).masked_fill(~seen, -math.inf)
            rl = torch.logsumexp(x, -1)
            p = torch.exp(x - rl[:, None])
            oo = p @ vh
            ds = p * (dh @ vh.T - (oo * dh).sum(-1, keepdim=True)) * scale
            want[0][0, h, i:i + 2048] = oo
            want[1][0, h, i:i + 2048] = ds @ kh
            want[2][0, 0] += ds.T @ qh
            want[3][0, 0] += p.T @ dh
            far = max(far, float((lse[0, h, i:i + 2048].double() - rl).abs().max()))
    assert far < 1e-5 * (1 + float(lse.abs().max()))
    step = orc.HALF_STEP[dtype]
    for name, a, b in zip(("o", "dq", "dk", "dv"), (o,) + tuple(grads), want):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel < 2 * math.sqrt(2) * step * (1.5 if name == "dq" else 1.0), (name, rel)


def test_two_graphs_share_a_workspace():
    q, k, v, do = (t.cuda() for t in make_inputs(1, 4, 1500, 128, 43, Hkv=2))
    ways = [dict(causal=True, window=70, sinks=4), dict(causal=True, window=300, sinks=150)]
    need = max(fa.bwd_workspace_size(1, 4, 1500, 128, True, Hkv=2, window=w["window"], sinks=w["sinks"]) for w in ways)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    eager = []
    for w in ways:
        o, lse = fa.fwd_scored(q, k, v, **w)
        eager.append((o, lse) + tuple(fa.bwd_scored(q, k, v, o, do, lse, **w)))
    graphs, res = [], []
    for w in ways:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = fa.fwd_scored(q, k, v, **w)
            res.append((o, lse) + tuple(fa.bwd_scored(q, k, v, o, do, lse, workspace=ws, **w)))
        graphs.append(g)
    for order in ((0, 1), (1, 0, 0, 1)):
        for r in res:
            for t in r:
                t.fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for r, e in zip(res, eager):
            assert all(torch.equal(a, b) for a, b in zip(r, e))


def test_two_streams_at_once():
    calls = []
    for seed, (window, sinks) in enumerate(((70, 4), (300, 150), (20, 1))):
        q, k, v, do = (t.cuda() for t in make_inputs(2, 4, 1100, 64, 44 + seed, Hkv=2))
        calls.append((q, k, v, do, dict(causal=True, window=window, sinks=sinks)))

    def run(c, stream=None):
        q, k, v, do, how = c
        o, lse = fa.fwd_scored(q, k, v, stream=stream, **how)
        return (o, lse) + tuple(fa.bwd_scored(q, k, v, o, do, lse, stream=stream, **how))
    want = [run(c) for c in calls]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in calls]
    got = [run(c, s) for _ in range(5) for c, s in zip(calls, sides)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % len(calls)]))
    assert fa.device_status() == 0


def test_paged_long_cache():
    """Pages whose byte offsets pass 32 bits, and a context of 100000 tokens, of which the window and the sinks are read."""
    page, Hkv, D, ctx, window, sinks = 64, 8, 128, 100000, 500, 70
    pages = (1 << 32) // (page * Hkv * D * 2) + 9
    kc, vc = (torch.full((pages, page, Hkv, D), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(45)
    table = torch.randint(0, pages, (1, -(-ctx // page)), generator=g, dtype=torch.int32)
    table[0, -12:] = torch.arange(pages - 12, pages, dtype=torch.int32)
    table[0, :2] = torch.tensor([pages - 13, 0], dtype=torch.int32)
    seen = list(range(sinks)) + list(range(ctx - window, ctx))
    k, v = torch.randn((2, len(seen), Hkv, D), generator=g).half()
    for i, p in enumerate(seen):
        at = (int(table[0, p // page]), p % page)
        kc[at], vc[at] = k[i].cuda(), v[i].cuda()
    q = torch.randn((1, 16, 1, D), generator=g).half()
    scale = 1.0 / math.sqrt(D)
    ro, rl, bo, bl = orc.scored_fwd(q, k.transpose(0, 1)[None], v.transpose(0, 1)[None], scale,
                                    seen=lambda z: orc.visible(1, len(seen)))
    for splits in (0, 1, 8):
        o, lse = fa.fwd_paged_scored(q.cuda(), kc, vc, table.cuda(), i32([ctx]), window=window, sinks=sinks, splits=splits)
        within(lse, rl, bl, "lse")
        within(o, ro, bo, "o")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
