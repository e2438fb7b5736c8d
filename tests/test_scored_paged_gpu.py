"""Scored attention over a paged cache (fa_fwd_paged_scored) against the fp64
oracle: single tokens and ragged chunks, caps, bias, window, splits, short and
empty contexts, bad pages."""

import math

import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300 import _native
from attention_sm_flashattention_gb300.inputs import make_paged_inputs
from oracle import scored as orc
from test_scored_gpu import slopes_of, within

pytestmark = pytest.mark.gpu


def run_case(B, H, Hkv, Nq, lens, D, page, seed, q_lens=None, cap=0.0, bias=False, window=0, causal=True,
             dtype=torch.float16, splits=0, wide=1.0, table_edit=None, ctx_edit=None):
    q, kc, vc, table, ctx = make_paged_inputs(B, H, Hkv, Nq, lens, D, page, seed, dtype=dtype)
    q = (q.float() * wide).to(dtype)
    if table_edit:
        table_edit(table)
    if ctx_edit:
        ctx_edit(ctx)
    ql = torch.tensor(q_lens, dtype=torch.int32) if q_lens is not None else None
    sl = slopes_of(H) if bias else None
    scale = 1.0 / math.sqrt(D)
    o, lse = fa.fwd_paged_scored(*(t.cuda() for t in (q, kc, vc, table, ctx)),
                                 q_lens=ql.cuda() if ql is not None else None, causal=causal, scale=scale, softcap=cap,
                                 slopes=sl.cuda() if bias else None, window=window, splits=splits)
    assert fa.device_status() == 0
    ro, rl, bo, bl = orc.paged_scored_fwd(q, kc, vc, table.numpy(), ctx.numpy(), q_lens, causal, scale, cap, sl,
                                          window, dtype)
    within(lse, rl, bl, "lse")
    within(o, ro, bo, "o")
    return o, lse


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 64), (256, 16), (256, 64)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_tokens(D, page, splits, dtype):
    run_case(3, 8, 2, 1, [1, 130, 517], D, page, 31, cap=20.0, bias=True, dtype=dtype, splits=splits, wide=3.0)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("Nq,q_lens", [(5, [5, 1, 3]), (40, [40, 0, 17]), (200, [129, 200, 1]), (130, None)])
def test_chunks(Nq, q_lens, splits, D):
    run_case(3, 6, 2, Nq, [300, 450, 211], D, 32, 32, q_lens=q_lens, cap=15.0, bias=True, splits=splits, wide=2.0)


@pytest.mark.parametrize("splits", [1, 2, 7])
@pytest.mark.parametrize("window", [1, 16, 100, 129, 100000])
@pytest.mark.parametrize("Nq", [1, 70, 150])
def test_window(Nq, window, splits):
    run_case(2, 4, 2, Nq, [777, 300], 128, 64, 33, q_lens=[Nq, max(1, Nq // 2)], window=window, splits=splits)


@pytest.mark.parametrize("splits", [1, 5])
def test_not_causal(splits):
    run_case(2, 4, 1, 9, [400, 33], 64, 16, 34, q_lens=[9, 4], causal=False, bias=True, splits=splits)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("Nq", [1, 4, 140])
def test_contexts_shorter_than_chunk_and_empty(Nq, splits):
    def edit(ctx):
        ctx[0], ctx[1], ctx[2] = 0, -5, min(2, Nq)
    run_case(4, 4, 2, Nq, [200, 200, 200, 200], 128, 32, 35, ctx_edit=edit, bias=True, splits=splits)
    run_case(4, 4, 2, Nq, [200, 200, 200, 200], 128, 32, 35, q_lens=[0, 0, 0, 0], splits=splits)

    def past(ctx):
        ctx[:] = 10 ** 6  # clamped to the table
    run_case(2, 4, 2, Nq, [256, 256], 128, 32, 36, ctx_edit=past, splits=splits)


def test_q_lens_out_of_range_are_clamped():
    a = run_case(2, 2, 1, 6, [100, 100], 64, 16, 37, q_lens=[-3, 99])
    assert not a[0][0].any()


def test_bad_pages_read_as_zeros():
    def edit(table):
        table[0, 1], table[1, 0], table[1, 2] = -7, 10 ** 6, 2 ** 31 - 1
    run_case(2, 4, 2, 3, [90, 64], 128, 16, 38, table_edit=edit, cap=5.0)


@pytest.mark.parametrize("D", [64, 256])
def test_stale_rows_may_be_anything(D):
    q, kc, vc, table, ctx = make_paged_inputs(2, 4, 2, 3, [37, 90], D, 16, 39)
    args = dict(q_lens=torch.tensor([2, 3], dtype=torch.int32).cuda(), window=50, softcap=9.0)
    out = []
    for junk in (0.0, float("nan"), float("inf")):
        k2, v2 = kc.clone(), vc.clone()
        used = torch.zeros(kc.shape[:2], dtype=torch.bool)
        for b in range(2):
            for p in range(int(ctx[b])):
                if p > int(ctx[b]) - int(args["q_lens"][b]) - 50:  # visible to the first new token
                    used[table[b, p // 16], p % 16] = True
        k2[~used], v2[~used] = junk, junk
        q2 = q.clone()
        q2[0, :, 2:] = junk
        out.append(fa.fwd_paged_scored(*(t.cuda() for t in (q2, k2, v2, table, ctx)), **args))
    for a in out[1:]:
        assert torch.equal(a[0], out[0][0]) and torch.equal(a[1], out[0][1])


def test_split_into_many_and_workspace():
    q, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(2, 8, 2, 2, [2000, 700], 128, 64, 41))
    one = fa.fwd_paged_scored(q, kc, vc, table, ctx, window=300, splits=1)
    need = _native.lib().fa_fwd_paged_split_workspace_size(2, 8, 2, 128, 256)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    many = fa.fwd_paged_scored(q, kc, vc, table, ctx, window=300, splits=256, workspace=ws)
    # both within one rounding of P and of o of the exact result
    assert float((one[0] - many[0]).abs().max()) <= 4 * 2.0 ** -11 * float(vc.abs().max())
    assert float((one[1] - many[1]).abs().max()) <= 1e-5
    with pytest.raises(_native.FaError):
        fa.fwd_paged_scored(q, kc, vc, table, ctx, splits=256, workspace=ws[: need - 256])


# More units than SMs.  1, 4 and 30 rows share a K/V head (at most 32 take the
# replicated form from four slices up), 40 do not fit it; 5 and 9 slices are
# not whole units of four.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [0, 4, 5, 9])
@pytest.mark.parametrize("H,Hkv,Nq", [(8, 8, 1), (32, 8, 1), (12, 2, 5), (16, 2, 5)])
def test_many_units(H, Hkv, Nq, splits, D):
    lens = [int(x) for x in torch.randint(Nq, 1500, (24,), generator=torch.Generator().manual_seed(7))]
    run_case(24, H, Hkv, Nq, lens, D, 16, 42, cap=20.0, splits=splits, wide=3.0)
    run_case(24, H, Hkv, Nq, lens, D, 64, 43, bias=True, window=400, splits=splits, dtype=torch.bfloat16)


def test_two_graphs_share_a_workspace():
    a = [t.cuda() for t in make_paged_inputs(3, 8, 2, 1, [900, 30, 411], 128, 64, 44)]
    b = [t.cuda() for t in make_paged_inputs(3, 8, 2, 1, [77, 1200, 600], 128, 64, 45)]
    ws = torch.empty(_native.lib().fa_fwd_paged_split_workspace_size(3, 8, 1, 128, 8), dtype=torch.uint8, device="cuda")
    want = [fa.fwd_paged_scored(*x, softcap=9.0, splits=8) for x in (a, b)]
    graphs, got = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(fa.fwd_paged_scored(*x, softcap=9.0, splits=8, workspace=ws))
        graphs.append(g)
    for _ in range(3):  # in turn on one stream: each graph writes its slices before it reads them
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_calls_on_two_streams_at_once():
    a = [t.cuda() for t in make_paged_inputs(8, 8, 2, 1, [2000] * 8, 128, 64, 46)]
    b = [t.cuda() for t in make_paged_inputs(8, 8, 2, 60, [1500] * 8, 128, 64, 47)]
    want = [fa.fwd_paged_scored(*x, softcap=9.0) for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [fa.fwd_paged_scored(*x, softcap=9.0, stream=s) for x, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("splits", [1, 4])
def test_pages_past_32_bit_offsets(splits):
    """The same pages at the front of a cache and behind 2^31 of its values."""
    q, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(2, 8, 2, 3, [300, 129], 128, 64, 48))
    n, (page, Hkv, D) = kc.shape[0], kc.shape[1:]
    far = 2 ** 31 // (page * Hkv * D) + 5
    big = [torch.empty((far + n, page, Hkv, D), dtype=kc.dtype, device="cuda") for _ in range(2)]
    for t, s in zip(big, (kc, vc)):
        t[far:] = s
    want = fa.fwd_paged_scored(q, kc, vc, table, ctx, softcap=9.0, splits=splits)
    got = fa.fwd_paged_scored(q, *big, torch.where(table < 0, table, table + far), ctx, softcap=9.0, splits=splits)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # and rows written there
    pos = torch.arange(3, device="cuda").repeat(2, 1)
    freqs, _ = fa.rotary_freqs(D)
    slots = torch.arange(6, device="cuda").reshape(2, 3)
    k_new, v_new = q[:, :Hkv], q[:, Hkv:2 * Hkv]
    near = fa.rotary_and_cache(q, k_new, v_new, pos, freqs, slots, kc, vc)
    assert torch.equal(fa.rotary_and_cache(q, k_new, v_new, pos, freqs, slots + far * page, *big), near)
    assert torch.equal(big[0][far:], kc) and torch.equal(big[1][far:], vc)
