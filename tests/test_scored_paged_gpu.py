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
