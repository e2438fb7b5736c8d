"""Scored attention at its edges: values that are not finite, rows that see nothing beside them, key ranges with
gaps, saturated caps, positions before the context, arguments past 32 bits."""

import math

import numpy as np
import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300 import _native
from attention_sm_flashattention_gb300.inputs import make_inputs, make_paged_inputs
from oracle import scored as orc
from test_scored_gpu import slopes_of
from test_scored_paged_gpu import run_case as paged_case

pytestmark = pytest.mark.gpu
NAN = float("nan")
FORMS = [(c, b) for c in (0.0, 5.0) for b in (False, True)]


def is_nan_exactly(t, rows):
    """NaN in all of the truth-valued rows, finite in the others."""
    bad = torch.isnan(t).reshape(t.shape[:3] + (-1,))
    return bool((bad.all(-1) == rows).all() and (bad.any(-1) == rows).all() and torch.isfinite(t[~rows]).all())


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_nan_stay_nan(D, cap, bias):
    Z, H, N = 2, 2, 200
    q, k, v, _ = (t.cuda() for t in make_inputs(Z, H, N, D, 61))
    args = dict(causal=True, softcap=cap, slopes=slopes_of(H).cuda() if bias else None)
    rows = torch.zeros((Z, H, N), dtype=torch.bool, device="cuda")
    rows[0, 1, 7], rows[1, 0, 150] = True, True
    bad = q.clone()
    bad[rows] = NAN
    o, lse = fa.fwd_scored(bad, k, v, **args)
    assert is_nan_exactly(o, rows) and is_nan_exactly(lse, rows)
    bad = k.clone()
    bad[rows] = NAN  # each query sees its own key alone
    o, lse = fa.fwd_scored(q, bad, v, window=1, **args)
    assert is_nan_exactly(o, rows) and is_nan_exactly(lse, rows)


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Nq", [1, 150])
def test_paged_rows_of_nan_stay_nan(Nq, D, cap, bias):
    q, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(2, 4, 2, Nq, [400, 300], D, 64, 62))
    rows = torch.zeros((2, 4, Nq), dtype=torch.bool, device="cuda")
    rows[0, 1, 0], rows[1, 3, Nq - 1] = True, True
    q[rows] = NAN
    o, lse = fa.fwd_paged_scored(q, kc, vc, table, ctx, softcap=cap, slopes=slopes_of(4).cuda() if bias else None, splits=1)
    assert is_nan_exactly(o, rows) and is_nan_exactly(lse, rows)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_products_past_32_bits_are_capped(D, sign, bias):
    """Products that overflow to an infinity are -cap or cap: equal scores."""
    Z, H, N, cap = 1, 2, 200, 5.0
    q, k, v, do = (t.to(torch.bfloat16).cuda() for t in make_inputs(Z, H, N, D, 67))
    q, k = torch.full_like(q, sign * 1e25), torch.full_like(k, 1e25)
    sl = torch.zeros(H).cuda() if bias else None
    o, lse = fa.fwd_scored(q, k, v, causal=True, softcap=cap, slopes=sl)
    n = torch.arange(1, N + 1, device="cuda", dtype=torch.float64)
    want = v.double().cumsum(2) / n[:, None]
    mean = v.double().abs().cumsum(2) / n[:, None]
    # the result's rounding, half a step, and N sums in fp32
    assert bool(((o.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * mean).all())
    # a score is off by 16 half steps of the cap at most
    assert bool(((lse.double() - (sign * cap + n.log())).abs() <= 2.0 ** -24 * (16 * cap + 64)).all())
    dq, dk, dv = fa.bwd_scored(q, k, v, o, do, lse, causal=True, softcap=cap, slopes=sl)
    assert not dq.any() and not dk.any() and torch.isfinite(dv).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Nq,window", [(1, 0), (1, 60), (40, 0)])
@pytest.mark.parametrize("splits", [2, 4, 9])
def test_slices_of_nan_stay_nan(splits, Nq, window, D):
    q, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(2, 4, 2, Nq, [1200, 900], D, 64, 63))
    rows = torch.zeros((2, 4, Nq), dtype=torch.bool, device="cuda")
    rows[0, 1, 0], rows[1, 3, Nq - 1] = True, True
    bad = q.clone()
    bad[rows] = NAN
    o, lse = fa.fwd_paged_scored(bad, kc, vc, table, ctx, window=window, splits=splits)
    assert is_nan_exactly(o, rows) and is_nan_exactly(lse, rows)
    # a NaN key of one slice reaches every row that sees it
    kc[table[0, 1199 // 64 - 1 if Nq > 1 else 1199 // 64].long(), 3, 0] = NAN
    o, lse = fa.fwd_paged_scored(q, kc, vc, table, ctx, window=window, splits=splits)
    rows = torch.zeros_like(rows)
    rows[0, :2] = True
    assert is_nan_exactly(o, rows) and is_nan_exactly(lse, rows)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("splits", [1, 2, 9])
def test_unscored_slices_of_nan_stay_nan(splits, D):
    q, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(2, 4, 2, 3, [1200, 900], D, 64, 64))
    rows = torch.zeros((2, 4, 3), dtype=torch.bool, device="cuda")
    rows[0, 1, 0], rows[1, 3, 2] = True, True
    bad = q.clone()
    bad[rows] = NAN
    o, lse = fa.fwd_paged(bad, kc, vc, table, ctx, splits=splits)
    assert is_nan_exactly(o, rows) and is_nan_exactly(lse, rows)
    kc[table[0, 2].long(), 3, 0] = NAN  # in one slice of several
    o, lse = fa.fwd_paged(q, kc, vc, table, ctx, splits=splits)
    rows = torch.zeros_like(rows)
    rows[0, :2] = True
    assert is_nan_exactly(o, rows) and is_nan_exactly(lse, rows)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_selected_blocks_of_nan_stay_nan(D):
    q, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(1, 2, 1, 3, [300], D, 64, 64))
    sel = torch.tensor([[[0, 2, 4]]], dtype=torch.int32, device="cuda")
    rows = torch.zeros((1, 2, 3), dtype=torch.bool, device="cuda")
    rows[0, 1, 1] = True
    q[rows] = NAN
    o, lse = fa.fwd_sparse(q, kc, vc, table[:, None, [0, 2, 4]].contiguous(), sel,
                           torch.tensor([[3]], dtype=torch.int32, device="cuda"), ctx)
    assert is_nan_exactly(o, rows) and is_nan_exactly(lse, rows)


@pytest.mark.parametrize("cap,bias", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_that_see_nothing_are_zero_beside_nan_values(D, cap, bias):
    Z, H, N = 1, 2, 150
    q, k, v, _ = (t.cuda() for t in make_inputs(Z, H, N, D, 65))
    v[0, 0, 4] = NAN
    r = torch.tensor([0, N], dtype=torch.int32).repeat(Z, N, 1)
    r[0, ::3] = 0
    o, lse = fa.fwd_scored(q, k, v, softcap=cap, slopes=slopes_of(H).cuda() if bias else None,
                           key_ranges=fa.key_ranges(N, N, ranges=r.cuda()))
    assert not o[:, :, ::3].any() and torch.isneginf(lse[:, :, ::3]).all()
    assert torch.isnan(o[0, 0, 1]).all() and torch.isfinite(o[0, 1]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("splits", [1, 4])
def test_rows_behind_the_new_tokens_are_zero_beside_nan_values(splits, D):
    q, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(2, 4, 2, 9, [300, 200], D, 64, 66))
    vc[table[0, 0].long(), 3] = NAN
    o, lse = fa.fwd_paged_scored(q, kc, vc, table, ctx, q_lens=torch.tensor([4, 9], dtype=torch.int32).cuda(), splits=splits)
    assert not o[0, :, 4:].any() and torch.isneginf(lse[0, :, 4:]).all()
    assert torch.isnan(o[0, :, :4]).all() and torch.isfinite(o[1]).all()


def gap_case(N, kind):
    """(ranges [1, N, 2], keys that no query sees)"""
    r = torch.zeros((1, N, 2), dtype=torch.int32)
    if kind == "two":      # rows at the front and rows at the back, in turn
        r[0, ::2, 1] = 10
        r[0, 1::2, 0], r[0, 1::2, 1] = N - 40, N - 30
    elif kind == "comb":   # short ranges all over, gaps of one key upwards, every seventh row empty
        lo = (torch.arange(N) * 37) % (N - 3)
        lo = lo // 11 * 11
        r[0, :, 0], r[0, :, 1] = lo, lo + 4
        r[0, ::7] = 5
    else:                  # a gap on a tile's border, inside one query tile alone
        r[0, :, 1] = 120
        r[0, 60:, 0], r[0, 60:, 1] = 140, 200
    seen = torch.zeros(N, dtype=torch.bool)
    for lo, hi in r[0].tolist():
        seen[lo:hi] = True
    return r, ~seen


@pytest.mark.parametrize("junk", [NAN, float("inf")])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (10.0, False), (10.0, True)])
@pytest.mark.parametrize("kind", ["two", "comb", "border"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_in_a_gap_may_be_anything(D, kind, cap, bias, junk):
    H, N = 2, 300
    q, k, v, do = (t.cuda() for t in make_inputs(1, H, N, D, 69))
    r, blind = gap_case(N, kind)
    kr = fa.key_ranges(N, N, ranges=r.cuda())
    args = dict(softcap=cap, slopes=slopes_of(H).cuda() if bias else None, key_ranges=kr)
    out = []
    for fill in (0.0, junk):
        k2, v2 = k.clone(), v.clone()
        k2[:, :, blind], v2[:, :, blind] = fill, fill
        o, lse = fa.fwd_scored(q, k2, v2, **args)
        out.append((o, lse) + tuple(fa.bwd_scored(q, k2, v2, o, do, lse, **args)))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert not out[1][3][:, :, blind].any() and not out[1][4][:, :, blind].any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_in_a_gap_of_one_tile_may_be_anything_for_it(D):
    """Keys that the rows of one 128-row tile leave out, and another tile's rows see."""
    H, N = 2, 384
    q, k, v, do = (t.cuda() for t in make_inputs(1, H, N, D, 70))
    r = torch.zeros((1, N, 2), dtype=torch.int32)
    r[0, :, 1] = 20
    r[0, 1:128:2, 0], r[0, 1:128:2, 1] = 310, 350   # tile 0: [0, 20) and [310, 350)
    r[0, 128:, 1] = 200                             # the others: [0, 200)
    kr = fa.key_ranges(N, N, ranges=r.cuda())
    want = fa.fwd_scored(q, k, v, key_ranges=kr, softcap=8.0)
    v[:, :, 100] = NAN
    o, lse = fa.fwd_scored(q, k, v, key_ranges=kr, softcap=8.0)
    assert torch.equal(o[:, :, :128], want[0][:, :, :128]) and torch.equal(lse, want[1])
    assert torch.isnan(o[:, :, 128:]).all()


def test_arguments_past_the_range_of_the_c_types():
    q, k, v, do = (t.cuda() for t in make_inputs(1, 2, 100, 64, 73))
    want = fa.fwd_scored(q, k, v, causal=True)
    for wide in (100, 2 ** 31, 2 ** 32 + 5, 2 ** 70):  # hides nothing
        o, lse = fa.fwd_scored(q, k, v, causal=True, window=wide)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    pq, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(1, 2, 2, 1, [100], 64, 64, 73))
    for kw in (dict(window=-2 ** 32), dict(window=-2 ** 32 + 5), dict(softcap=1e-60), dict(softcap=-1e-60)):
        for call in (lambda **a: fa.fwd_scored(q, k, v, causal=True, **a),
                     lambda **a: fa.bwd_scored(q, k, v, *want[:1], do, want[1], causal=True, **a),
                     lambda **a: fa.fwd_paged_scored(pq, kc, vc, table, ctx, **a)):
            with pytest.raises(_native.FaError):
                call(**kw)
    with pytest.raises(_native.FaError):
        fa.fwd_paged_scored(pq, kc, vc, table, ctx, splits=2 ** 32 + 1)


def test_workspaces_are_refused_before_a_launch():
    from attention_sm_flashattention_gb300 import api
    q, k, v, do = (t.cuda() for t in make_inputs(1, 2, 100, 64, 74))
    o, lse = fa.fwd_scored(q, k, v, causal=True)
    wide = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20)
    pq, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(1, 2, 2, 1, [300], 64, 64, 74))
    for ws in (wide, torch.empty(1 << 20, dtype=torch.uint8)):
        for call in (lambda: fa.bwd_scored(q, k, v, o, do, lse, causal=True, workspace=ws),
                     lambda: fa.bwd(q, k, v, o, do, lse, causal=True, workspace=ws),
                     lambda: fa.fwd_paged_scored(pq, kc, vc, table, ctx, splits=2, workspace=ws),
                     lambda: fa.fwd_paged(pq, kc, vc, table, ctx, splits=2, workspace=ws)):
            with pytest.raises(ValueError):
                call()
    floats = torch.empty(api.bwd_workspace_size(1, 2, 100, 64, True) // 4, device="cuda")  # any type that has the bytes
    want = fa.bwd_scored(q, k, v, o, do, lse, causal=True)
    for a, b in zip(want, fa.bwd_scored(q, k, v, o, do, lse, causal=True, workspace=floats)):
        assert torch.equal(a, b)
    for a, b in zip(fa.bwd(q, k, v, o, do, lse, causal=True), fa.bwd(q, k, v, o, do, lse, causal=True, workspace=floats)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Nq", [6, 140])
def test_rows_before_position_zero_see_nothing(Nq, D, splits, causal):
    def edit(ctx):
        ctx[0], ctx[1], ctx[2] = 3, 0, 5
    o, lse = paged_case(4, 4, 2, Nq, [400] * 4, D, 32, 71, q_lens=[Nq, Nq, 5, Nq - 1], causal=causal, bias=True,
                        ctx_edit=edit, splits=splits)
    assert not o[0, :, :Nq - 3].any() and torch.isneginf(lse[0, :, :Nq - 3]).all()
    assert torch.isfinite(lse[0, :, Nq - 3:]).all() and torch.isfinite(lse[2, :, :5]).all()


@pytest.mark.parametrize("D", [64, 256])
def test_a_tile_before_position_zero_reads_no_values(D):
    q, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(1, 2, 2, 200, [200], D, 32, 72))
    ctx[0] = 30  # the first 128 rows lie before the context
    vc[:] = NAN
    o, lse = fa.fwd_paged_scored(q, kc, vc, table, ctx, causal=False, splits=1)
    assert not o[:, :, :170].any() and torch.isneginf(lse[:, :, :170]).all() and torch.isnan(o[:, :, 170:]).all()


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_gradients_of_saturated_scores(D, sign, bias):
    """Scores of 5.5 to 8.5 times the cap, where 1 - tanh^2 is 7e-5 to 2e-7: gradients keep their relative precision
    on both sides.  Half of the features carry the product, the others make dq differ between keys."""
    Z, H, N, cap, dt = 1, 2, 64, 2.0, torch.bfloat16
    _, k, v, do = make_inputs(Z, H, N, D, 68, dtype=dt)
    scale, half = 1.0 / math.sqrt(D), D // 2
    times = torch.linspace(5.5, 8.5, N)  # x / cap of the rows
    q = torch.zeros((Z, H, N, D))
    q[..., :half] = (sign * times * cap / (scale * half))[:, None]
    q = q.to(dt)
    k[..., :half] = 1.0
    sl = torch.full((H,), 1e-3) if bias else None
    args = dict(scale=scale, softcap=cap, slopes=sl.cuda() if bias else None)
    o, lse = fa.fwd_scored(*(t.cuda() for t in (q, k, v)), **args)
    got = [t.double().cpu().numpy() for t in
           fa.bwd_scored(*(t.cuda() for t in (q, k, v)), o, do.cuda(), lse, **args)[:2]]
    qn, kn, vn, dn = (t.double().numpy() for t in (q, k, v, do))
    u, s64 = 2.0 ** -8, float(np.float32(scale))
    pos = np.arange(N)
    for h in range(H):
        slope = float(sl[h]) if bias else 0.0
        oo, _, p, t = orc.head_fwd(qn[0, h], kn[0, h], vn[0, h], s64, cap, slope, np.ones((N, N), bool), pos, pos)
        x = qn[0, h] @ kn[0, h].T * s64 / cap
        fac = 4 * np.exp(-2 * np.abs(x)) / (1 + np.exp(-2 * np.abs(x))) ** 2  # 1 - tanh^2 without cancellation
        dp = dn[0, h] @ vn[0, h].T
        delta = (oo * dn[0, h]).sum(1, keepdims=True)
        ds = p * fac * (dp - delta)
        # dS: its rounding to bf16, half a step; p and the factor within 2^-14 (exponents up to 25 with an error of
        # 2^-19, fp32 reciprocals); Delta from the o that was rounded, p's rounding in it among that
        d_delta = (orc.fwd_bound(oo, p, vn[0, h], orc.F32 * 128, dt, N) * np.abs(dn[0, h])).sum(1, keepdims=True)
        d_dp = orc.F32 * D * (np.abs(dn[0, h]) @ np.abs(vn[0, h]).T)
        e = (u + 2.0 ** -14) * np.abs(ds) + p * fac * (d_delta + d_dp)
        for g, ref, off in ((got[0][0, h], s64 * ds @ kn[0, h], s64 * e @ np.abs(kn[0, h])),
                            (got[1][0, h], s64 * ds.T @ qn[0, h], s64 * e.T @ np.abs(qn[0, h]))):
            bound = off + u * (np.abs(ref) + off)
            assert (np.abs(g - ref) <= bound).all(), float((np.abs(g - ref) / bound).max())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Nq,window", [(5, 0), (20, 70), (300, 0), (300, 90)])
@pytest.mark.parametrize("bias", [False, True])
def test_gaps_with_grouped_heads_and_causal_limits(bias, Nq, window, D):
    """The few rows of grouped heads share a tile; a causal limit and a window cut the ranges; rows may end up empty."""
    Z, H, Hkv, Nk = 2, 6, 2, 300
    q, k, v, do = (t.cuda() for t in make_inputs(Z, H, Nq, D, 75, Hkv=Hkv, Nk=Nk))
    lo = (torch.arange(Z * Nq).reshape(Z, Nq) * 53) % 260 // 20 * 20
    r = torch.stack([lo, lo + 1 + torch.arange(Nq) % 9], -1).int().contiguous()
    for causal in (False, True) if window == 0 else (True,):
        blind = torch.stack([~torch.from_numpy(orc.visible(Nq, Nk, causal=causal, window=window, ranges=r[z].numpy()).any(0))
                             for z in range(Z)])[:, None].expand(Z, Hkv, Nk)
        assert blind.any() and not blind.all()
        args = dict(causal=causal, window=window, softcap=7.0, slopes=slopes_of(H).cuda() if bias else None,
                    key_ranges=fa.key_ranges(Nq, Nk, ranges=r.cuda()))
        out = []
        for fill in (0.0, NAN):
            k2, v2 = k.clone(), v.clone()
            k2[blind], v2[blind] = fill, fill
            o, lse = fa.fwd_scored(q, k2, v2, **args)
            out.append((o, lse) + tuple(fa.bwd_scored(q, k2, v2, o, do, lse, **args)))
        for a, b in zip(*out):
            assert torch.equal(a, b)
        assert not out[1][3][blind].any() and not out[1][4][blind].any()
