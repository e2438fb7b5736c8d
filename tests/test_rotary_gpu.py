"""Rotary positions (fa_rotary, fa_rotary_and_cache) against the fp64 oracle.

Tolerance: the result is one rounding of x0 c - x1 s to 16 bits (half a step),
with c and s off by a few 2^-24 and the angle by 2^-32 turns."""

import math

import numpy as np
import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from oracle import scored as orc

pytestmark = pytest.mark.gpu
HALF = orc.HALF_STEP


def near(got, want, x, dtype, mscale=1.0):
    got = got.double().cpu().numpy()
    big = np.abs(x.double().cpu().numpy()).max() * abs(mscale)
    tol = HALF[dtype] * np.abs(want) + big * (16 * 2.0 ** -24 + 2 * math.pi * 2.0 ** -31) + orc.TINY[dtype]
    d = np.abs(got - want)
    assert (d <= tol).all(), f"off by {(d - tol).max():.3e} past the bound"


def inputs(Z, H, Hkv, N, D, dtype, seed, far=5000):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((Z, N, H + 2 * Hkv, D), generator=g).to(dtype).cuda()
    q, k, v = (t.transpose(1, 2) for t in qkv.split([H, Hkv, Hkv], 2))
    pos = (torch.randint(0, far + 1, (Z, 1), generator=g) + torch.arange(N)[None]).cuda()
    return q, k, v, pos


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (256, 256), (256, 32), (64, 2), (128, 20),
                                   (256, 250)])
def test_rotary(D, rot, interleaved, dtype):
    q, k, _, pos = inputs(2, 5, 2, 37, D, dtype, 51)
    freqs, _ = fa.rotary_freqs(rot)
    qo, ko = fa.rotary(q, k, pos, freqs, interleaved=interleaved)
    assert qo.is_contiguous() and ko.is_contiguous()
    for y, x in ((qo, q), (ko, k)):
        near(y, orc.rotary(x, pos, freqs, interleaved), x, dtype)
        assert torch.equal(y[..., rot:], x[..., rot:])
    dq, dk = fa.rotary_bwd(qo, ko, pos, freqs, interleaved=interleaved)
    for y, x in ((dq, qo), (dk, ko)):
        near(y, orc.rotary(x, pos, freqs, interleaved, inverse=True), x, dtype)


@pytest.mark.parametrize("Z,N", [(1, 1), (1, 2), (3, 1), (1, 16), (2, 17), (1, 4097)])
def test_lengths(Z, N):
    q, k, _, pos = inputs(Z, 3, 1, N, 128, torch.float16, 52)
    freqs, _ = fa.rotary_freqs(128)
    qo, ko = fa.rotary(q, k, pos, freqs)
    near(qo, orc.rotary(q, pos, freqs), q, torch.float16)
    near(ko, orc.rotary(k, pos, freqs), k, torch.float16)
    assert torch.equal(fa.rotary(q, None, pos, freqs), qo)


def test_far_and_negative_positions():
    q, k, _, _ = inputs(1, 2, 1, 6, 64, torch.float16, 53)
    pos = torch.tensor([[0, -1, -123456, 10 ** 6, 2 ** 31 + 5, 2 ** 40 + 3]]).cuda()
    freqs, _ = fa.rotary_freqs(64)
    qo, _ = fa.rotary(q, k, pos, freqs)
    want = orc.rotary(q, pos, freqs)
    big = float(q.abs().max())
    # the frequency in turns is rounded to 53 bits: off by 2^-51 of a turn per position at most
    slack = np.abs(pos.cpu().numpy()).astype(np.float64)[:, None, :, None] * 2.0 ** -51 * 2 * math.pi * big
    d = np.abs(qo.double().cpu().numpy() - want)
    assert (d <= HALF[torch.float16] * np.abs(want) + big * 20 * 2.0 ** -24 + slack).all()


def test_shared_positions_strides_and_in_place():
    q, k, v, pos = inputs(2, 4, 2, 33, 128, torch.bfloat16, 54)
    freqs, _ = fa.rotary_freqs(64)
    shared = pos[0].contiguous()
    a = fa.rotary(q, k, shared, freqs, mscale=1.25)
    want = orc.rotary(q, shared[None].expand(2, -1), freqs, mscale=1.25)
    near(a[0][..., :64], want[..., :64], q, torch.bfloat16, 1.25)
    # misaligned rows: a view one value into a wider buffer
    wide = torch.zeros((2, 4, 33, 131), dtype=torch.bfloat16, device="cuda")
    wide[..., 1:129] = q
    b = fa.rotary(wide[..., 1:129], k, shared, freqs, mscale=1.25)
    assert torch.equal(b[0], a[0]) and torch.equal(b[1], a[1])
    # into strided outputs, and in place
    out = tuple(torch.full((2, 33, t.shape[1], 128), 7.0, dtype=t.dtype, device="cuda").transpose(1, 2) for t in (q, k))
    c = fa.rotary(q, k, shared, freqs, mscale=1.25, out=out)
    assert c[0] is out[0] and torch.equal(c[0], a[0]) and torch.equal(c[1], a[1])
    fa.rotary(q, k, shared, freqs, mscale=1.25, out=(q, k))
    assert torch.equal(q, a[0]) and torch.equal(k, a[1])


@pytest.mark.parametrize("rot,D", [(128, 128), (20, 128), (64, 64), (256, 256)])
@pytest.mark.parametrize("Z,N", [(3, 1), (2, 50)])
def test_rotary_and_cache(rot, D, Z, N):
    q, k, v, pos = inputs(Z, 6, 2, N, D, torch.float16, 55)
    freqs, _ = fa.rotary_freqs(rot)
    pages, page = 11, 16
    g = torch.Generator().manual_seed(2)
    slots = torch.randperm(pages * page, generator=g)[: Z * N].reshape(Z, N)
    slots[0, 0] = -1
    if N > 1:
        slots[1, 3] = pages * page  # past the cache
        slots[1, 4] = 2 ** 40
    kc = torch.randn((pages, page, 2, D), generator=g).half().cuda()
    vc = torch.randn((pages, page, 2, D), generator=g).half().cuda()
    k0, v0 = kc.clone(), vc.clone()
    qo = fa.rotary_and_cache(q, k, v, pos, freqs, slots.cuda(), kc, vc, interleaved=True)
    wq, wk = fa.rotary(q, k, pos, freqs, interleaved=True)
    assert torch.equal(qo, wq)
    ok = (slots >= 0) & (slots < pages * page)
    for z, n in ok.nonzero().tolist():
        s = int(slots[z, n])
        k0[s // page, s % page] = wk[z, :, n]
        v0[s // page, s % page] = v[z, :, n]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_empty_batch_and_graph():
    freqs, _ = fa.rotary_freqs(64)
    q = torch.empty((2, 3, 0, 64), dtype=torch.float16, device="cuda")
    assert fa.rotary(q, None, torch.empty((2, 0), dtype=torch.int64, device="cuda"), freqs).shape == q.shape
    q, k, _, pos = inputs(1, 3, 1, 20, 64, torch.float16, 56)
    fa.rotary(q, k, pos, freqs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo, ko = fa.rotary(q, k, pos, freqs)
    pos += 17
    graph.replay()
    torch.cuda.synchronize()
    a, b = fa.rotary(q, k, pos, freqs)
    assert torch.equal(a, qo) and torch.equal(b, ko)


def test_training_step_and_decode_step():
    """The operators in a row, as a model's layer calls them."""
    Z, H, Hkv, N, D, page = 2, 4, 2, 200, 64, 16
    q, k, v, pos = inputs(Z, H, Hkv, N, D, torch.float16, 57, far=0)
    freqs, _ = fa.rotary_freqs(D)
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625], device="cuda")
    rules = dict(causal=True, softcap=20.0, slopes=slopes)
    qr, kr = fa.rotary(q, k, pos, freqs)
    vr = v.contiguous()
    o, lse = fa.fwd_scored(qr, kr, vr, **rules)
    do = torch.randn_like(o)
    dq, dk, dv = fa.bwd_scored(qr, kr, vr, o, do, lse, **rules)
    gq, gk = fa.rotary_bwd(dq, dk, pos, freqs)
    # the turn is orthogonal: gradients keep their length (one rounding of each value)
    for a, b in ((gq, dq), (gk, dk)):
        assert abs(float(a.double().norm() / b.double().norm()) - 1) < 2.0 ** -10
    # the same sequence through the cache: all but the last tokens as a chunk, then token by token
    pages = Z * ((N + page - 1) // page)
    kc = torch.zeros((pages, page, Hkv, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).reshape(Z, -1).int().cuda()

    def slots(a, b):
        p = torch.arange(a, b, device="cuda")
        return (table[:, p // page].long() * page + p % page).contiguous()

    done = []
    for a, b in [(0, N - 3)] + [(n, n + 1) for n in range(N - 3, N)]:
        qn = fa.rotary_and_cache(q[:, :, a:b], k[:, :, a:b], v[:, :, a:b], pos[:, a:b].contiguous(), freqs, slots(a, b),
                                 kc, vc)
        ctx = torch.full((Z,), b, dtype=torch.int32, device="cuda")
        done.append(fa.fwd_paged_scored(qn, kc, vc, table, ctx, softcap=20.0, slopes=slopes))
    oc, lc = torch.cat([x[0] for x in done], 2), torch.cat([x[1] for x in done], 2)
    # both are within P's and o's rounding of the exact result
    assert float((oc.float() - o.float()).abs().max()) <= 4 * 2.0 ** -11 * float(v.abs().max())
    assert float((lc - lse).abs().max()) <= 2e-5
