"""Pins of the scored-attention and rotary oracle, the scaled frequencies, and
the entry points' refusals (all on the CPU)."""

import math

import numpy as np
import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300 import _native
from oracle import attention as dense
from oracle import scored as orc


def draw(*shapes, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g, dtype=torch.float64) for s in shapes]


@pytest.mark.parametrize("cap,bias,mask", [(0.0, False, "causal"), (3.0, True, "causal"), (2.0, False, "docs"),
                                           (0.0, True, "prefix")])
def test_against_autograd(cap, bias, mask):
    """torch's fp64 autograd of the definition, grouped heads."""
    Z, H, Hkv, N, D = 2, 4, 2, 13, 8
    q, k, v, do = draw((Z, H, N, D), (Z, Hkv, N, D), (Z, Hkv, N, D), (Z, H, N, D))
    ids = torch.tensor([[0] * 5 + [1] * 8, [3] * 2 + [4] * 10 + [3]])
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.7]) if bias else None

    def seen(z):
        if mask == "docs":
            return orc.visible(N, N, causal=True, docs=ids[z].numpy())
        return orc.visible(N, N, causal=True) if mask == "causal" else orc.visible(N, N, prefix=4 + z)

    o, lse, _, _ = orc.scored_fwd(q, k, v, 0.25, cap, slopes, seen)
    grads, _ = orc.scored_bwd(q, k, v, do, 0.25, cap, slopes, seen)
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    kk, vv = (t.repeat_interleave(H // Hkv, 1) for t in leaves[1:])
    x = leaves[0] @ kk.transpose(-1, -2) * 0.25
    if cap:
        x = cap * torch.tanh(x / cap)
    if bias:
        far = (torch.arange(N)[:, None] - torch.arange(N)[None]).abs().double()
        x = x - slopes.double()[None, :, None, None] * far
    vis = torch.stack([torch.from_numpy(seen(z)) for z in range(Z)])[:, None]
    x = x.masked_fill(~vis, -math.inf)
    y = torch.softmax(x, -1) @ vv
    assert np.abs(o - y.detach().numpy()).max() < 1e-12
    assert np.abs(lse - torch.logsumexp(x, -1).detach().numpy()).max() < 1e-12
    for a, b in zip(grads, torch.autograd.grad(y, leaves, do)):
        assert np.abs(a - b.numpy()).max() < 1e-12


def test_without_rules_equals_the_dense_oracle():
    q, k, v = draw((1, 2, 9, 8), (1, 2, 9, 8), (1, 2, 9, 8), seed=1)
    o, lse, _, _ = orc.scored_fwd(q, k, v, 0.4, seen=lambda z: orc.visible(9, 9, causal=True))
    ro, rl = dense.attn_fwd_ref(q, k, v, True, 0.4)
    assert np.abs(o - ro).max() < 1e-12 and np.abs(lse - rl).max() < 1e-12


def test_rows_that_see_nothing():
    q, k, v, do = draw((1, 1, 4, 8), (1, 1, 6, 8), (1, 1, 6, 8), (1, 1, 4, 8), seed=2)
    r = np.array([[0, 6], [2, 2], [5, 3], [1, 2]])
    seen = lambda z: orc.visible(4, 6, ranges=r)  # noqa: E731
    o, lse, _, _ = orc.scored_fwd(q, k, v, 0.4, seen=seen)
    assert not o[0, 0, 1:3].any() and np.isneginf(lse[0, 0, 1:3]).all()
    assert np.allclose(o[0, 0, 3], v[0, 0, 1].numpy())
    g, _ = orc.scored_bwd(q, k, v, do, 0.4, seen=seen)
    assert not g[0][0, 0, 1:3].any()


def test_paged_equals_dense():
    q, kc, vc = draw((1, 2, 3, 8), (4, 4, 1, 8), (4, 4, 1, 8), seed=3)
    table = np.array([[2, 0, 3]])
    o, lse, _, _ = orc.paged_scored_fwd(q, kc, vc, table, [10], [2], True, 0.4, 3.0, [0.2, 0.4], 5)
    rows = torch.cat([kc[2], kc[0], kc[3]])[:10, 0], torch.cat([vc[2], vc[0], vc[3]])[:10, 0]
    ro, rl, _, _ = orc.scored_fwd(q[:, :, :2], rows[0][None, None], rows[1][None, None], 0.4, 3.0, [0.2, 0.4],
                                  lambda z: orc.visible(2, 10, causal=True, window=5))
    assert np.abs(o[:, :, :2] - ro).max() < 1e-13 and np.abs(lse[:, :, :2] - rl).max() < 1e-13
    assert not o[:, :, 2].any() and np.isneginf(lse[:, :, 2]).all()


def test_rotary_oracle():
    x, = draw((1, 2, 5, 12), seed=4)
    pos = np.array([[0, 1, 2, 7, 3]])
    f = np.array([1.0, 0.1, 0.01, 0.5])
    for il in (False, True):
        y = orc.rotary(x, pos, f, il)
        assert np.array_equal(y[..., 8:], x.numpy()[..., 8:]) and np.allclose(y[:, :, 0], x.numpy()[:, :, 0])
        assert np.abs(orc.rotary(y, pos, f, il, inverse=True) - x.numpy()).max() < 1e-14
        # products depend on the difference of positions alone
        a, b = orc.rotary(x, pos, f, il), orc.rotary(x, pos + 1000, f, il)
        assert np.abs(a[0, 0] @ a[0, 1].T - b[0, 0] @ b[0, 1].T).max() < 1e-11
    pair = orc.rotary(x, pos, f, True)[0, 0, 3, :2]
    z = complex(x[0, 0, 3, 0], x[0, 0, 3, 1]) * complex(math.cos(7.0), math.sin(7.0))
    assert abs(pair[0] - z.real) < 1e-14 and abs(pair[1] - z.imag) < 1e-14


def test_scaled_frequencies():
    plain, one = fa.rotary_freqs(64, device="cpu")
    assert one == 1.0 and torch.allclose(plain, 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64), rtol=1e-14)
    lin, _ = fa.rotary_freqs(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, plain / 4, rtol=1e-14)
    ntk, _ = fa.rotary_freqs(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == plain[0] and abs(float(ntk[-1] * 4 / plain[-1]) - 1) < 1e-12
    yarn, m = fa.rotary_freqs(64, scaling="yarn", factor=4.0, original_len=4096, device="cpu")
    assert abs(m - (0.1 * math.log(4.0) + 1)) < 1e-15
    turns = plain * 4096 / (2 * math.pi)
    assert torch.equal(yarn[turns > 45], plain[turns > 45])
    assert torch.allclose(yarn[turns < 0.7], plain[turns < 0.7] / 4, rtol=1e-14)
    assert ((yarn <= plain) & (yarn >= plain / 4 * (1 - 1e-14))).all()
    for bad in (dict(rot=3), dict(rot=0), dict(rot=2, scaling="ntk", factor=2.0), dict(rot=8, scaling="x"),
                dict(rot=8, scaling="yarn", factor=2.0), dict(rot=8, factor=0.5)):
        with pytest.raises(ValueError):
            fa.rotary_freqs(device="cpu", **bad)


P = 4096  # a pointer value that is never read: every call below is refused before a launch
INVALID, UNSUPPORTED, WORKSPACE = _native.FA_ERR_INVALID_ARG, _native.FA_ERR_UNSUPPORTED, _native.FA_ERR_WORKSPACE


def fwd(**kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, Z=1, H=4, Hkv=2, Nq=8, Nk=8, D=64, causal=1, scale=0.1, softcap=0.0, slopes=None,
             window=0, mask=None, mask_bytes=0, dtype=0, stream=None)
    a.update(kw)
    return _native.lib().fa_fwd_scored(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=P + 8), INVALID), (dict(lse=P + 2), INVALID), (dict(softcap=-1.0), INVALID),
    (dict(softcap=math.inf), INVALID), (dict(softcap=math.nan), INVALID), (dict(window=-1), INVALID),
    (dict(window=4, causal=0), INVALID), (dict(slopes=P + 1), INVALID), (dict(mask=P + 4, mask_bytes=1 << 20), INVALID),
    (dict(mask=P, mask_bytes=64), WORKSPACE), (dict(dtype=2), INVALID), (dict(H=3), INVALID), (dict(Z=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(D=96), UNSUPPORTED), (dict(Nq=9), UNSUPPORTED), (dict(causal=2), INVALID),
    (dict(window=5, Nk=1 << 30), UNSUPPORTED)])
def test_fwd_scored_refusals(kw, code):
    assert fwd(**kw) == code


# softcap 4096 is the largest: a score's error, a few 2^-24 of the cap, is then a few 2^-12, one rounding of a
# probability to fp16; scale / softcap has to be a finite factor
@pytest.mark.parametrize("softcap,scale,refused", [
    (4096.0, 0.1, False), (4097.0, 0.1, True), (1e6, 0.1, True), (3e38, 0.1, True), (1e-30, 0.1, False),
    (1e-38, 10.0, True), (1e-45, 1.0, True), (30.0, 3e38, True)])
def test_softcap_range(softcap, scale, refused):
    assert (fwd(softcap=softcap, scale=scale) == UNSUPPORTED) == refused
    for call in (bwd, paged):
        assert (call(softcap=softcap, scale=scale) == UNSUPPORTED) == refused


def bwd(**kw):
    a = dict(q=P, k=P, v=P, o=P, do=P, lse=P, dq=P, dk=P, dv=P, ws=P, ws_bytes=1 << 20, Z=1, H=4, Hkv=2, Nq=8, Nk=8,
             D=64, causal=1, scale=0.1, softcap=0.0, slopes=None, window=0, mask=None, mask_bytes=0, dtype=0, stream=None)
    a.update(kw)
    return _native.lib().fa_bwd_scored(*a.values())


def paged(**kw):
    a = dict(q=P, kc=P, vc=P, table=P, ctx=P, q_lens=None, o=P, lse=P, ws=None, ws_bytes=0, B=1, H=4, Hkv=2, Nq=1, D=64,
             pages=4, page=16, max_pages=4, splits=1, causal=1, scale=0.1, softcap=0.0, slopes=None, window=0, dtype=0,
             stream=None)
    a.update(kw)
    return _native.lib().fa_fwd_paged_scored(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(do=None), INVALID), (dict(softcap=-1.0), INVALID), (dict(window=1, causal=0), INVALID),
    (dict(mask=P, mask_bytes=8), WORKSPACE), (dict(dtype=-1), INVALID), (dict(D=32), UNSUPPORTED)])
def test_bwd_scored_refusals(kw, code):
    a = dict(q=P, k=P, v=P, o=P, do=P, lse=P, dq=P, dk=P, dv=P, ws=P, ws_bytes=1 << 20, Z=1, H=4, Hkv=2, Nq=8, Nk=8,
             D=64, causal=1, scale=0.1, softcap=0.0, slopes=None, window=0, mask=None, mask_bytes=0, dtype=0, stream=None)
    a.update(kw)
    assert _native.lib().fa_bwd_scored(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), INVALID), (dict(q_lens=P + 2), INVALID), (dict(splits=0, ws=P), INVALID),
    (dict(splits=257, ws=P), INVALID), (dict(splits=2), WORKSPACE), (dict(splits=2, ws=P + 4), WORKSPACE),
    (dict(softcap=-2.0), INVALID), (dict(window=3, causal=0), INVALID), (dict(page=24), UNSUPPORTED),
    (dict(D=256, page=128), UNSUPPORTED), (dict(max_pages=1 << 28), UNSUPPORTED), (dict(pages=0), INVALID)])
def test_paged_scored_refusals(kw, code):
    a = dict(q=P, kc=P, vc=P, table=P, ctx=P, q_lens=None, o=P, lse=P, ws=None, ws_bytes=0, B=1, H=4, Hkv=2, Nq=1, D=64,
             pages=4, page=16, max_pages=4, splits=1, causal=1, scale=0.1, softcap=0.0, slopes=None, window=0, dtype=0,
             stream=None)
    a.update(kw)
    assert _native.lib().fa_fwd_paged_scored(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(docs=None), INVALID), (dict(prefix=P), INVALID), (dict(docs=P + 2), INVALID), (dict(Z=0), INVALID),
    (dict(docs=None, ranges=P + 4), INVALID), (dict(Nq=9), UNSUPPORTED), (dict(mask=None), WORKSPACE),
    (dict(nbytes=156), WORKSPACE), (dict(mask=P + 8), WORKSPACE), (dict(Nk=0x7fffffff), UNSUPPORTED)])
def test_key_ranges_refusals(kw, code):
    a = dict(docs=P, prefix=None, ranges=None, mask=P, nbytes=4096, Z=1, Nq=8, Nk=8, stream=None)
    a.update(kw)
    assert _native.lib().fa_key_ranges(*a.values()) == code
    assert _native.lib().fa_key_ranges_size(2, 130, 300) == 4 * (520 + 2 * 2 * 4 + 2 * 3 * 4 + 2 * 300 * 2)


S3 = (_native.ctypes.c_longlong * 3)(512, 64, 64)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(q=P + 1), INVALID), (dict(k_out=None), INVALID), (dict(pos=None), INVALID),
    (dict(pos=P + 4), INVALID), (dict(freqs=P + 4), INVALID), (dict(rot=7), UNSUPPORTED), (dict(rot=66), UNSUPPORTED),
    (dict(rot=0), INVALID), (dict(D=80), UNSUPPORTED), (dict(il=2), INVALID), (dict(inv=2), INVALID),
    (dict(mscale=math.inf), INVALID), (dict(dtype=7), INVALID), (dict(N=-1), INVALID), (dict(H=0), INVALID),
    (dict(N=0), 0), (dict(Z=1 << 20, N=1 << 20), UNSUPPORTED)])
def test_rotary_refusals(kw, code):
    a = dict(q=P, qs=S3, qo=P, qos=S3, k=P, ks=S3, k_out=P, kos=S3, pos=P, ps=0, freqs=P, Z=1, H=4, Hkv=2, N=8, D=64,
             rot=64, il=0, inv=0, mscale=1.0, dtype=0, stream=None)
    a.update(kw)
    assert _native.lib().fa_rotary(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(slots=None), INVALID), (dict(slots=P + 4), INVALID), (dict(kc=P + 8), INVALID), (dict(Hkv=0), INVALID),
    (dict(pages=0), INVALID), (dict(v=None), INVALID), (dict(rot=130), UNSUPPORTED), (dict(Z=0), 0)])
def test_rotary_and_cache_refusals(kw, code):
    a = dict(q=P, qs=S3, qo=P, qos=S3, k=P, ks=S3, v=P, vs=S3, pos=P, ps=0, freqs=P, slots=P, kc=P, vc=P, Z=1, H=4,
             Hkv=2, N=8, D=64, rot=64, il=0, mscale=1.0, pages=4, page=16, dtype=0, stream=None)
    a.update(kw)
    assert _native.lib().fa_rotary_and_cache(*a.values()) == code


def test_python_refusals():
    t = torch.zeros((1, 2, 4, 64), dtype=torch.float16)
    pos, f = torch.zeros((1, 4), dtype=torch.int64), torch.ones(32, dtype=torch.float64)
    for call in (lambda: fa.fwd_scored(t, t, t), lambda: fa.bwd_scored(t, t, t, t, t, t), lambda: fa.rotary(t, t, pos, f),
                 lambda: fa.rotary_and_cache(t, t, t, pos, f, pos, t, t), lambda: fa.key_ranges(4, 4),
                 lambda: fa.key_ranges(4, 4, doc_ids=torch.zeros((1, 4), dtype=torch.int32)),
                 lambda: fa.fwd_paged_scored(t, t, t, pos, pos)):
        with pytest.raises(ValueError):
            call()
