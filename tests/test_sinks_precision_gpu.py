"""Gradients of windows with sinks as a whole: their relative error against the
definition in 64 bits, where the sinks take most of the probability and point
one way, so that an error of Delta reaches dQ and dK undiminished.

Tolerance: what the roundings to 16 bits that these operators are meant to have
come to for the very inputs, by doing them in 64 bits: P and dS once (operands
of products), the result once; and, in dQ, Delta from the 16-bit O in the key
tiles that hold no sink.  The two parts are independent of each other, so their
squares add.  5% for the rest, which is in 32 bits: scores are off by a few
2^-24 of at most 72 (the cap of 50 in base 2), so P by 1.5e-5 of itself, and a
rounding to fp16 is off by 1.4e-4 in the mean, ten times as much: 1% of the sum of
squares; the means over 10^5 values and more move by less."""

import math

import pytest
import torch

import attention_sm_flashattention_gb300 as fa

pytestmark = pytest.mark.gpu


def inputs(H, Hkv, N, D, sinks, cap, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda h: torch.randn((1, h, N, D), generator=g, device="cuda")  # noqa: E731
    q, k, v, do = (normal(H) + 0.5) * (2.0 if cap else 1.0), normal(Hkv), normal(Hkv), normal(H)
    k[:, :, :sinks] += 0.7
    v[:, :, :sinks] *= 0.1
    return [t.to(dtype) for t in (q, k, v, do)]


def expected(q, k, v, do, o, scale, cap, window, sinks, dtype):
    """[(exact gradient, norm of the error that its roundings come to)] of dq, dk, dv."""
    G, N, D = q.shape[1] // k.shape[1], q.shape[2], q.shape[3]
    q, k, v, do, o = (t[0].double() for t in (q, k, v, do, o))
    kk, vv = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    key, pos = torch.arange(N, device=q.device)[None, :], torch.arange(N, device=q.device)[:, None]
    seen = (key <= pos) & ((key > pos - window) | (key < sinks))
    x, fac = q @ kk.transpose(1, 2) * scale, 1.0
    if cap:
        t = torch.tanh(x / cap)
        x, fac = cap * t, 1 - t * t
    p = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
    delta = ((p @ vv) * do).sum(-1, keepdim=True)
    ds = p * fac * (do @ vv.transpose(1, 2) - delta)
    bits = lambda t: t.to(dtype).double()  # noqa: E731
    shared = lambda t: t.reshape(k.shape[0], G, N, D).sum(1)  # noqa: E731
    tile = 64 if D == 256 else 128
    plain = key >= -(-sinks // tile) * tile
    off = ((o * do).sum(-1, keepdim=True) - delta) * scale * ((p * fac).masked_fill(~plain, 0.0) @ kk)
    out = []
    for exact, rounded, extra in ((scale * ds @ kk, scale * bits(ds) @ kk, off),
                                  (shared(scale * ds.transpose(1, 2) @ q), shared(scale * bits(ds).transpose(1, 2) @ q), 0 * q),
                                  (shared(p.transpose(1, 2) @ do), shared(bits(p).transpose(1, 2) @ do), 0 * q)):
        out.append((exact, math.hypot(float((bits(rounded) - exact).norm()), float(extra.norm()))))
    return out


def check(D, window, sinks, cap, dtype, N=900, seed=3):
    q, k, v, do = inputs(4, 2, N, D, sinks, cap, dtype, seed)
    how = dict(causal=True, softcap=cap, window=window, sinks=sinks)
    o, lse = fa.fwd_scored(q, k, v, **how)
    grads = fa.bwd_scored(q, k, v, o, do, lse, **how)
    assert fa.device_status() == 0
    for name, got, (exact, error) in zip(("dq", "dk", "dv"), grads,
                                         expected(q, k, v, do, o, 1 / math.sqrt(D), cap, window, sinks, dtype)):
        off = float((got[0].double() - exact).norm())
        assert off <= 1.05 * error, f"{name}: relative error {off / float(exact.norm()):.3e}, roundings {error / float(exact.norm()):.3e}"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 50.0])
@pytest.mark.parametrize("window,sinks", [(64, 8), (300, 4), (200, 60)])
def test_relative_error(window, sinks, cap, D, dtype):
    check(D, window, sinks, cap, dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 50.0])
@pytest.mark.parametrize("window,sinks", [(300, 100), (300, 200), (100, 400)])
def test_relative_error_with_sinks_in_several_tiles(window, sinks, cap, D, dtype):
    check(D, window, sinks, cap, dtype)
