"""Rotary positions with several axes against the fp64 oracle, axis by axis.

Tolerance as for one axis (test_rotary_gpu.py): one rounding of x0 c - x1 s to
16 bits, c and s off by a few 2^-24 and the angle by 2^-32 turns."""

import numpy as np
import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from oracle import scored as orc
from test_rotary_gpu import inputs, near

pytestmark = pytest.mark.gpu


def grid(A, Z, N, seed, far=10 ** 6):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-far, far, (A, Z, N), generator=g).cuda()


def want(x, positions, axes, freqs, interleaved=False, inverse=False, mscale=1.0):
    """Each pair from the oracle's turn by its own axis; one without an axis by position 0."""
    rot = 2 * freqs.numel()
    if positions.dim() == 2:
        positions = positions[:, None].expand(-1, x.shape[0], -1)
    y = x.double().cpu().numpy().copy()
    for a in list(range(positions.shape[0])) + [None]:
        p = torch.zeros_like(positions[0]) if a is None else positions[a]
        t = orc.rotary(x, p, freqs, interleaved, inverse, mscale)
        ax = axes.cpu().numpy()
        pairs = np.nonzero((ax < 0) | (ax >= positions.shape[0]) if a is None else ax == a)[0]
        for at in ((2 * pairs, 2 * pairs + 1) if interleaved else (pairs, pairs + rot // 2)):
            y[..., at] = t[..., at]
    return y


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("D,rot,A", [(64, 64, 3), (64, 16, 2), (128, 128, 3), (128, 64, 4), (256, 256, 2), (256, 32, 1),
                                     (64, 2, 3), (128, 20, 3), (256, 250, 5)])
def test_rotary_axes(D, rot, A, dealt, interleaved, dtype):
    q, k, _, _ = inputs(2, 5, 2, 37, D, dtype, 61)
    pos = grid(A, 2, 37, 62)
    freqs, _ = fa.rotary_freqs(rot)
    share = rot // 2 // A
    axes = fa.rotary_axes([rot // 2 - share * (A - 1)] + [share] * (A - 1), dealt)
    how = dict(interleaved=interleaved, axes=axes)
    qo, ko = fa.rotary(q, k, pos, freqs, **how)
    for y, x in ((qo, q), (ko, k)):
        near(y, want(x, pos, axes, freqs, interleaved), x, dtype)
        assert torch.equal(y[..., rot:], x[..., rot:])
    dq, dk = fa.rotary_bwd(qo, ko, pos, freqs, **how)
    for y, x in ((dq, qo), (dk, ko)):
        near(y, want(x, pos, axes, freqs, interleaved, inverse=True), x, dtype)


@pytest.mark.parametrize("Z,N", [(1, 1), (1, 2), (3, 1), (1, 16), (2, 17), (1, 4097)])
@pytest.mark.parametrize("rot", [128, 20])
def test_lengths(rot, Z, N):
    q, k, _, _ = inputs(Z, 3, 1, N, 128, torch.float16, 63)
    pos, axes = grid(3, Z, N, 64), fa.rotary_axes([rot // 2 - 2, 1, 1], dealt=True)
    freqs, _ = fa.rotary_freqs(rot)
    qo, ko = fa.rotary(q, k, pos, freqs, axes=axes)
    near(qo, want(q, pos, axes, freqs), q, torch.float16)
    near(ko, want(k, pos, axes, freqs), k, torch.float16)
    assert torch.equal(fa.rotary(q, None, pos, freqs, axes=axes), qo)


@pytest.mark.parametrize("rot", [64, 20])
def test_equal_axes_are_one_axis(rot):
    """Bit for bit: text tokens, whose position is the same on every axis."""
    q, k, _, pos = inputs(2, 4, 2, 100, 64, torch.bfloat16, 65)
    freqs, _ = fa.rotary_freqs(rot)
    a = fa.rotary(q, k, pos, freqs, mscale=1.25)
    b = fa.rotary(q, k, torch.stack([pos] * 3), freqs, mscale=1.25, axes=fa.rotary_axes([rot // 2 - 6, 3, 3], True))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("rot", [64, 20])
def test_pairs_without_an_axis_are_scaled_alone(rot):
    q, k, _, _ = inputs(1, 2, 1, 9, 64, torch.float16, 66)
    pos, freqs = grid(2, 1, 9, 67), fa.rotary_freqs(rot)[0]
    axes = torch.tensor([(-1, 0, 2, 1, 1 << 30, -(1 << 31))[j % 6] for j in range(rot // 2)], dtype=torch.int32).cuda()
    qo, _ = fa.rotary(q, k, pos, freqs, mscale=0.5, axes=axes)
    near(qo, want(q, pos, axes, freqs, mscale=0.5), q, torch.float16, 0.5)
    still = (axes < 0) | (axes > 1)
    assert torch.equal(qo[..., :rot // 2][..., still], q[..., :rot // 2][..., still] * 0.5)


def test_shared_positions_in_place_and_strides():
    q, k, _, _ = inputs(3, 4, 2, 50, 128, torch.float16, 68)
    freqs, axes, pos = fa.rotary_freqs(128)[0], fa.rotary_axes([32, 16, 16]), grid(3, 1, 50, 69)[:, 0].contiguous()
    qo, ko = fa.rotary(q, k, pos, freqs, axes=axes)
    near(qo, want(q, pos, axes, freqs), q, torch.float16)
    near(ko, want(k, pos, axes, freqs), k, torch.float16)
    same = fa.rotary(q, k, pos[:, None].expand(3, 3, 50).contiguous(), freqs, axes=axes)
    assert torch.equal(same[0], qo) and torch.equal(same[1], ko)
    fa.rotary(q, k, pos, freqs, axes=axes, out=(q, k))  # q and k: views of a projection's output
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("rot", [128, 64, 20])
@pytest.mark.parametrize("Z,N", [(4, 1), (2, 70)])
def test_into_the_cache(rot, Z, N):
    q, k, v, _ = inputs(Z, 6, 2, N, 128, torch.bfloat16, 70)
    pos, freqs, axes = grid(3, Z, N, 71), fa.rotary_freqs(rot)[0], fa.rotary_axes([rot // 2 - 4, 2, 2], dealt=True)
    pages, page = Z * N // 16 + 3, 16
    caches = [torch.full((pages, page, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    g = torch.Generator().manual_seed(72)
    slots = torch.randperm(pages * page, generator=g)[:Z * N].reshape(Z, N).cuda()
    slots[0, 0] = -1
    qo, ko = fa.rotary(q, k, pos, freqs, interleaved=True, axes=axes)
    out = fa.rotary_and_cache(q, k, v, pos, freqs, slots, *caches, interleaved=True, axes=axes)
    assert torch.equal(out, qo)
    ref = [torch.full_like(c, 7.0) for c in caches]
    live = slots.flatten() >= 0
    for c, x in zip(ref, (ko, v)):
        c.flatten(0, 1)[slots.flatten()[live]] = x.transpose(1, 2).flatten(0, 1)[live]
    assert all(torch.equal(a, b) for a, b in zip(caches, ref))


def test_captured():
    q, k, _, _ = inputs(2, 4, 2, 33, 64, torch.float16, 73)
    pos, freqs, axes = grid(3, 2, 33, 74), fa.rotary_freqs(64)[0], fa.rotary_axes([16, 8, 8])
    qo, ko = (torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k))
    fa.rotary(q, k, pos, freqs, out=(qo, ko), axes=axes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.rotary(q, k, pos, freqs, out=(qo, ko), axes=axes)
    pos.copy_(grid(3, 2, 33, 75))
    graph.replay()
    a, b = fa.rotary(q, k, pos, freqs, axes=axes)
    assert torch.equal(a, qo) and torch.equal(b, ko)


def test_gradient_against_differences():
    """d sum(w . rotary(x)) / dx, by central differences of the oracle's turn (linear: they are exact but for rounding)."""
    q, _, _, _ = inputs(1, 1, 1, 5, 64, torch.float16, 76)
    w, _, _, _ = inputs(1, 1, 1, 5, 64, torch.float16, 77)
    pos, freqs, axes = grid(2, 1, 5, 78, far=50), fa.rotary_freqs(64)[0], fa.rotary_axes([20, 12])
    got = fa.rotary_bwd(w, None, pos, freqs, axes=axes)
    for at in ((0, 0, 3, 5), (0, 0, 4, 45), (0, 0, 0, 63)):
        tot = []
        for s in (1, -1):
            x = q.double().clone()
            x[at] += s
            tot.append(float((want(x, pos, axes, freqs) * w.double().cpu().numpy()).sum()))
        assert abs(float(got[at]) - (tot[0] - tot[1]) / 2) <= 2.0 ** -11 * abs(float(got[at])) + 1e-5


def test_refusals():
    q, k, _, pos = inputs(2, 2, 1, 9, 64, torch.float16, 79)
    freqs, axes = fa.rotary_freqs(64)[0], fa.rotary_axes([16, 8, 8])
    p3 = torch.stack([pos] * 3)
    for bad in (dict(axes=axes[:-1]), dict(axes=axes.long()), dict(axes=axes.cpu()), dict(positions=pos[0]),
                dict(positions=p3[:, :1].contiguous()), dict(positions=p3.int()), dict(positions=p3[:0]),
                dict(positions=p3.transpose(0, 1))):
        how = dict(positions=p3, axes=axes) | bad
        with pytest.raises(ValueError):
            fa.rotary(q, k, how["positions"], freqs, axes=how["axes"])
    with pytest.raises(ValueError):  # without axes, one axis
        fa.rotary(q, k, p3, freqs)
