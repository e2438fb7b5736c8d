"""Page tables (cache_step, cache_release) against the oracle, value by value:
whole numbers, so nothing may differ.  And a serving loop that uses them with
rotary positions on several axes and windows with sinks."""

import math
import random

import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from oracle import paging as orc
from oracle import scored as sorc
from test_scored_gpu import within

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(rng, B, max_pages, page, lens, spare, spoil=False):
    """Tables of sequences of `lens` tokens, a stack of the pages that are left, as lists."""
    held = [min(-(-max(n, 0) // page), max_pages) for n in lens]
    pages = sum(held) + spare
    ids = list(range(pages))
    rng.shuffle(ids)
    table = [[-1] * max_pages for _ in range(B)]
    for b, n in enumerate(held):
        for i in range(n):
            table[b][i] = ids.pop()
    if spoil:
        for b in range(B):
            table[b][rng.randrange(max_pages)] = rng.choice([-1, -5, pages, 2 ** 31 - 1])
    stack = ids + [0] * (pages - len(ids))
    return stack, len(ids), table, pages


def check_step(stack, count, table, lens, q_lens, N, page, in_place):
    want = orc.step(stack, count, table, lens, q_lens, N, page)
    s, c, t, n = i32(stack), i32([count]), i32(table), i32(lens)
    q = i32(q_lens) if q_lens is not None else None
    B = len(lens)
    out = None
    if in_place:
        # odd addresses: 8-byte aligned outputs
        room = torch.full((2, B * N + 1), -9, dtype=torch.int64, device="cuda")
        out = (room[0, 1:].view(B, N), room[1, 1:].view(B, N), n, c)
    got = fa.cache_step(s, c, t, n, q, N, page, out=out)
    for a, b in zip(got, want[:4]):
        assert a.flatten().tolist() == torch.tensor(b, dtype=torch.int64).flatten().tolist()
    assert t.tolist() == want[4]
    if in_place:
        assert (room[:, 0] == -9).all()
    else:  # inputs are left alone
        assert n.tolist() == lens and c.tolist() == [count]
    assert s.tolist() == stack
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [1, 16, 64, 100])
@pytest.mark.parametrize("B,N", [(1, 1), (3, 1), (64, 1), (2049, 1), (5, 2), (700, 3), (3, 1000), (1, 5000), (40, 129),
                                 (1025, 2), (2048, 1)])
def test_step(B, N, page, in_place):
    rng = random.Random(B * 1000 + N + page)
    max_pages = -(-(300 + N) // page)
    lens = [rng.choice([0, 0, page, rng.randint(0, 300)]) for _ in range(B)]
    q = None if rng.random() < 0.3 else [rng.choice([0, N, rng.randint(0, N)]) for _ in range(B)]
    stack, count, table, _ = pool(rng, B, max_pages, page, lens, sum(-(-(N + page) // page) for _ in range(B)) + 3)
    want = check_step(stack, count, table, lens, q, N, page, in_place)
    assert want[3] >= 0 and (q is not None or min(min(r) for r in want[0]) >= 0)


@pytest.mark.parametrize("seed", range(12))
def test_step_odd_inputs(seed):
    """Too few pages, rows that end, lengths and counts out of range, entries that name no page."""
    rng = random.Random(seed)
    B, N, page, max_pages = rng.choice([1, 7, 90]), rng.choice([1, 9, 60]), rng.choice([3, 16]), 5
    lens = [rng.choice([-4, 0, 1, page * max_pages - 1, page * max_pages, page * max_pages + 7, 2 ** 31 - 1,
                        rng.randint(0, page * max_pages)]) for _ in range(B)]
    q = [rng.choice([-3, 0, 1, N, N + 5, 2 ** 31 - 1]) for _ in range(B)]
    stack, count, table, pages = pool(rng, B, max_pages, page, lens, rng.choice([1, 4, 50]), spoil=True)
    for c in (count, -2, pages + 9):
        check_step(stack, c, table, lens, q, N, page, in_place=seed % 2 == 0)


@pytest.mark.parametrize("B,max_pages", [(1, 1), (1, 300), (5, 7), (64, 128), (129, 33), (1000, 3), (33, 1500)])
def test_release(B, max_pages):
    rng = random.Random(B + max_pages)
    page = 16
    for spoil, share in ((False, 0.4), (True, 0.4), (True, 1.0), (False, 0.0)):
        lens = [rng.choice([0, 1, page * max_pages, rng.randint(0, page * max_pages)]) for _ in range(B)]
        stack, count, table, pages = pool(rng, B, max_pages, page, lens, 5, spoil)
        done = [rng.random() < share for _ in range(B)]
        lens = [rng.choice([-3, n, n + 10 ** 6]) if rng.random() < 0.1 else n for n in lens]
        for in_place in (False, True):
            wl, wc, ws = orc.release(stack, count, table, lens, done, page)
            s, c, t, n = i32(stack), i32([count]), i32(table), i32(lens)
            got = fa.cache_release(s, c, t, n, torch.tensor(done, device="cuda"), page, out=(n, c) if in_place else None)
            assert got[0].tolist() == wl and got[1].tolist() == [wc] and s.tolist() == ws and t.tolist() == table


def test_pages_given_back_twice_do_not_overfill():
    stack, table = list(range(6)), [[0, 1, 2, 3]] * 3
    wl, wc, ws = orc.release(stack, 4, table, [64] * 3, [True] * 3, 16)
    s = i32(stack)
    got = fa.cache_release(s, i32([4]), i32(table), i32([64] * 3), torch.ones(3, dtype=torch.bool, device="cuda"), 16)
    assert wc == 6 and got[1].tolist() == [6] and s.tolist() == ws and got[0].tolist() == wl


def test_refusals():
    s, c = fa.page_pool(8)
    t, n = i32([[-1] * 4] * 2), i32([0, 0])
    out = [torch.zeros((2, 3), dtype=torch.int64, device="cuda") for _ in range(2)] + [i32([0, 0]), i32([0])]
    for bad in ((out[0], out[0], out[2], out[3]), (out[0], out[1], n[:1], out[3]), (out[0], out[1], s[:2], out[3]),
                (out[0], out[1], out[2], n[:1]), (out[0].int(), out[1], out[2], out[3])):
        with pytest.raises(ValueError):
            fa.cache_step(s, c, t, n, None, 3, 16, out=bad)
    with pytest.raises(ValueError):
        fa.cache_step(s, c, t, n, None, 0, 16)
    done = torch.zeros(2, dtype=torch.bool, device="cuda")
    for bad in ((n, n[:1]), (s[:2], out[3])):
        with pytest.raises(ValueError):
            fa.cache_release(s, c, t, n, done, 16, out=bad)
    with pytest.raises(ValueError):
        fa.cache_release(s, c, t, n, done.int(), 16)
    with pytest.raises(Exception, match="workspace"):
        fa.cache_release(s, c, t, n, done, 16, workspace=torch.zeros(2, dtype=torch.int32, device="cuda"))


def test_other_stream():
    """A call on a stream of its own, ordered by the caller."""
    rng = random.Random(5)
    lens = [rng.randint(0, 500) for _ in range(300)]
    stack, count, table, _ = pool(rng, 300, 40, 16, lens, 900)
    want = orc.step(stack, count, table, lens, None, 9, 16)
    s, c, t, n = i32(stack), i32([count]), i32(table), i32(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.cache_step(s, c, t, n, None, 9, 16, stream=side)
    back = fa.cache_release(s, got[3], t, got[2], torch.ones(300, dtype=torch.bool, device="cuda"), 16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got[0].tolist() == want[0] and t.tolist() == want[4]
    wl, wc, ws = orc.release(stack, want[3], want[4], want[2], [True] * 300, 16)
    assert back[0].tolist() == wl and back[1].tolist() == [wc] and s.tolist() == ws


@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(captured):
    """Prefill of a ragged batch, then single tokens, then a sequence that ends and another in its place: tables, rotary
    positions on three axes into the cache, and attention within a window with sinks, against the oracle over the whole
    sequences.  The single-token step as a graph that moves itself on, or call by call."""
    B, H, Hkv, D, page, max_pages, window, sinks, N0 = 3, 4, 2, 64, 16, 12, 24, 5, 70
    dtype = torch.float16
    g = torch.Generator().manual_seed(7)
    stack, count = fa.page_pool(B * max_pages + 2)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((stack.numel(), page, Hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    freqs, _ = fa.rotary_freqs(D)
    axes = fa.rotary_axes([16, 8, 8], dealt=True)
    scale = 1.0 / math.sqrt(D)
    seqs = [[] for _ in range(B)]  # per sequence: (k, v, position) of its tokens, as the oracle keeps them

    def grid(pos):  # [B, N] -> [3, B, N]: frames of 4 by 5
        return torch.stack([pos // 20, pos // 5 % 4, pos % 5])

    def step(q, k, v, q_lens, N):
        slots, pos, _, _ = fa.cache_step(stack, count, table, lens, q_lens, N, page, out=(slots_of[N], pos_of[N], lens, count))
        qr = fa.rotary_and_cache(q, k, v, grid(pos), freqs, slots, kc, vc, axes=axes)
        return fa.fwd_paged_scored(qr, kc, vc, table, lens, q_lens=q_lens, window=window, sinks=sinks)

    slots_of = {n: torch.empty((B, n), dtype=torch.int64, device="cuda") for n in (1, N0)}
    pos_of = {n: torch.empty((B, n), dtype=torch.int64, device="cuda") for n in (1, N0)}

    def draw(N):
        return [torch.randn((B, h, N, D), generator=g).to(dtype) for h in (H, Hkv, Hkv)]

    def check(q, k, v, new, o, lse):
        for b in range(B):
            n0 = len(seqs[b])
            pos = torch.arange(n0, n0 + new[b])[None]
            seqs[b] += [(k[b, :, i], v[b, :, i]) for i in range(new[b])]
            if not seqs[b] or new[b] == 0:
                assert new[b] > 0 or (o[b, :, new[b]:] == 0).all()
                continue
            # rounded to 16 bits after the turn, as the cache and the queries are
            turned = lambda x, p: torch.tensor(turn_oracle(x, grid(p))).to(dtype)  # noqa: E731
            n = len(seqs[b])
            ks = turned(torch.stack([t[0] for t in seqs[b]], 1)[None], torch.arange(n)[None])
            vs = torch.stack([t[1] for t in seqs[b]], 1)[None]
            qs = turned(q[b:b + 1, :, :new[b]], pos)
            ro, rl, bo, bl = sorc.scored_fwd(qs, ks, vs, scale, seen=lambda z: sorc.visible(
                new[b], n, causal=True, window=window, sinks=sinks), dtype=dtype)
            # a turned value next to a border may round the other way: half a step of q and k more
            slack = 2 * sorc.HALF_STEP[dtype] * 2 * float(qs.float().norm(dim=-1).max() * ks.float().norm(dim=-1).max()) * scale
            within(lse[b:b + 1, :, :new[b]], rl, bl + slack, "lse")
            within(o[b:b + 1, :, :new[b]], ro, bo + 2 * slack * float(vs.abs().max()), "o")
            assert (o[b, :, new[b]:] == 0).all()

    def turn_oracle(x, positions):
        y = x.double().numpy().copy()
        for a in range(3):
            t = sorc.rotary(x, positions[a], freqs)
            pairs = (axes.cpu() == a).nonzero().flatten().numpy()
            for at in (pairs, pairs + D // 2):
                y[..., at] = t[..., at]
        return y

    # prefill
    x, new = draw(N0), [70, 33, 0]
    check(*x, new, *step(*(t.cuda() for t in x), i32(new), N0))
    # single tokens
    q1, k1, v1 = (torch.empty((B, h, 1, D), dtype=dtype, device="cuda") for h in (H, Hkv, Hkv))
    ones = i32([1, 1, 1])

    def one():
        return step(q1, k1, v1, ones, 1)

    if captured:
        warm = [t.clone() for t in (stack, count, table, lens, kc, vc)]
        for t in (q1, k1, v1):
            t.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            one()
        torch.cuda.current_stream().wait_stream(side)
        for t, w in zip((stack, count, table, lens, kc, vc), warm):
            t.copy_(w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = one()
        run = lambda: (graph.replay(), res)[1]  # noqa: E731
    else:
        run = one
    for i in range(40):
        if i == 20:  # sequence 0 ends; another takes its place with the next token
            fa.cache_release(stack, count, table, lens, torch.tensor([True, False, False], device="cuda"), page,
                             out=(lens, count))
            seqs[0] = []
        x = draw(1)
        for t, s in zip((q1, k1, v1), x):
            t.copy_(s)
        check(*x, [1, 1, 1], *run())
    assert lens.tolist() == [len(s) for s in seqs]
    held = sum(-(-len(s) // page) for s in seqs)
    assert count.tolist() == [stack.numel() - held]
    taken = [p for b in range(B) for p in table[b, :-(-len(seqs[b]) // page)].tolist()]
    assert sorted(taken + stack[:count.item()].tolist()) == list(range(stack.numel()))
    assert fa.device_status() == 0


# Sizes on both sides of the choice between one block for the call and two launches.
@pytest.mark.parametrize("B,max_pages", [(1, 256), (1, 257), (32, 256), (31, 129), (32, 257), (33, 31), (17, 1)])
def test_release_in_one_block_and_in_several(B, max_pages):
    rng = random.Random(7 * B + max_pages)
    page = 4
    for spoil, share in ((False, 0.5), (True, 1.0)):
        lens = [rng.choice([0, 1, page * max_pages, rng.randint(0, page * max_pages)]) for _ in range(B)]
        stack, count, table, pages = pool(rng, B, max_pages, page, lens, 3, spoil)
        done = [rng.random() < share for _ in range(B)]
        for c in (count, -2, pages + 9):
            for in_place in (False, True):
                wl, wc, ws = orc.release(stack, c, table, lens, done, page)
                s, k, t, n = i32(stack), i32([c]), i32(table), i32(lens)
                got = fa.cache_release(s, k, t, n, torch.tensor(done, device="cuda"), page, out=(n, k) if in_place else None)
                assert got[0].tolist() == wl and got[1].tolist() == [wc] and s.tolist() == ws and t.tolist() == table
