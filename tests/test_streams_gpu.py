"""Calls on a stream of their own beside queued work of the current stream: the memory of what they return, and of
their workspaces, is neither read nor written by that work."""

import pytest
import torch

import attention_sm_flashattention_gb300 as fa
from attention_sm_flashattention_gb300.inputs import make_inputs, make_paged_inputs
from test_scored_gpu import doc_ids

pytestmark = pytest.mark.gpu
WAIT = 30_000_000  # cycles that the current stream is busy for, about 15 ms


def calls(seed):
    """name -> call(stream): everything that allocates."""
    q, k, v, do = (t.cuda() for t in make_inputs(2, 8, 1024, 64, seed))
    o, lse = fa.fwd(q, k, v)
    so, sl = fa.fwd_scored(q, k, v, softcap=9.0)
    pq, kc, vc, table, ctx = (t.cuda() for t in make_paged_inputs(8, 8, 2, 64, [1500] * 8, 64, 64, seed))
    sel = torch.arange(8, dtype=torch.int32, device="cuda").repeat(8, 2, 1)
    pages, count = table[:, None, :8].repeat(1, 2, 1).contiguous(), torch.full((8, 2), 8, dtype=torch.int32, device="cuda")
    pos, (freqs, _) = torch.arange(seed, seed + 1024, device="cuda"), fa.rotary_freqs(64)
    ids = doc_ids(64, 4096, seed, 100).cuda()
    slots = torch.arange(2 * 1024, device="cuda").reshape(2, 1024)
    cache = [torch.zeros((32, 64, 8, 64), dtype=q.dtype, device="cuda") for _ in range(2)]
    return {
        "fwd": lambda s: fa.fwd(q, k, v, stream=s),
        "bwd": lambda s: fa.bwd(q, k, v, o, do, lse, stream=s),
        "fwd_paged": lambda s: fa.fwd_paged(pq, kc, vc, table, ctx, stream=s),
        "fwd_paged_split": lambda s: fa.fwd_paged(pq, kc, vc, table, ctx, splits=4, stream=s),
        "fwd_sparse": lambda s: fa.fwd_sparse(pq, kc, vc, pages, sel, count, ctx, stream=s),
        "fwd_scored": lambda s: fa.fwd_scored(q, k, v, softcap=9.0, stream=s),
        "bwd_scored": lambda s: fa.bwd_scored(q, k, v, so, do, sl, softcap=9.0, stream=s),
        "fwd_paged_scored": lambda s: fa.fwd_paged_scored(pq, kc, vc, table, ctx, stream=s, splits=4),
        "key_ranges": lambda s: (fa.key_ranges(4096, 4096, doc_ids=ids, stream=s).buffer,),
        "rotary": lambda s: fa.rotary(q, k, pos, freqs, stream=s),
        "rotary_bwd": lambda s: fa.rotary_bwd(q, k, pos, freqs, stream=s),
        "rotary_and_cache": lambda s: (fa.rotary_and_cache(q, k, v, pos, freqs, slots, *cache, stream=s),),
    }


NAMES = ["fwd", "bwd", "fwd_paged", "fwd_paged_split", "fwd_sparse", "fwd_scored", "bwd_scored", "fwd_paged_scored",
         "key_ranges", "rotary", "rotary_bwd", "rotary_and_cache"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_queued_work_still_reads_is_left_alone(name):
    call = calls(81)[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in want]
    sizes += [sum(sizes), 8 * 2 * 8 * 1024, 4 * 4 * 8 * 8 * 64 * 65]  # workspaces too
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    copies = [torch.zeros_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    for c, t in zip(copies, held):
        c.copy_(t)
    del held, t  # freed, and read by the copies that wait behind the sleep
    got = call(side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(bool((c == 7).all()) for c in copies)


@pytest.mark.parametrize("name", NAMES)
def test_results_may_be_freed_while_the_current_stream_still_reads_them(name):
    first, second = calls(82)[name], calls(83)[name]
    want = [t.clone() for t in first(None)]
    side = torch.cuda.Stream()
    for _ in range(2):  # (the allocator's blocks of the side stream are there)
        first(side)
    torch.cuda.synchronize()
    got = first(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(WAIT)
    copies = [t.clone() for t in got]
    del got
    for _ in range(3):
        second(side)
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", [n for n in NAMES if n != "rotary_and_cache"])
def test_captured_on_a_side_stream(name):
    """A graph whose capture forks to the call's stream and joins again."""
    call = calls(84)[name]
    want = [t.clone() for t in call(None)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    call(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = call(side)
        here.wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(2):
        for t in copies:
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(copies, want):
            assert torch.equal(a, b)
